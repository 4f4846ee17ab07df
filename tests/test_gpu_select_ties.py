"""Equal scores between key blocks that hold the same rows in another order: the block
of the lowest index is kept.  Everything is integers here (a bf16 value is a whole
number up to 255 * 2^14, a block's sum below 2^29, so past the 24 bits of fp32), and
so are the expected scores: sums of q over a block times sums of k, int64, all blocks
being equally long."""
import numpy as np
import pytest
import torch

import block_sparse_attention_tsr_gb300 as tsr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()


def whole(r, shape, shift):
    x = r.integers(128, 256, shape) * r.choice([-1, 1], shape)
    return x << r.integers(0, shift + 1, shape)


def select(sq, sk, keep):
    s = np.einsum("hid,hjd->hij", sq, sk)                       # int64: exact
    order = np.argsort(-s, axis=2, kind="stable")
    out = np.zeros(s.shape, np.uint8)
    np.put_along_axis(out, order[:, :, :keep], 1, axis=2)
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("b,n", [(48, 200), (80, 120), (24, 700), (300, 20), (64, 60)])
def test_permuted_rows_tie(b, n, d):
    """n / 2 pairs of key blocks, the second of each the first's rows shuffled; an odd
    `keep` cuts a pair in every row."""
    H, r = 2, np.random.default_rng(b + d)
    k = whole(r, (H, n // 2, b, d), 14)
    other = np.stack([np.stack([blk[r.permutation(b)] for blk in head]) for head in k])
    k = np.concatenate([k, other], 1)
    q = whole(r, (H, n, b, d), 0)
    sq, sk = q.sum(2), k.sum(2)
    assert np.array_equal(sk[:, : n // 2], sk[:, n // 2:])
    qt, kt = (torch.from_numpy(x.reshape(1, H, n * b, d).astype(np.float32)).bfloat16().cuda() for x in (q, k))
    assert np.array_equal(kt.double().cpu().numpy().reshape(k.shape), k)
    for keep in (1, 7, n // 2 - 1):
        got = tsr.tsr_block_select(qt, kt, keep, bq=b, bk=b)[0].cpu().numpy()
        assert np.array_equal(got, select(sq, sk, keep))
