"""Block selection on the GPU against exact arithmetic: block means and scores in
fp64 (pairwise sums of at most 2^12 bf16 values, products of the means), a stable
sort, and no tolerance: the selected blocks have to be the same.  Random scores
differ by far more than fp64 rounding; where a test makes equal scores it makes
them of equal blocks, whose sums are the same whatever their order."""
import numpy as np
import pytest
import torch

import block_sparse_attention_tsr_gb300 as tsr
import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()


def means(x, b):
    """Block means; a block with a value that is not finite is NaN."""
    N = x.shape[2]
    with np.errstate(invalid="ignore"):
        m = np.stack([x[:, :, i:i + b].mean(2) for i in range(0, N, b)], 2)
    return np.where(np.isfinite(m), m, np.nan)


def select(q, k, keep, bq, bk, first=0, diagonal=False):
    q, k = (x.double().cpu().numpy() for x in (q, k))
    N = q.shape[2]
    with np.errstate(invalid="ignore"):
        s = np.einsum("bhid,bhjd->bhij", means(q, bq), means(k, bk))
    B, H, nq, nk = s.shape
    out = np.zeros(s.shape, np.uint8)
    for i in range(nq):
        forced = set(range(min(first, nk)))
        if diagonal:
            lo, hi = i * bq, min(N, (i + 1) * bq) - 1
            forced |= {j for j in range(nk) if j * bk <= hi and min(N, (j + 1) * bk) - 1 >= lo}
        rest = np.array([j for j in range(nk) if j not in forced], int)
        for b in range(B):
            for h in range(H):
                out[b, h, i, list(forced)] = 1
                n = keep - len(forced)
                if n > 0 and len(rest):
                    sc = np.where(np.isnan(s[b, h, i, rest]), -np.inf, s[b, h, i, rest])
                    nan = np.isnan(s[b, h, i, rest])
                    order = sorted(range(len(rest)), key=lambda r: (nan[r], -sc[r], rest[r]))
                    out[b, h, i, rest[order[:n]]] = 1
    return out


def check(q, k, keep, bq=64, bk=64, **kw):
    got = tsr.tsr_block_select(q, k, keep, bq=bq, bk=bk, **kw).cpu().numpy()
    assert np.array_equal(got, select(q, k, keep, bq, bk, **kw))
    return got


def qk(B, H, N, d, seed=0):
    return [x.cuda() for x in W.qkv(B, H, N, d, seed)[:2]]


@pytest.mark.parametrize("B,H,N,d,bq,bk,keep", [
    (1, 2, 1024, 64, 64, 64, 5),
    (2, 3, 1001, 128, 64, 64, 3),
    (1, 2, 2000, 128, 16, 16, 31),
    (1, 1, 5003, 64, 32, 48, 40),
    (1, 3, 777, 128, 200, 24, 7),
    (1, 2, 1, 64, 64, 64, 1),              # one token
    (1, 2, 15, 128, 16, 16, 1),
    (1, 1, 65, 64, 64, 16, 2),             # a block of one token
    (2, 1, 300, 64, 4096, 100, 2),         # one query block
    (1, 1, 300, 64, 100, 4096, 1),         # one key block
    (1, 1, 300, 64, 2 ** 31 - 1, 2 ** 31 - 1, 1),
    (1, 1, 20000, 64, 512, 16, 200),       # 1,250 blocks a row: the most that registers hold
    (1, 1, 21000, 128, 300, 16, 77),       # more
    (1, 1, 30000, 64, 512, 16, 700),       # rows longer than shared memory holds
    (2, 3, 40000, 64, 64, 48, 31),         # long calls: means and selection of several
    (1, 9, 32001, 128, 64, 64, 60),        # heads at once, uneven chunks of heads
])
def test_against_exact_scores(B, H, N, d, bq, bk, keep):
    q, k = qk(B, H, N, d, seed=N + keep)
    got = check(q, k, keep, bq, bk)
    assert np.all(got.sum(-1) == min(keep, got.shape[-1]))


@pytest.mark.parametrize("first,diagonal", [(0, True), (1, False), (3, True), (100, False), (6, True)])
@pytest.mark.parametrize("keep", [1, 4, 9, 50])
def test_forced_blocks(keep, first, diagonal):
    q, k = qk(1, 2, 1300, 64, 3)
    check(q, k, keep, 48, 80, first=first, diagonal=diagonal)


def test_equal_scores_go_to_the_lowest_index():
    q, k = qk(1, 2, 1024, 64, 5)
    q[0, 0, 64:128] = 0                                        # every score of a query block equal
    k[0, 1] = k[0, 1, :64].repeat(16, 1)                       # every key block equal
    check(q, k, 5)
    k[0, 0, 512:] = k[0, 0, :512]                              # pairs of equal blocks
    check(q, k, 6)
    check(torch.zeros_like(q), k, 7, bk=16, bq=256)            # all rows, 64 equal scores


def test_scores_closer_than_the_fast_bound():
    """Every score within the fast bound of every other: 2048 key blocks whose means
    differ only in channels that weigh little."""
    for bk, N in ((16, 1024), (16, 16 * 1000)):
        g = torch.Generator().manual_seed(N)
        k = torch.randn((1, 1, N, 64), generator=g) * 0.001
        k[..., 0] = 100.0
        q = torch.randn((1, 1, N, 64), generator=g) * 0.01
        q[..., 0] = 100.0
        check(q.bfloat16().cuda(), k.bfloat16().cuda(), 13, bq=512, bk=bk)


def test_small_and_large_values():
    q, k = qk(1, 2, 640, 64, 8)
    check((q.float() * 1e-20).bfloat16(), (k.float() * 1e10).bfloat16(), 3)
    check((q.float() * 1e20).bfloat16(), (k.float() * 1e20).bfloat16(), 3)     # scores past fp32
    check((q.float() * 1e-25).bfloat16(), (k.float() * 1e-25).bfloat16(), 3)   # scores below fp32


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_values_that_are_not_finite(value):
    q, k = qk(1, 3, 1100, 64, 9)
    k[0, 0, 130, 3] = value                                    # one key block of a head
    q[0, 1, 700, 60] = value                                   # one query block
    check(q, k, 4)
    check(q, k, 40, bk=16)
    check(q, k, 4, diagonal=True, first=1)


def test_cancelling_sums():
    """Means far smaller than the values they are means of."""
    q, k = qk(1, 1, 512, 64, 10)
    k[:, :, 0::2] = 0
    k[:, :, 0::2, :32] = 3.0e4
    k[:, :, 1::2, :32] = -3.0e4
    check(q, k, 3)


def test_streams_workspaces_and_graphs():
    q, k = qk(1, 2, 1500, 128, 11)
    want = tsr.tsr_block_select(q, k, 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = tsr.tsr_block_select(q, k, 6, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")     # a dirty workspace
    assert torch.equal(tsr.tsr_block_select(q, k, 6, workspace=ws), want)
    out, graph = torch.empty_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tsr.tsr_block_select(q, k, 6, out=out, workspace=ws)
    q.copy_(q.flip(2))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, tsr.tsr_block_select(q, k, 6))


def test_selected_attention_is_attention_over_the_selection():
    """select, plan, attend, against the oracle over the same blocks."""
    import oracle
    q, k, v = W.qkv(1, 2, 1500, 64, 12)
    blocks = tsr.tsr_block_select(q.cuda(), k.cuda(), 6, bq=64, bk=32, first=1, diagonal=True)
    spec = W.MaskSpec(W.MASK_UNIFORM, 1, 2, 1500, bq=64, bk=32, blocks=blocks.cpu().numpy())
    plan = tsr.tsr_plan(tsr.make_mask(tsr.UNIFORM, 1, 2, 1500, 64, bq=64, bk=32, blocks=blocks))
    out, lse = tsr.tsr_bsa_forward(q.cuda(), k.cuda(), v.cuda(), plan)
    want, want_lse = oracle.attention(spec, q, k, v)
    d = np.abs(out.float().cpu().numpy() - want)
    assert d.max() <= 2e-2 and d.mean() <= 2e-3                # as the forward's own tests
    assert np.abs(lse.cpu().numpy() - want_lse).max() <= 1e-3 * max(1.0, np.abs(want_lse).max())


def test_binding_refusals():
    q, k = qk(1, 1, 128, 64)
    for a, b, kw in ((q.float(), k, {}), (q, k[:, :, :64], {}), (q.cpu(), k, {}),
                     (q, k, dict(out=torch.empty((1, 1, 2, 3), dtype=torch.uint8, device="cuda"))),
                     (q.transpose(2, 3), k.transpose(2, 3), {})):
        with pytest.raises((ValueError, tsr.TsrError)):
            tsr.tsr_block_select(a, b, 1, **kw)
    with pytest.raises(tsr.TsrError):
        tsr.tsr_block_select(q, k, 0)
    with pytest.raises(tsr.TsrError):
        tsr.tsr_block_select(q, k, 1, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
