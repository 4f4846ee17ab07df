"""Rows of scores beyond shared memory: more strips of query blocks than resident CTAs,
whose slots of the workspace are used again and again."""
import pytest
import torch

import block_sparse_attention_tsr_gb300 as tsr
import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,H", [(26448, 10), (27001, 6)])       # 1,653 and 1,688 blocks a row
def test_many_strips_equal_one_head_at_a_time(N, H, d):
    """A head alone has at most 106 strips, a slot for each."""
    q, k = (t.cuda() for t in W.qkv(1, H, N, d, N)[:2])
    k[0, 1, 16:] = k[0, 1, :16].repeat(N // 16 + 1, 1)[: N - 16]    # equal blocks: the long way out
    kw = dict(bq=16, bk=16, first=1, diagonal=True)
    need = tsr.tsr_block_select(q, k, 40, **kw)
    ws = torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda")       # dirty: NaN scores
    assert torch.equal(tsr.tsr_block_select(q, k, 40, workspace=ws, **kw), need)
    for h in range(H):
        one = tsr.tsr_block_select(q[:, h:h + 1].contiguous(), k[:, h:h + 1].contiguous(), 40, **kw)
        assert torch.equal(need[:, h:h + 1], one)
