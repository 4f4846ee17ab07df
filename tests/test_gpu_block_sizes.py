"""UNIFORM masks whose blocks are longer than any sequence, up to 2^31 - 1 tokens (the
sizes tsr_block_select takes): such a block holds all N tokens, so every call has to
give, bit for bit, what it gives for blocks of 4,096 tokens at N = 300."""
import ctypes

import pytest
import torch

import block_sparse_attention_tsr_gb300 as tsr
import workloads as W

pytestmark = pytest.mark.gpu

B, H, N, D = 1, 3, 300, 64
HUGE = [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 64), (64, 2 ** 31 - 1), (2 ** 31 - 200, 2 ** 28 + 5), (1 << 24, 1 << 30)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()


def blocks_of(bq, bk):
    """Heads that differ: head 0 sees nothing, head 1 all, head 2 every second block."""
    b = torch.zeros((B, H, W.cdiv(N, bq), W.cdiv(N, bk)), dtype=torch.uint8)
    b[:, 1] = 1
    b[:, 2].view(-1)[::2] = 1
    return b.cuda()


def mask_of(bq, bk, blocks):
    return tsr.make_mask(tsr.UNIFORM, B, H, N, D, bq=bq, bk=bk, blocks=blocks)


def small(b):
    return b if b == 64 else 4096


@pytest.mark.parametrize("bq,bk", HUGE)
def test_forward_backward_and_counts(bq, bk):
    q, k, v = (t.cuda() for t in W.qkv(B, H, N, D, 1))
    do = W.qkv(B, H, N, D, 2)[0].cuda()
    got = []
    for x, y in ((bq, bk), (small(bq), small(bk))):
        blocks = blocks_of(x, y)
        mask = mask_of(x, y, blocks)
        opts = {"bn": 64, "orient": tsr.ORIENT_ROWS}
        plan = tsr.tsr_plan(mask, opts)
        st = plan.stats()
        assert st["n_logical_total"] == blocks.numel() and st["n_logical_on"] == int(blocks.sum())
        out, lse = tsr.tsr_bsa_forward(q, k, v, plan)
        plan.update(mask)
        again, _ = tsr.tsr_bsa_forward(q, k, v, plan)
        assert torch.equal(out, again)
        bwd = tsr.tsr_backward_plan(mask)
        got.append((out, lse, *tsr.tsr_bsa_backward(q, k, v, out, lse, do, bwd)))
        bwd.device_status()
        assert torch.all(out[:, 0] == 0) and torch.all(lse[:, 0] == -float("inf"))
        assert torch.isfinite(lse[:, 1]).all() and all(torch.all(t[:, 0] == 0) for t in got[-1][2:])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("bq,bk", HUGE)
def test_one_call_entry_points(bq, bk):
    q, k, v = W.qkv(B, H, N, D, 3)
    L = tsr.lib()
    f = L.tsr_attention_noalloc
    f.argtypes, f.restype = [ctypes.c_void_p] * 7, ctypes.c_int
    got = []
    for x, y in ((bq, bk), (small(bq), small(bk))):
        blocks = blocks_of(x, y)
        out, lse = torch.empty_like(q), torch.empty((B, H, N))
        tsr.tsr_attention_host(tsr.UNIFORM, B, H, N, D, q, k, v, out, lse, bq=x, bk=y, blocks=blocks.cpu())
        dq, dk, dv, do = q.cuda(), k.cuda(), v.cuda(), torch.empty_like(q, device="cuda")
        dl = torch.empty((B, H, N), device="cuda")
        mask = mask_of(x, y, blocks)
        st = f(ctypes.byref(mask.struct), *(t.data_ptr() for t in (dq, dk, dv, do, dl)),
               torch.cuda.current_stream().cuda_stream)
        assert st == 0, L.tsr_last_error()
        assert torch.all(do[:, 0] == 0) and torch.isfinite(dl[:, 1]).all()
        got.append((out, lse, do, dl))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("b", [2 ** 31 - 1, 2 ** 24])
def test_selection_plans_and_attends(b):
    """The mask that a selection of such blocks makes."""
    q, k, v = (t.cuda() for t in W.qkv(B, H, N, D, 4))
    blocks = tsr.tsr_block_select(q, k, 1, bq=b, bk=b)
    assert blocks.shape == (B, H, 1, 1) and torch.all(blocks == 1)
    out, _ = tsr.tsr_bsa_forward(q, k, v, tsr.tsr_plan(mask_of(b, b, blocks)))
    want, _ = tsr.tsr_bsa_forward(q, k, v, tsr.tsr_plan(mask_of(4096, 4096, blocks)))
    assert torch.equal(out, want)
