"""Tensors whose element offsets pass 2^31: the first and last heads of a call have
to equal, bit for bit, calls on those heads alone."""
import pytest
import torch

import block_sparse_attention_tsr_gb300 as tsr

pytestmark = pytest.mark.gpu

B, H, N, D = 1, 132, 131072, 128          # 2.2e9 elements, 4.4 GB a tensor


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()
    yield
    torch.cuda.empty_cache()


def make(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty((B, H, N, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g)


def heads(t, h):
    return t[:, h:h + 1].contiguous()


def mask(blocks, h):
    return tsr.make_mask(tsr.UNIFORM, B, h, N, D, bq=4096, bk=4096, blocks=blocks.contiguous())


def test_rotation_and_selection():
    q, k = make(1), make(2)
    grid, dims = (128, 32, 32), (44, 42, 42)
    r = tsr.tsr_rope(q, dims, grid=grid)
    token_major = torch.empty((B, N, H, D), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    tsr.tsr_rope_backward(r, dims, grid=grid, out=token_major)
    sel = tsr.tsr_block_select(q, k, 9, bq=512, bk=256, diagonal=True)
    for h in (0, 127, H - 1):
        one = tsr.tsr_rope(heads(q, h), dims, grid=grid)
        assert torch.equal(r[:, h:h + 1], one)
        assert torch.equal(token_major[:, h:h + 1], tsr.tsr_rope_backward(one, dims, grid=grid))
        assert torch.equal(sel[:, h:h + 1], tsr.tsr_block_select(heads(q, h), heads(k, h), 9, bq=512, bk=256,
                                                                 diagonal=True))


def test_backward():
    q, k, v, do = (make(s) for s in (1, 2, 3, 4))
    n = N // 4096
    blocks = torch.zeros((B, H, n, n), dtype=torch.uint8, device="cuda")
    i = torch.arange(n, device="cuda")
    blocks[:, :, i, (i * 5) % n] = 1
    blocks[:, :, 3] = 0
    out, lse = tsr.tsr_bsa_forward(q, k, v, tsr.tsr_plan(mask(blocks, H)))
    plan = tsr.tsr_backward_plan(mask(blocks, H))
    got = tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan)
    torch.cuda.synchronize()
    plan.device_status()
    for h in (0, 127, H - 1):
        one = tsr.tsr_bsa_backward(*(heads(t, h) for t in (q, k, v, out)), heads(lse, h), heads(do, h),
                                   tsr.tsr_backward_plan(mask(blocks[:, h:h + 1], 1)))
        for a, b in zip(got, one):
            assert torch.equal(a[:, h:h + 1], b)
