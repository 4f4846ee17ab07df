"""Tensors past 2^31 elements through the norm with rotation and the linear layers: values
at both ends and around 2^31, against fp64 on the rows that they come from."""
import numpy as np
import pytest
import torch
from test_gpu_linear import check_backward, check_forward
from test_gpu_norm_rope import check_backward as norm_backward
from test_gpu_norm_rope import check_forward as norm_forward

import block_sparse_attention_tsr_gb300 as tsr

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()
    yield
    torch.cuda.empty_cache()


def test_norm_rope_past_2_31():
    B, H, N, d, dims = 2, 5, 1 << 21, 128, (44, 42, 42)
    grid = (128, 128, 128)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((B, H, N, d), generator=g, device="cuda", dtype=BF)
    w = torch.randn((d,), generator=g, device="cuda")
    y = tsr.tsr_norm_rope(x, w, dims, grid=grid)
    rows = torch.tensor([0, 1, 2 ** 20, 2 ** 21 - 2, 2 ** 21 - 1])
    pos = np.stack(np.unravel_index(rows.numpy(), grid), 1)
    check = lambda a, b: norm_forward(a, w, b, pos, dims)
    check(x[:, :, rows], y[:, :, rows])
    # the gradient in place of dout, at the same places
    dy = y
    want = [tsr.tsr_norm_rope_backward(dy[b:, h:h + 1, r:r + 1][:1], x[b:, h:h + 1, r:r + 1][:1], w, dims,
                                       positions=torch.tensor(pos[i:i + 1], dtype=torch.int32, device="cuda"))[0].clone()
            for i, r in enumerate(rows.tolist()) for b, h in ((0, 0), (1, 4))]
    dx, dw = tsr.tsr_norm_rope_backward(dy, x, w, dims, grid=grid, out=dy)
    got = [dx[b:b + 1, h:h + 1, r:r + 1] for r in rows.tolist() for b, h in ((0, 0), (1, 4))]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.isfinite(dw).all()


def test_linear_past_2_31():
    T, K, M = (1 << 18) + 77, 64, 8264
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=BF)
    x, w, b = rand(T, K), rand(M, K) * 0.125, rand(M)
    assert T * M > 2 ** 31
    out, pre = tsr.tsr_linear(x, w, b, activation="silu", pre=True)
    at = torch.tensor([0, 255, 256, 2 ** 31 // M, 2 ** 31 // M + 1, T - 78, T - 2, T - 1])
    check_forward(out[at], x[at], w, b, "silu", None, pre[at])
    # rows of ones with few others: dweight and dbias have an exact form
    dout = out
    dout.zero_()
    dout[at] = rand(len(at), M)
    dx, dw, db = tsr.tsr_linear_backward(dout, x, w, activation="silu", pre=pre)
    check_backward((dx[at], dw, db), dout[at], x[at], w, "silu", pre[at], norm=False)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[at.cuda()] = False
    assert not dx[rest].any()


def test_norm_rope_gradients_past_2_31():
    """Against the formulas: rows of gradients around 2^31 elements and at both ends, all other
    rows zero, so that dweight is the sum of theirs alone and dx zero everywhere else."""
    B, H, N, d, dims = 2, 5, 1 << 21, 128, (44, 42, 42)
    grid = (128, 128, 128)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((B, H, N, d), generator=g, device="cuda", dtype=BF)
    w = torch.randn((d,), generator=g, device="cuda")
    rows = torch.tensor([0, 1, 2 ** 20 - 1, 2 ** 20, 2 ** 21 - 2, 2 ** 21 - 1])
    at = rows.cuda()
    dy = torch.zeros_like(x)
    dy[:, :, at] = torch.randn((B, H, len(rows), d), generator=g, device="cuda", dtype=BF)
    pos = np.stack(np.unravel_index(rows.numpy(), grid), 1)
    dx, dw = tsr.tsr_norm_rope_backward(dy, x, w, dims, grid=grid)
    norm_backward(dy[:, :, at], x[:, :, at], w, dx[:, :, at], dw, pos, dims)
    dx[:, :, at] = 0
    assert not dx.any()
