"""The norm of every head's row with the position rotation, and its gradients, on the GPU
against the definition in fp64.

Tolerances, from the arithmetic (u: half a step of the output's type, 2^-8 bf16, 2^-11
fp16, 2^-24 fp32):
  r = rsqrt(mean + eps): the sum of squares is 16 fused steps and 5 butterfly adds at most
    (128 lanes x pairs: below 25 * 2^-24), its half enters r, rsqrtf is within 2 ulp:
    1.2e-6 of r.
  y: that, two products and the rotation's 1e-6 (|a| + |b|): 2.5e-6 (|a| + |b|).
  dx = r (g w - x r^2 S / d): r enters three times (3.6e-6), g's rotation 1e-6, the sum S
    1.5e-6, four products 2.4e-7: 8e-6 of r (|g| |w| + |x| r^2 / d sum |g| |w| |x|).
  dw: g and xhat are off by 2.2e-6; of the sums' adds a term meets at most 2 H in its
    thread, 256 in its CTA and 51 over the CTAs (one or two items a CTA at these sizes):
    340 * 2^-24 = 2e-5 of sum |g| |xhat|, and u of the result.
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_tsr_gb300 as tsr
from oracle import layer

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()


def make(shape, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype).cuda()


def f64(t):
    return t.double().cpu().numpy()


def positions(pos, B):
    """Positions for the oracle's [..., N, d]: [N, axes] alike for every batch, or per batch."""
    return [pos[b] if pos.ndim == 3 else pos for b in range(B)]


def check_forward(x, w, got, pos, dims, theta=1e4, halves=False, eps=EPS):
    wd = np.ones(x.shape[-1]) if w is None else f64(w)
    assert got.dtype == x.dtype and got.shape == x.shape
    for b, p in enumerate(positions(pos, x.shape[0])):
        want, size = layer.norm_rotate(f64(x[b]), wd, p, dims, eps, theta, halves)
        tol = HALF_STEP[x.dtype] * np.abs(want) + 2.5e-6 * size + TINY[x.dtype]
        assert np.all(np.abs(f64(got[b]) - want) <= tol)


def check_backward(dy, x, w, dx, dw, pos, dims, theta=1e4, halves=False, eps=EPS, adds=2e-5):
    wd = np.ones(x.shape[-1]) if w is None else f64(w)
    total, total_size = 0.0, 0.0
    for b, p in enumerate(positions(pos, x.shape[0])):
        want, part, size, part_size = layer.norm_rotate_gradients(f64(dy[b]), f64(x[b]), wd, p, dims, eps, theta, halves)
        assert np.all(np.abs(f64(dx[b]) - want) <= HALF_STEP[x.dtype] * np.abs(want) + 8e-6 * size + TINY[x.dtype])
        total, total_size = total + part, total_size + part_size
    if w is not None:
        assert dw.dtype == w.dtype and dw.shape == w.shape
        assert np.all(np.abs(f64(dw) - total) <= HALF_STEP[w.dtype] * np.abs(total) + adds * total_size + TINY[w.dtype])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("B,H,grid,d,dims", [
    (1, 2, (4, 6, 5), 64, (16, 24, 24)),
    (2, 3, (3, 7, 5), 128, (44, 42, 42)),      # axes that end inside a 16-byte piece
    (1, 5, (2, 3, 11), 128, (32, 48, 48)),
    (1, 11, (1, 1, 1), 64, (20, 20, 20)),      # one token, channels left over
    (3, 1, (7, 9), 32, (8, 16)),
    (1, 2, (101,), 256, (256,)),
    (2, 9, (13,), 256, (128,)),                # half of the widest head
    (1, 3, (5, 2, 2, 3), 40, (8, 2, 4, 6)),    # rows of five 16-byte pieces
    (1, 4, (3, 3, 3), 6, (2, 2, 2)),
    (1, 13, (5,), 2, (2,)),
])
def test_layouts_against_the_definition(B, H, grid, d, dims, halves, dtype):
    N = int(np.prod(grid))
    pos = layer.coordinates(grid)
    x = make((B, N, H, d), dtype, 1, 3.0).transpose(1, 2)    # token-major in, head-major out
    w = make((d,), torch.float32 if halves else dtype, 2)
    got = tsr.tsr_norm_rope(x, w, dims, grid=grid, halves=halves)
    assert got.is_contiguous()
    check_forward(x, w, got, pos, dims, halves=halves)
    dy = make((B, H, N, d), dtype, 3)
    back = torch.empty((B, N, H, d), dtype=dtype, device="cuda").transpose(1, 2)
    dx, dw = tsr.tsr_norm_rope_backward(dy, x, w, dims, grid=grid, halves=halves, out=back)
    assert dx is back
    check_backward(dy, x, w, dx, dw, pos, dims, halves=halves)


@pytest.mark.parametrize("halves", [False, True])
def test_far_positions_per_batch(halves):
    B, H, N, d, dims = 2, 3, 257, 64, (16, 24, 16)
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-10 ** 6, 10 ** 6, (B, N, 3), generator=g, dtype=torch.int32)
    x, w, dy = make((B, H, N, d), torch.float32, 1), make((d,), torch.float32, 2), make((B, H, N, d), torch.float32, 3)
    for p in (pos, pos[1]):
        kw = dict(positions=p.cuda().contiguous(), theta=5e5, halves=halves)
        check_forward(x, w, tsr.tsr_norm_rope(x, w, dims, **kw), p.numpy(), dims, 5e5, halves)
        dx, dw = tsr.tsr_norm_rope_backward(dy, x, w, dims, **kw)
        check_backward(dy, x, w, dx, dw, p.numpy(), dims, 5e5, halves)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("offset", [1, 2, 4, 8])
def test_unaligned_and_strided(offset, halves):
    """Rows that start at any element, with gaps, inside one fused projection; the
    memory between the rows stays as it was."""
    B, H, grid, d, dims, N = 2, 3, (3, 5, 2), 64, (16, 24, 24), 30
    pos = layer.coordinates(grid)
    buf = make((B, N, 3, H, d + offset), torch.bfloat16, 2)
    x = buf[:, :, 1, :, offset:].transpose(1, 2)
    w = make((d + 1,), torch.bfloat16, 5)[1:]
    out = torch.full((B, H, N, d + 2 * offset), 7.0, dtype=torch.bfloat16, device="cuda")
    view = out[..., offset:offset + d]
    tsr.tsr_norm_rope(x, w, dims, grid=grid, halves=halves, out=view)
    check_forward(x, w, view, pos, dims, halves=halves)
    assert torch.all(out[..., :offset] == 7.0) and torch.all(out[..., offset + d:] == 7.0)
    dy = make((B, N, H, d + offset), torch.bfloat16, 6)[..., offset:].transpose(1, 2)
    out.fill_(7.0)
    _, dw = tsr.tsr_norm_rope_backward(dy, x, w, dims, grid=grid, halves=halves, out=view)
    check_backward(dy, x, w, view, dw, pos, dims, halves=halves)
    assert torch.all(out[..., :offset] == 7.0) and torch.all(out[..., offset + d:] == 7.0)


@pytest.mark.parametrize("dims", [(16, 24, 24), (6, 10, 14)])
def test_several_tensors_in_place_and_without_weight(dims):
    """Q and K of different head counts, K without a weight, in one launch; in place."""
    grid, N, d = (4, 3, 5), 60, 64
    pos = layer.coordinates(grid)
    q, k = make((2, 7, N, d), torch.bfloat16, 4), make((2, N, 2, d), torch.bfloat16, 5).transpose(1, 2)
    w = make((d,), torch.float32, 6)
    a, b = tsr.tsr_norm_rope([q, k], [w, None], dims, grid=grid)
    check_forward(q, w, a, pos, dims)
    check_forward(k, None, b, pos, dims)
    ga, gb = make(q.shape, torch.bfloat16, 7), make(k.shape, torch.bfloat16, 8)
    (dq, dk), (dwq, dwk) = tsr.tsr_norm_rope_backward([ga, gb], [q, k], [w, None], dims, grid=grid)
    assert dwk is None
    check_backward(ga, q, w, dq, dwq, pos, dims)
    check_backward(gb, k, None, dk, None, pos, dims)
    again = tsr.tsr_norm_rope_backward([ga, gb], [q, k], [w, None], dims, grid=grid)
    assert torch.equal(again[1][0], dwq) and torch.equal(again[0][0], dq)       # the same bits
    # in place: the gradient over dout, the output over x
    g2 = ga.clone()
    assert torch.equal(tsr.tsr_norm_rope_backward(g2, q, w, dims, grid=grid, out=g2)[0], dq)
    q2, k2 = q.clone(), k.clone()
    tsr.tsr_norm_rope((q2, k2), (w, None), dims, grid=grid, out=(q2, k2))
    assert torch.equal(q2, a) and torch.equal(k2, b)
    # a broadcast input: a gradient for each of its uses
    one = make((1, 1, N, d), torch.bfloat16, 9).expand(2, 7, N, d)
    check_forward(one, w, tsr.tsr_norm_rope(one, w, dims, grid=grid), pos, dims)
    dx, dw = tsr.tsr_norm_rope_backward(ga, one, w, dims, grid=grid)
    check_backward(ga, one, w, dx, dw, pos, dims)


def test_many_rows_and_one_row():
    """Enough tokens that a CTA takes many items, and a single row."""
    grid, d, dims = (21, 30, 13), 128, (44, 42, 42)
    N = 8190
    pos = layer.coordinates(grid)
    x, w, dy = make((1, 2, N, d), torch.bfloat16, 1), make((d,), torch.float32, 2), make((1, 2, N, d), torch.bfloat16, 3)
    check_forward(x, w, tsr.tsr_norm_rope(x, w, dims, grid=grid), pos, dims)
    dx, dw = tsr.tsr_norm_rope_backward(dy, x, w, dims, grid=grid)
    check_backward(dy, x, w, dx, dw, pos, dims)
    x1, dy1 = x[:, :1, :1], dy[:, :1, :1]
    one = tsr.tsr_norm_rope_backward(dy1, x1, w, dims, grid=(1, 1, 1))
    check_backward(dy1, x1, w, *one, pos[:1], dims)


def test_gradient_against_differences():
    """<dy, f(x + h v) - f(x - h v)> / 2h against <dx, v>, and the same for the weight, in
    fp32: the quotient's truncation is h^2 of f''' (below 1e-5 of the norms' product at h =
    2^-8), its rounding 2^-24 / h of |f| (2e-5); 1e-4 covers both."""
    grid, dims, d, h = (3, 4, 5), (10, 12, 14), 40, 2.0 ** -8
    x, v, dy = (make((2, 3, 60, d), torch.float32, s) for s in (7, 8, 9))
    w, vw = make((d,), torch.float32, 10), make((d,), torch.float32, 11)
    f = lambda x, w: tsr.tsr_norm_rope(x, w, dims, grid=grid, halves=True).double()
    dx, dw = tsr.tsr_norm_rope_backward(dy, x, w, dims, grid=grid, halves=True)
    size = dy.double().norm() * f(x, w).norm()
    lhs = ((f(x + h * v, w) - f(x - h * v, w)) * dy.double()).sum() / (2 * h)
    assert abs(lhs - (dx.double() * v.double()).sum()) <= 1e-4 * size
    lhs = ((f(x, w + h * vw) - f(x, w - h * vw)) * dy.double()).sum() / (2 * h)
    assert abs(lhs - (dw.double() * vw.double()).sum()) <= 1e-4 * size


def test_zero_rows_large_rows_and_values_that_are_not_finite():
    grid, dims, d = (2, 3), (8, 4), 16
    x = make((1, 2, 6, d), torch.bfloat16)
    x[0, 0, 1] = 0
    x[0, 0, 2] *= 2.0 ** 50
    x[0, 1, 3, 5] = float("inf")
    x[0, 1, 4, 13] = float("nan")
    w = make((d,), torch.float32, 1)
    y = tsr.tsr_norm_rope(x, w, dims, grid=grid)
    good = torch.ones(1, 2, 6, dtype=torch.bool)
    good[0, 1, 3] = good[0, 1, 4] = False
    want, size = layer.norm_rotate(f64(x[0, 0]), f64(w), layer.coordinates(grid), dims, EPS)
    assert np.all(np.abs(f64(y[0, 0]) - want) <= 2.0 ** -8 * np.abs(want) + 2.5e-6 * size)
    assert torch.all(y[0, 0, 1] == 0)
    assert torch.isfinite(y.cpu()[good]).all()                    # other rows do not hear of them
    assert torch.isnan(y[0, 1, 4]).all()                          # a NaN is in its row's sum
    # an infinity makes r = 0: its own pair is NaN, the rest of its row 0
    row = y[0, 1, 3].cpu()
    assert torch.isnan(row[4:6]).all() and (row[:4] == 0).all() and (row[6:] == 0).all()


def test_graph_capture_and_another_stream():
    grid, dims = (4, 4, 4), (16, 24, 24)
    x, dy, w = make((1, 3, 64, 64), torch.bfloat16), make((1, 3, 64, 64), torch.bfloat16, 1), make((64,), torch.bfloat16, 2)
    want, want_b = tsr.tsr_norm_rope(x, w, dims, grid=grid), tsr.tsr_norm_rope_backward(dy, x, w, dims, grid=grid)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = tsr.tsr_norm_rope(x, w, dims, grid=grid, stream=s)
    got_b = tsr.tsr_norm_rope_backward(dy, x, w, dims, grid=grid, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(got_b, want_b))
    out, graph = torch.empty_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tsr.tsr_norm_rope(x, w, dims, grid=grid, out=out)
        dx, dw = tsr.tsr_norm_rope_backward(dy, x, w, dims, grid=grid)
    x.mul_(-2)
    dy.mul_(3)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, tsr.tsr_norm_rope(x, w, dims, grid=grid))
    a, b = tsr.tsr_norm_rope_backward(dy, x, w, dims, grid=grid)
    assert torch.equal(dx, a) and torch.equal(dw, b)


def test_binding_refusals():
    x, w = make((1, 2, 12, 16), torch.bfloat16), make((16,), torch.bfloat16)
    for bad in (make((8,), torch.bfloat16), make((16,), torch.float16), make((1, 16), torch.bfloat16), [w, w], w.cpu()):
        with pytest.raises(ValueError):
            tsr.tsr_norm_rope(x, bad, (8, 8), grid=(3, 4))
    for t in (x.cpu(), x.double(), x.transpose(2, 3), x[0], [x, x.float()]):
        with pytest.raises((ValueError, tsr.TsrError)):
            tsr.tsr_norm_rope(t, None, (8, 8), grid=(3, 4))
    with pytest.raises(ValueError):
        tsr.tsr_norm_rope([x, x.clone()], [w, w.float()], (8, 8), grid=(3, 4))
    with pytest.raises(tsr.TsrError):
        tsr.tsr_norm_rope(x, w, (8, 8), grid=(3, 4), eps=0.0)
    dy = x.clone()
    for bad in (dict(dout=dy[:, :1]), dict(dout=dy.float()), dict(out=dy.float()), dict(dweight=w.float()),
                dict(x=[x, dy], dout=[x.clone(), x.clone()], weight=[w, w])):
        args = dict(dout=dy, x=x, weight=w)
        args.update(bad)
        with pytest.raises(ValueError):
            tsr.tsr_norm_rope_backward(axis_dims=(8, 8), grid=(3, 4), **args)
    with pytest.raises(tsr.TsrError):
        tsr.tsr_norm_rope_backward(dy, x, w, (8, 8), grid=(3, 4), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("halves,d,dims", [(False, 64, (16, 24, 24)), (True, 64, (16, 24, 24)), (False, 6, (2, 2))])
@pytest.mark.parametrize("eps", [2.0 ** -149, 2.0 ** -140, 2.0 ** -126, 2.0 ** -100])
def test_gradient_at_the_smallest_eps(eps, halves, d, dims, dtype):
    """Any eps > 0 of fp32 is taken: a row of zeros has r = eps^-1/2, up to 2^74.5, and the
    gradient r (g o w), finite in these types; rows beside it of 2^-55 to 2^55 (their squares
    stay inside fp32's normal range)."""
    grid, H = (2, 3, 2)[:len(dims)], 5
    N, pos = int(np.prod(grid)), layer.coordinates(grid)
    x, dy, w = make((1, H, N, d), dtype, 1), make((1, H, N, d), dtype, 2), make((d,), torch.float32, 3)
    x[0, :, 0] = 0
    x[0, 2] = 0
    x[0, 3] = torch.sign(x[0, 3]) * 2.0 ** -55
    x[0, 4] *= 2.0 ** 55
    kw = dict(eps=eps, grid=grid, halves=halves)
    y = tsr.tsr_norm_rope(x, w, dims, **kw)
    assert torch.all(y[0, :, 0] == 0) and torch.all(y[0, 2] == 0)
    check_forward(x, w, y, pos, dims, halves=halves, eps=eps)
    dx, dw = tsr.tsr_norm_rope_backward(dy, x, w, dims, **kw)
    assert torch.isfinite(dx).all()
    check_backward(dy, x, w, dx, dw, pos, dims, halves=halves, eps=eps)
