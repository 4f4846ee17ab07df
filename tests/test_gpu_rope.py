"""Rotary positions over several axes on the GPU against the definition in fp64.

Tolerance, from the arithmetic: the rounding to the output type is off by half a
step of the value, u |y| with u = 2^-8 (bf16), 2^-11 (fp16; half a subnormal step
2^-25 at least), 2^-24 (fp32).  Before it, the angle in half turns is one float in
[-1, 1) (2^-24 pi of a radian), sincospi is within 2 ulp (2^-22), and the two
products and their sum add 3 * 2^-24, each times at most |a| + |b|: below 1e-6
(|a| + |b|).
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_tsr_gb300 as tsr

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()


def coordinates(grid):
    return np.stack([x.ravel() for x in np.meshgrid(*[np.arange(g) for g in grid], indexing="ij")], 1)


def rotate(x, pos, dims, theta, halves, inverse):
    """[B, H, N, d] fp64, and the sum |a| + |b| of each element's pair."""
    y, size, at = x.copy(), np.zeros_like(x), 0
    pos = np.broadcast_to(pos, (x.shape[0],) + pos.shape[-2:]).astype(np.float64)
    for ax, D in enumerate(dims):
        for j in range(D // 2):
            i0, i1 = (at + j, at + D // 2 + j) if halves else (at + 2 * j, at + 2 * j + 1)
            ang = pos[:, :, ax] * theta ** (-2.0 * j / D)
            ang = (-ang if inverse else ang)[:, None]
            a, b = x[..., i0], x[..., i1]
            y[..., i0], y[..., i1] = a * np.cos(ang) - b * np.sin(ang), a * np.sin(ang) + b * np.cos(ang)
            size[..., i0] = size[..., i1] = np.abs(a) + np.abs(b)
        at += D
    return y, size


def check(x, got, pos, dims, theta=1e4, halves=False, inverse=False):
    xd = x.double().cpu().numpy()
    want, size = rotate(xd, pos, dims, theta, halves, inverse)
    tol = HALF_STEP[x.dtype] * np.abs(want) + 1e-6 * size + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)
    assert got.dtype == x.dtype and got.shape == x.shape
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
    rest = sum(dims)
    assert torch.equal(got[..., rest:], x[..., rest:])      # channels past the axes: bit for bit


def make(shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("B,H,grid,d,dims", [
    (1, 2, (4, 6, 5), 64, (16, 24, 24)),
    (2, 3, (3, 7, 5), 128, (44, 42, 42)),      # axes that end inside a 16-byte piece
    (1, 5, (2, 3, 11), 128, (32, 48, 48)),
    (1, 1, (1, 1, 1), 64, (20, 20, 20)),       # one token, channels left over
    (3, 1, (7, 9), 32, (8, 16)),
    (1, 2, (101,), 256, (256,)),
    (1, 3, (5, 2, 2, 3), 40, (8, 2, 4, 6)),
    (1, 4, (3, 3, 3), 6, (2, 2, 2)),
])
def test_layouts_against_the_definition(B, H, grid, d, dims, halves, dtype):
    N = int(np.prod(grid))
    x = make((B, N, H, d), dtype).transpose(1, 2)           # token-major in, head-major out
    got = tsr.tsr_rope(x, dims, grid=grid, halves=halves)
    assert got.is_contiguous()
    check(x, got, coordinates(grid), dims, halves=halves)
    back = torch.empty((B, N, H, d), dtype=dtype, device="cuda").transpose(1, 2)
    assert tsr.tsr_rope_backward(got, dims, grid=grid, halves=halves, out=back) is back
    check(got, back, coordinates(grid), dims, halves=halves, inverse=True)


@pytest.mark.parametrize("halves", [False, True])
def test_positions_far_and_negative(halves):
    B, H, N, d, dims = 2, 3, 257, 64, (16, 24, 16)
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-10 ** 6, 10 ** 6, (B, N, 3), generator=g, dtype=torch.int32)
    x = make((B, H, N, d), torch.float32, 1)
    check(x, tsr.tsr_rope(x, dims, positions=pos.cuda(), theta=5e5, halves=halves), pos.numpy(), dims, 5e5, halves)
    # shared by the batch
    check(x, tsr.tsr_rope(x, dims, positions=pos[0].cuda().contiguous(), halves=halves), pos[0].numpy(), dims,
          halves=halves)


def test_extreme_positions_return_to_the_start():
    """theta = 1: every pair turns by the position itself; 2^31 - 1 and -2^31 too."""
    pos = torch.tensor([[2 ** 31 - 1], [-2 ** 31], [0], [-1]], dtype=torch.int32)
    x = make((1, 1, 4, 8), torch.float32)
    check(x, tsr.tsr_rope(x, (8,), positions=pos.cuda(), theta=1.0), pos.numpy(), (8,), theta=1.0)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("offset", [1, 2, 4, 8])
def test_unaligned_and_strided(offset, halves):
    """Rows that start at any element, with gaps, inside one fused projection; the
    memory between the rows stays as it was."""
    B, H, grid, d, dims = 2, 3, (3, 5, 2), 64, (16, 24, 24)
    N = 30
    buf = make((B, N, 3, H, d + offset), torch.bfloat16, 2)
    x = buf[:, :, 1, :, offset:].transpose(1, 2)
    out = torch.full((B, H, N, d + 2 * offset), 7.0, dtype=torch.bfloat16, device="cuda")
    view = out[..., offset:offset + d]
    tsr.tsr_rope(x, dims, grid=grid, halves=halves, out=view)
    check(x, view, coordinates(grid), dims, halves=halves)
    assert torch.all(out[..., :offset] == 7.0) and torch.all(out[..., offset + d:] == 7.0)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("dims", [(16, 24, 24), (6, 10, 14)])
def test_in_place_and_several_tensors(dims, halves):
    """Q and K of different head counts in one launch; in place; a broadcast input."""
    grid, N, d = (4, 3, 5), 60, 64
    pos = coordinates(grid)
    q, k = make((2, 7, N, d), torch.bfloat16, 4), make((2, N, 2, d), torch.bfloat16, 5).transpose(1, 2)
    a, b = tsr.tsr_rope([q, k], dims, grid=grid, halves=halves)
    check(q, a, pos, dims, halves=halves)
    check(k, b, pos, dims, halves=halves)
    q2, k2 = q.clone(), k.clone()
    tsr.tsr_rope((q2, k2), dims, grid=grid, halves=halves, out=(q2, k2))
    assert torch.equal(q2, a) and torch.equal(k2, b)
    one = make((1, 1, N, d), torch.bfloat16, 6)
    wide = tsr.tsr_rope(one.expand(2, 3, N, d), dims, grid=grid, halves=halves)
    check(one.expand(2, 3, N, d), wide, pos, dims, halves=halves)


def test_gradient_against_differences():
    """<g, R(x + h v) - R(x - h v)> / 2h = <R^T g, v>; the map is linear, so the
    difference quotient is exact up to fp32 rounding of R(x): each of the 2 n terms
    is off by about 1e-7 |x g|, at random; 1e-5 of the norms' product is far above."""
    grid, dims, d = (3, 4, 5), (10, 12, 14), 40
    x, v, g = (make((2, 3, 60, d), torch.float32, s) for s in (7, 8, 9))
    f = lambda t: tsr.tsr_rope(t, dims, grid=grid, halves=True)
    lhs = ((f(x + v).double() - f(x - v).double()) * g.double()).sum() / 2
    rhs = (tsr.tsr_rope_backward(g, dims, grid=grid, halves=True).double() * v.double()).sum()
    assert abs(lhs - rhs) <= 1e-5 * g.double().norm() * v.double().norm()


def test_infinities_stay_in_their_pair():
    x = make((1, 1, 6, 16), torch.bfloat16)
    x[0, 0, 2, 4], x[0, 0, 3, 15] = float("inf"), float("nan")
    y = tsr.tsr_rope(x, (8, 6), grid=(2, 3))
    bad = ~torch.isfinite(y[0, 0])
    allowed = torch.zeros_like(bad)
    allowed[2, 4:6] = True
    allowed[3, 15] = True                                  # past the axes: copied
    assert torch.equal(bad & ~allowed, torch.zeros_like(bad)) and bad[2, 4] and bad[3, 15]


def test_graph_capture_and_another_stream():
    grid, dims = (4, 4, 4), (16, 24, 24)
    x = make((1, 3, 64, 64), torch.bfloat16)
    want = tsr.tsr_rope(x, dims, grid=grid)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = tsr.tsr_rope(x, dims, grid=grid, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out, graph = torch.empty_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tsr.tsr_rope(x, dims, grid=grid, out=out)
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, tsr.tsr_rope(x, dims, grid=grid))


def test_binding_refusals():
    x = make((1, 2, 12, 16), torch.bfloat16)
    for bad in (dict(), dict(grid=(3, 4), positions=torch.zeros((12, 2), dtype=torch.int32, device="cuda")),
                dict(grid=(12,)), dict(positions=torch.zeros((12, 2), dtype=torch.int64, device="cuda")),
                dict(positions=torch.zeros((11, 2), dtype=torch.int32, device="cuda")),
                dict(grid=(3, 4), out=torch.empty((1, 2, 12, 18), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            tsr.tsr_rope(x, (8, 8), **bad)
    for t in (x.cpu(), x.double(), x.transpose(2, 3), x[0], [x, x.float()], [x, x[:, :, :5]]):
        with pytest.raises((ValueError, tsr.TsrError)):
            tsr.tsr_rope(t, (8, 8), grid=(3, 4))
    with pytest.raises(tsr.TsrError) as e:
        tsr.tsr_rope(x, (8, 8), grid=(3, 5))
    assert e.value.status == 1
