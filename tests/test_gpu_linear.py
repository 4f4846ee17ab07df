"""Linear layers with their epilogue, and their gradients, on the GPU against the formulas
in fp64.

Tolerances, from the arithmetic (u: half a step of the type, 2^-8 bf16, 2^-11 fp16):
  a product of k terms: the tensor cores add 16 products at a time to an fp32 sum, each add
    off by at most 2^-23 of the terms' absolute sum: acc = (k / 16 + 32) 2^-23 sum |a| |b|
    (32: the bias, the residual and the parts of a split product).
  activation: slope at most 1.13, the exponential within 1e-5 where it counts: 1.13 acc +
    1e-5 |z|; then u of the output.  fp16: half a subnormal step more.
  dz: 1e-5 (1 + |z|) |dout| from the slope, and u |dz| as an operand where an activation
    makes it; an output's error is the sum of its terms' and u of itself.
  In the 2-norm the roundings of dz and of the output are independent, at most u / sqrt(3)
    of each value in the root mean square: together 0.82 u, checked against u (sizes where
    the sums have enough terms; the rest is below 0.05 u).
"""
import math

import pytest
import torch

import block_sparse_attention_tsr_gb300 as tsr

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()
    yield
    tsr.tsr_linear_device_status()


def make(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def rows(t):
    """[B, N, features] of [N, f], [B, N, f] or head-major [B, H, N, d], in fp64."""
    t = t.double()
    return t[None] if t.dim() == 2 else t.transpose(1, 2).flatten(2) if t.dim() == 4 else t


def act(z, name):
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z / (1 + torch.exp(-z)) if name == "silu" else z


def slope(z, name):
    if name is None:
        return torch.ones_like(z)
    z = z.clone().requires_grad_(True)
    with torch.enable_grad():
        return torch.autograd.grad(act(z, name).sum(), z)[0]


def acc(a, b, k):
    return (k / 16 + 32) * 2.0 ** -23 * (a.abs() @ b.abs())


def near(got, want, tol, dtype):
    assert got.dtype == dtype
    err = (rows(got) - want).abs()
    bad = ~(err <= tol + U[dtype] * want.abs() + TINY[dtype])
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{float(rows(got)[bad][0])} for {float(want[bad][0])}")


def check_forward(got, x, w, bias=None, activation=None, residual=None, pre=None):
    xd, wd = rows(x), w.double()
    z, off = xd @ wd.t(), acc(xd, wd.t(), w.shape[1])
    if bias is not None:
        z = z + bias.double()
        off = off + 2.0 ** -22 * bias.double().abs()
    if pre is not None:
        near(pre, z, off, x.dtype)
    y, off = act(z, activation), 1.13 * off + (1e-5 * z.abs() if activation else 0)
    if residual is not None:
        y = y + rows(residual)
        off = off + 2.0 ** -22 * rows(residual).abs()
    near(got, y, off, x.dtype)


def check_backward(grads, dout, x, w, activation=None, pre=None, norm=True):
    dx, dw, db = grads
    dtype, u = x.dtype, U[x.dtype] if activation else 0.0
    g, xd, wd = rows(dout), rows(x), w.double()
    z = rows(pre) if activation else torch.zeros_like(g)
    dz = g * slope(z, activation)
    off = (1e-5 * (1 + z.abs()) * g.abs()) if activation else torch.zeros_like(g)
    rounded = off + u * dz.abs() + (TINY[dtype] if activation else 0)
    flat = lambda t: t.flatten(0, 1)
    T = flat(xd).shape[0]
    for got, want, tol in (
            (dx, dz @ wd, rounded @ wd.abs() + acc(dz, wd, w.shape[0])),
            (dw, flat(dz).t() @ flat(xd), flat(rounded).t() @ flat(xd).abs() + acc(flat(dz).t(), flat(xd), T)),
            (db, flat(dz).sum(0), flat(off).sum(0) + (T / 64 + 64) * 2.0 ** -24 * flat(dz).abs().sum(0))):
        if got is None:
            continue
        near(got[None] if got.dim() == 1 else got, want[None] if want.dim() < 3 else want,
             tol[None] if tol.dim() < 3 else tol, dtype)
        if norm:
            assert (rows(got[None] if got.dim() == 1 else got) - want).norm() <= U[dtype] * want.norm()


# batches, tokens, in features, out features: each kind of tile, in all three products, whole,
# cut along k, and both in one launch
SIZES = [(1, 1, 8, 8), (1, 2, 256, 2048), (1, 5, 1160, 264), (2, 33, 200, 1544), (1, 130, 72, 64),
         (1, 200, 1160, 1544), (2, 350, 264, 1544), (3, 257, 1160, 8), (1, 5001, 1160, 1544), (1, 3000, 136, 72),
         (2, 333, 4096, 2048), (1, 4096, 512, 512), (3, 129, 64, 320), (5, 1, 512, 512),
         (1, 130, 1120, 3944), (1, 72, 1352, 3560), (1, 355, 3392, 264), (2, 1, 3192, 32), (1, 1283, 2264, 1576),
         (1, 2593, 1176, 1712), (1, 2674, 3456, 520), (1, 6588, 3360, 8), (2, 657, 2744, 1592), (1, 329, 264, 3432),
         (1, 65, 3744, 1392), (1, 517, 3224, 2536), (3, 526, 2704, 1320), (1, 1, 16, 2336),
         (1, 65, 2456, 4128), (1, 33, 2616, 3952), (5, 65, 3584, 392), (1, 71, 4120, 2664), (3, 11, 4056, 2464),
         (1, 354, 392, 3256)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B,N,K,M", SIZES)
def test_forward_sizes(B, N, K, M, dtype):
    x, w = make((B, N, K), dtype, 1), make((M, K), dtype, 2, K ** -0.5)
    check_forward(tsr.tsr_linear(x, w), x, w)
    b, r = make((M,), dtype, 3), make((B, N, M), dtype, 4)
    out, pre = tsr.tsr_linear(x, w, b, activation="gelu_tanh", residual=r, pre=True)
    check_forward(out, x, w, b, "gelu_tanh", r, pre)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B,N,K,M", SIZES)
def test_backward_sizes(B, N, K, M, dtype):
    x, w = make((B, N, K), dtype, 1), make((M, K), dtype, 2, K ** -0.5)
    dout, pre = make((B, N, M), dtype, 3), make((B, N, M), dtype, 4)
    norm = B * N * M * K > 10 ** 6
    check_backward(tsr.tsr_linear_backward(dout, x, w), dout, x, w, norm=norm)
    got = tsr.tsr_linear_backward(dout, x, w, activation="silu", pre=pre)
    check_backward(got, dout, x, w, "silu", pre, norm=norm)
    again = tsr.tsr_linear_backward(dout, x, w, activation="silu", pre=pre)
    assert all(torch.equal(a, b) for a, b in zip(got, again))          # the same bits


@pytest.mark.parametrize("activation", [None, "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("B,H,N,d,G,e", [(1, 3, 300, 64, 5, 128), (2, 2, 77, 128, 3, 64), (2, 1, 1, 64, 2, 64),
                                         (1, 4, 900, 128, 4, 128), (3, 5, 20, 192, 1, 320)])
def test_head_major(B, H, N, d, G, e, activation):
    """The attention's layout in and out, and its gradients."""
    K, M = H * d, G * e
    x, w, b = make((B, H, N, d), BF, 1), make((M, K), BF, 2, K ** -0.5), make((M,), BF, 3)
    r, dout = make((B, G, N, e), BF, 4), make((B, G, N, e), BF, 5)
    out, pre = tsr.tsr_linear(x, w, b, activation=activation, residual=r, heads=G, pre=True)
    assert out.shape == (B, G, N, e) and out.is_contiguous()
    check_forward(out, x, w, b, activation, r, pre)
    dx, dw, db = tsr.tsr_linear_backward(dout, x, w, activation=activation, pre=pre)
    assert dx.shape == x.shape
    check_backward((dx, dw, db), dout, x, w, activation, pre, norm=False)
    # the same features token-major
    flat = lambda t: t.transpose(1, 2).flatten(2).contiguous()
    assert torch.equal(flat(out), tsr.tsr_linear(flat(x), w, b, activation=activation, residual=flat(r)))


def test_strided_rows_stay_apart():
    """Slices of wider rows in and out; the memory between them stays as it was."""
    B, N, K, M = 2, 70, 136, 200
    x = make((B, N + 3, K + 24), BF, 1)[:, 3:, 8:8 + K]
    w, b = make((M, K), BF, 2, K ** -0.5), make((M,), BF, 3)
    wide = torch.full((B, N, 3, M + 8), 7.0, dtype=BF, device="cuda")
    kept = torch.full((B, N, M + 16), 7.0, dtype=BF, device="cuda")
    out, pre, res = wide[:, :, 1, :M], kept[..., 8:8 + M], make((B, N, 2 * M), BF, 4)[..., M:]
    tsr.tsr_linear(x, w, b, activation="silu", residual=res, out=out, pre=pre)
    check_forward(out, x, w, b, "silu", res, pre)
    assert (wide[:, :, 0] == 7).all() and (wide[:, :, 2] == 7).all() and (wide[..., M:] == 7).all()
    assert (kept[..., :8] == 7).all() and (kept[..., 8 + M:] == 7).all()
    dout = make((B, N, 3 * M), BF, 5)[..., M:2 * M]
    dx = torch.full((B, N, K + 8), 7.0, dtype=BF, device="cuda")
    got = tsr.tsr_linear_backward(dout, x, w, activation="silu", pre=pre, dx=dx[..., :K])
    check_backward(got, dout, x, w, "silu", pre, norm=False)
    assert (dx[..., K:] == 7).all()
    # tokens of single rows, and rows in another order than batch, token
    t = make((N, B, K), BF, 6).transpose(0, 1)
    check_forward(tsr.tsr_linear(t, w, b), t, w, b)
    check_forward(tsr.tsr_linear(t[0], w, b), t[0], w, b)


def test_in_place_residual_and_partial_gradients():
    x, w, b = make((1, 300, 128), BF, 1), make((256, 128), BF, 2, 0.1), make((256,), BF, 3)
    r = make((1, 300, 256), BF, 4)
    want = tsr.tsr_linear(x, w, b, activation="gelu", residual=r)
    stream = r.clone()
    assert tsr.tsr_linear(x, w, b, activation="gelu", residual=stream, out=stream) is stream
    assert torch.equal(stream, want)
    dout, pre = make((1, 300, 256), BF, 5), make((1, 300, 256), BF, 6)
    full = tsr.tsr_linear_backward(dout, x, w, activation="gelu", pre=pre)
    check_backward(full, dout, x, w, "gelu", pre)
    for i in range(3):
        got = tsr.tsr_linear_backward(dout, x, w, activation="gelu", pre=pre, need=[k == i for k in range(3)])
        assert torch.equal(got[i], full[i]) and [g is None for g in got] == [k != i for k in range(3)]


@pytest.mark.parametrize("activation", ["gelu", "gelu_tanh", "silu"])
def test_activations_over_their_range(activation):
    """An identity product: the activation and its slope at every bf16 value of a range,
    large ones, infinities and NaN among them."""
    n = 256
    v = torch.arange(2 ** 16, dtype=torch.int32).to(torch.int16).view(BF).cuda().view(n, n)
    eye = torch.eye(n, dtype=BF, device="cuda")
    fin = torch.isfinite(v) & (v.abs() < 1e30)
    x = torch.where(fin, v, torch.zeros_like(v))
    y, want = tsr.tsr_linear(x, eye, activation=activation), act(x.double(), activation)
    # the exponent is at most 70 where the result is above 1e-30, off by five roundings
    tol = 2.0 ** -8 * want.abs() + 70 * 5 * 2.0 ** -24 * want.abs() + 2.0 ** -126
    far = want.abs() < 1e-30                     # the exponential runs out of fp32's range there
    assert torch.all(((y.double() - want).abs() <= tol) | (far & (y.abs() < 2e-30)))
    z = v[None]
    dz = tsr.tsr_linear_backward(torch.ones_like(z), z, eye, activation=activation, pre=z, need=(True, False, False))[0][0]
    ok = torch.isfinite(v).all(-1)               # rows of the product without infinities or NaN
    # 0 or 1 beyond 15, within 1e-5 (further out the formula is inf / inf in fp64 too)
    big = slope(v.double().clamp(-15, 15), activation)
    off = (dz.double() - big).abs()
    assert torch.all((off <= 2.0 ** -8 * big.abs() + 1e-5 * (1 + v.double().abs().clamp(max=30)))[ok])
    assert torch.isnan(dz[torch.isnan(v).any(-1)]).any(-1).all()


def test_values_that_are_not_finite_stay_in_their_row():
    x, w = make((1, 300, 200), BF, 1), make((264, 200), BF, 2, 0.1)
    x[0, 7, 3], x[0, 290, 199] = float("inf"), float("nan")
    y = tsr.tsr_linear(x, w)
    bad = ~torch.isfinite(y[0]).all(-1)
    assert bad.nonzero().flatten().tolist() == [7, 290] and torch.isnan(y[0, 290]).all()
    w[5, 9] = float("nan")
    y = tsr.tsr_linear(x, w)
    assert torch.isnan(y[..., 5]).all() and torch.isfinite(y[0, 8]).sum() == 263


def test_gradient_against_differences():
    """<dout, f(x + h v) - f(x - h v)> / 2h against <dx, v>, likewise the weight and the
    bias.  fp16, with x, v, the weight and h powers of two that leave x +- h v exact: the
    outputs' roundings 2^-11 |f| are at random, over 2h = 2^-4: 2^-7 |dout| |f| / sqrt(n) of
    n = 80,000 terms, 2e-5 |dout| |f|; the truncation, dz^3 f''' / 6h with dz = 0.04, is
    2e-6 of it and the gradient's roundings 5e-6."""
    N, K, M, h = 200, 128, 400, 2.0 ** -5
    q = lambda shape, seed: torch.round(make(shape, torch.float32, seed) * 8).div(8).to(FP)
    x, w, b = q((N, K), 1), q((M, K), 2) * 0.125, q((M,), 3)
    dout = make((N, M), FP, 4)
    f = lambda x, w, b: tsr.tsr_linear(x, w, b, activation="gelu_tanh").double()
    out, pre = tsr.tsr_linear(x, w, b, activation="gelu_tanh", pre=True)
    grads = tsr.tsr_linear_backward(dout, x, w, activation="gelu_tanh", pre=pre)
    size = dout.double().norm() * out.double().norm()
    for k, (t, g) in enumerate(zip((x, w, b), grads)):
        v = torch.sign(make(t.shape, FP, 7 + k)) * (0.125 if k == 1 else 1)
        args = lambda s: [a + s * h * v if i == k else a for i, a in enumerate((x, w, b))]
        lhs = ((f(*args(1)) - f(*args(-1))) * dout.double()).sum() / (2 * h)
        assert abs(lhs - (g.double() * v.double()).sum()) <= 1e-4 * size


def test_graph_capture_and_streams():
    """Two calls at once on two streams, and a captured forward and backward replayed on new
    values."""
    x, w, b = make((1, 500, 256), BF, 1), make((512, 256), BF, 2, 0.06), make((512,), BF, 3)
    dout = make((1, 500, 512), BF, 4)

    def step():
        out, pre = tsr.tsr_linear(x, w, b, activation="silu", pre=True)
        return [out, *tsr.tsr_linear_backward(dout, x, w, activation="silu", pre=pre)]

    want = step()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(step())
    s.wait_stream(torch.cuda.current_stream())
    got.append([tsr.tsr_linear(x, w, b, activation="silu", stream=streams[0])])
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for g in got for a, c in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    x.mul_(-0.5)
    dout.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(captured, step()))


def test_binding_refusals():
    x, w, b = make((2, 20, 64), BF, 1), make((128, 64), BF, 2), make((128,), BF, 3)
    for bad in (dict(x=x.cpu()), dict(x=x.float()), dict(x=x[..., :32]), dict(x=x.transpose(1, 2)), dict(x=x[0, 0]),
                dict(weight=w.half()), dict(weight=w.t()), dict(weight=w[0]), dict(bias=b[:64]), dict(bias=b.float()),
                dict(activation="relu"), dict(heads=3), dict(residual=x), dict(out=torch.empty((2, 20, 128), device="cuda")),
                dict(pre=torch.empty((2, 20, 64), dtype=BF, device="cuda"))):
        with pytest.raises(ValueError):
            tsr.tsr_linear(**{**dict(x=x, weight=w, bias=b), **bad})
    for bad in (dict(x=x[..., 4:]), dict(x=x.expand(2, 20, 64)[:1].expand(2, 20, 64)), dict(heads=4)):
        with pytest.raises((ValueError, tsr.TsrError)):
            tsr.tsr_linear(**{**dict(x=x, weight=w, bias=b), **bad})
    with pytest.raises(tsr.TsrError) as e:       # a broadcast input
        tsr.tsr_linear(x[:1].expand(2, 20, 64), w)
    assert e.value.status == 1
    y = tsr.tsr_linear(x, w)
    for bad in (dict(dout=x), dict(dout=y.float()), dict(activation="gelu"), dict(dx=y), dict(dweight=w.float()),
                dict(dbias=w), dict(need=(True,)), dict(activation="gelu", pre=x)):
        with pytest.raises(ValueError):
            tsr.tsr_linear_backward(**{**dict(dout=y, x=x, weight=w), **bad})
    with pytest.raises(tsr.TsrError):
        tsr.tsr_linear_backward(y, x, w, need=(False, False, False))


@pytest.mark.parametrize("activation", [None, "silu"])
@pytest.mark.parametrize("B,N,K,M", [(1, 20011, 64, 64), (1, 19999, 264, 8), (2, 9001, 136, 96), (1, 12345, 8, 544),
                                     (3, 4700, 320, 264)])
def test_narrow_weight_gradients_of_many_tokens(B, N, K, M, activation):
    # one to four tiles cut into up to 76 parts; rows of 1 to 68 pieces of eight columns
    x, w = make((B, N, K), BF, 1), make((M, K), BF, 2, K ** -0.5)
    dout, pre = make((B, N, M), BF, 3), make((B, N, M), BF, 4) if activation else None
    grads = tsr.tsr_linear_backward(dout, x, w, activation=activation, pre=pre)
    check_backward(grads, dout, x, w, activation, pre)
    again = tsr.tsr_linear_backward(dout, x, w, activation=activation, pre=pre)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("N,K,M", [(1300, 4608, 5000), (4300, 4608, 5000), (30001, 776, 1032), (700, 6600, 4104)])
def test_groups_of_row_tiles(N, K, M):
    # operands past the size that two row tiles at a time are taken for; groups that are not full
    x, w = make((1, N, K), BF, 1), make((M, K), BF, 2, K ** -0.5)
    check_forward(tsr.tsr_linear(x, w), x, w)
    dout = make((1, N, M), BF, 3)
    check_backward(tsr.tsr_linear_backward(dout, x, w), dout, x, w)


@pytest.mark.parametrize("activation", ["gelu", "silu"])
@pytest.mark.parametrize("B,N,K,M", SIZES)
def test_fp16_sizes_with_the_other_activations(B, N, K, M, activation):
    # with a bias alone and with a residual alone, in every kind of tile
    x, w, b, r = make((B, N, K), FP, 1), make((M, K), FP, 2, K ** -0.5), make((M,), FP, 3), make((B, N, M), FP, 4)
    check_forward(tsr.tsr_linear(x, w, b, activation=activation), x, w, b, activation)
    check_forward(tsr.tsr_linear(x, w, activation=activation, residual=r), x, w, None, activation, r)
    if activation == "gelu":
        dout, pre = make((B, N, M), FP, 5), make((B, N, M), FP, 6)
        got = tsr.tsr_linear_backward(dout, x, w, activation=activation, pre=pre)
        check_backward(got, dout, x, w, activation, pre, norm=B * N * M * K > 10 ** 6)


@pytest.mark.parametrize("activation", [None, "gelu", "silu"])
def test_bf16_sizes_with_a_bias_alone(activation):
    for B, N, K, M in SIZES[::5]:
        x, w, b = make((B, N, K), BF, 1), make((M, K), BF, 2, K ** -0.5), make((M,), BF, 3)
        check_forward(tsr.tsr_linear(x, w, b, activation=activation), x, w, b, activation)


@pytest.mark.parametrize("activation", ["gelu", "gelu_tanh", "silu"])
def test_fp16_activations_over_their_range(activation):
    """An identity product: the activation and its slope at every fp16 value, subnormals,
    infinities and NaN among them.  As for bf16, five roundings of an exponent that is at most
    70 where the result counts; results below the smallest normal number are off by half a
    subnormal step more."""
    n = 256
    v = torch.arange(2 ** 16, dtype=torch.int32).to(torch.int16).view(FP).cuda().view(n, n)
    eye = torch.eye(n, dtype=FP, device="cuda")
    x = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    # beyond 70 the formula is z or 0 (in fp64 the tanh form's and the logistic's exponentials
    # stay finite to 700, z^3 does not keep them there)
    z = x.double()
    want = torch.where(z.abs() < 30, act(z.clamp(-30, 30), activation), z.clamp(min=0))
    y = tsr.tsr_linear(x, eye, activation=activation)
    assert torch.all((y.double() - want).abs() <= (2.0 ** -11 + 70 * 5 * 2.0 ** -24) * want.abs() + 2.0 ** -25)
    z = v[None]
    dz = tsr.tsr_linear_backward(torch.ones_like(z), z, eye, activation=activation, pre=z, need=(True, False, False))[0][0]
    ok = torch.isfinite(v).all(-1)
    s = slope(v.double().clamp(-15, 15), activation)
    off = (dz.double() - s).abs()
    assert torch.all((off <= 2.0 ** -11 * s.abs() + 1e-5 * (1 + v.double().abs().clamp(max=30)) + 2.0 ** -25)[ok])
    assert torch.isnan(dz[torch.isnan(v).any(-1)]).any(-1).all()


def test_fp16_values_past_the_range():
    """Sums past 65,504 are rounded to infinities of their sign, in their places alone; so is a
    dz past it, which is an operand in the tensors' type (dbias sums it before that)."""
    N, K, M = 300, 64, 72
    x, w = make((1, N, K), FP, 1), make((M, K), FP, 2, K ** -0.5)
    x[0, 5], x[0, 6], x[0, 7] = 0, 0, 0
    x[0, 5, 0], x[0, 6, 0], x[0, 7, 0] = 60000, -60000, 30000
    w[:, 0] = 2
    y, pre = tsr.tsr_linear(x, w, activation="silu", pre=True)
    assert torch.all(pre[0, 5] == float("inf")) and torch.all(pre[0, 6] == -float("inf")) and torch.all(pre[0, 7] == 60000)
    assert torch.all(y[0, 5] == float("inf")) and torch.all(y[0, 6] == 0) and torch.all(y[0, 7] == 60000)
    good = [i for i in range(N) if i not in (5, 6)]
    assert torch.isfinite(y[0, good]).all()
    # SiLU's slope at 2 is 1.0908: dz = 65,000 times that is past the range
    pre = torch.full((1, N, M), 2.0, dtype=FP, device="cuda")
    dout = make((1, N, M), FP, 3, 0.01)
    dout[0, 9, 4] = 65000
    x = make((1, N, K), FP, 4)
    dx, dw, db = tsr.tsr_linear_backward(dout, x, w, activation="silu", pre=pre)
    assert torch.isinf(dx[0, 9]).all() and torch.isfinite(dx[0, [i for i in range(N) if i != 9]]).all()
    assert not torch.isfinite(dw[4]).any() and torch.isfinite(dw[[i for i in range(M) if i != 4]]).all()
    dout[0, 9, 4], dout[0, 10, 4] = 60000, -60000
    db = tsr.tsr_linear_backward(dout, x, w, activation="silu", pre=pre, need=(False, False, True))[2]
    want = (dout.double() * slope(pre.double(), "silu")).sum((0, 1))
    tol = 2.0 ** -11 * want.abs() + 2.0 ** -25 + (1e-5 * 3 + (N / 64 + 64) * 2.0 ** -24) * dout.double().abs().sum((0, 1)) * 1.1
    assert torch.all((db.double() - want).abs() <= tol)


@pytest.mark.parametrize("B,N,K,M", [(1, 2593, 1176, 1712), (2, 333, 4096, 264), (1, 20011, 64, 64), (1, 5001, 1160, 1544),
                                     (1, 16, 2048, 512), (1, 355, 3392, 264)])
def test_workspaces_and_outputs_may_hold_anything(B, N, K, M):
    """Nothing is read from a workspace or an output before it was written in the call, and a
    workspace serves one call after another, of other shapes too."""
    x, w, dout = make((B, N, K), BF, 1), make((M, K), BF, 2, K ** -0.5), make((B, N, M), BF, 3)
    out, pre = tsr.tsr_linear(x, w, activation="silu", pre=True)
    grads = tsr.tsr_linear_backward(dout, x, w, activation="silu", pre=pre)
    space = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    small = make((1, 700, 264), BF, 4), make((1544, 264), BF, 5, 0.06)
    for byte in (0xFF, 0x01, None):
        if byte is not None:
            space.fill_(byte)
        a, b, c = (torch.full_like(t, float("nan")) for t in grads)
        y, z = torch.full_like(out, float("nan")), torch.full_like(out, float("nan"))
        tsr.tsr_linear(x, w, activation="silu", out=y, pre=z, workspace=space)
        tsr.tsr_linear(*small, workspace=space)
        tsr.tsr_linear_backward(dout, x, w, activation="silu", pre=pre, dx=a, dweight=b, dbias=c, workspace=space)
        assert all(torch.equal(s, t) for s, t in zip((y, z, a, b, c), (out, pre, *grads)))
