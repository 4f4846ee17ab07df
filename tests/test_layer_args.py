"""Argument checks of a layer's operators (norm with rotation, linear layers), on the host,
before anything is launched."""
import ctypes

import pytest

import block_sparse_attention_tsr_gb300 as tsr

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def L():
    tsr.build()
    return tsr.lib()


def _desc(**kw):
    d = tsr._RopeDesc()
    base = dict(B=1, N=64, d=64, dtype=0, n_axes=2, axis_dim=[32, 32], theta=1e4, grid=[8, 8])
    base.update(kw)
    for k, v in base.items():
        if isinstance(v, list):
            getattr(d, k)[:len(v)] = v
        else:
            setattr(d, k, v)
    return d


def _tensors(**kw):
    arr = (tsr._NormRopeTensor * 5)()
    for i in range(5):
        a = arr[i]
        a.x, a.weight, a.dout, a.out, a.dweight = (65536 * (5 * i + k + 1) for k in range(5))
        a.H = 2
        a.x_stride[:] = a.dout_stride[:] = a.out_stride[:] = [2 * 64 * 64, 64 * 64, 64]
    for k, v in kw.items():
        if isinstance(v, list):
            getattr(arr[0], k)[:] = v
        else:
            setattr(arr[0], k, v)
    return arr


def _both(L, d, t, n=1, eps=1e-6):
    ptr = ctypes.cast(t, ctypes.c_void_p)
    return (L.tsr_norm_rope(ctypes.byref(d), eps, ptr, n, None),
            L.tsr_norm_rope_backward(ctypes.byref(d), eps, ptr, n, 1 << 20, 1 << 40, None))


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(d=63), INVALID), (dict(d=258), INVALID), (dict(dtype=3), INVALID),
    (dict(n_axes=0), INVALID), (dict(axis_dim=[32, 31]), INVALID), (dict(axis_dim=[32, 34]), INVALID),
    (dict(grid=[8, 9]), INVALID), (dict(theta=0.0), INVALID), (dict(B=65536), UNSUPPORTED), (dict(positions=4098), INVALID),
])
def test_norm_rope_refuses_bad_shapes(L, kw, code):
    assert _both(L, _desc(**kw), _tensors()) == (code, code)
    n = ctypes.c_size_t(0)
    assert L.tsr_norm_rope_backward_workspace(ctypes.byref(_desc(**kw)), 1, ctypes.byref(n)) == code
    assert len(L.tsr_last_error()) > 0


@pytest.mark.parametrize("n,kw", [
    (0, {}), (5, {}), (1, dict(x=0)), (1, dict(out=0)), (1, dict(x=65537)), (1, dict(out=65537)), (1, dict(H=0)),
    (1, dict(weight=65537)), (1, dict(weight_dtype=1)), (1, dict(weight_dtype=3)), (2, dict(weight_dtype=2)),
    (1, dict(x_stride=[8192, -1, 64])), (1, dict(out_stride=[8192, 4096, 32])), (1, dict(out_stride=[8192, 0, 64])),
    (1, dict(out=65536, out_stride=[8192, 64, 128])), (1, dict(out_stride=[8192, 4032, 64])),
    (1, dict(x_stride=[8192, 4096, 1 << 60])), (2, dict(out=65536 * 6)), (2, dict(out=65536 * 9)),
])
def test_norm_rope_refuses_bad_tensors(L, n, kw):
    assert _both(L, _desc(), _tensors(**kw), n) == (INVALID, INVALID)
    assert len(L.tsr_last_error()) > 0


@pytest.mark.parametrize("n,kw", [
    (1, dict(dout=0)), (1, dict(dout=65537)), (1, dict(dweight=65537)), (1, dict(weight=0)),
    (1, dict(dweight=65536 * 2)), (1, dict(dweight=65536)), (1, dict(dweight=65536 * 4)), (2, dict(dweight=65536 * 10)),
    (1, dict(dout_stride=[8192, -1, 64])), (1, dict(dout=65536 * 4, dout_stride=[8192, 64, 128])),
    (2, dict(out=65536 * 8)),
])
def test_norm_rope_backward_refuses_bad_tensors(L, n, kw):
    assert _both(L, _desc(), _tensors(**kw), n)[1] == INVALID
    assert len(L.tsr_last_error()) > 0


@pytest.mark.parametrize("eps", [0.0, -1e-6, float("nan"), float("inf"), 1e-60, 1e39])
def test_norm_rope_refuses_bad_eps(L, eps):
    assert _both(L, _desc(), _tensors(), eps=eps) == (INVALID, INVALID)


def test_norm_rope_refuses_bad_workspaces(L):
    d, t, n = _desc(), ctypes.cast(_tensors(), ctypes.c_void_p), ctypes.c_size_t(0)
    assert L.tsr_norm_rope_backward_workspace(ctypes.byref(d), 1, ctypes.byref(n)) == 0 and n.value > 0
    call = lambda ws, size: L.tsr_norm_rope_backward(ctypes.byref(d), 1e-6, t, 1, ws, size, None)
    assert call(None, n.value) == INVALID
    assert call((1 << 20) + 16, n.value) == INVALID
    assert call(1 << 20, n.value - 1) == INVALID
    assert b"too small" in L.tsr_last_error()
    assert L.tsr_norm_rope_backward_workspace(ctypes.byref(d), 5, ctypes.byref(n)) == INVALID
    assert L.tsr_norm_rope_backward_workspace(ctypes.byref(d), 1, None) == INVALID
    assert L.tsr_norm_rope_backward_workspace(None, 1, ctypes.byref(n)) == INVALID
    assert L.tsr_norm_rope(None, 1e-6, t, 1, None) == INVALID
    assert L.tsr_norm_rope(ctypes.byref(d), 1e-6, None, 1, None) == INVALID


def _linear(**kw):
    d = tsr._LinearDesc()
    base = dict(B=2, N=50, in_heads=1, in_dim=128, out_heads=2, out_dim=64, dtype=0, activation=0)
    base.update(kw)
    for k, v in base.items():
        setattr(d, k, v)
    return d


def _args(**kw):
    a = tsr._LinearArgs()
    base = dict(x=1 << 20, weight=2 << 20, bias=3 << 20, residual=4 << 20, out=5 << 20, pre=6 << 20,
                x_stride=[50 * 128, 0, 128], residual_stride=[6400, 3200, 64], out_stride=[6400, 3200, 64],
                pre_stride=[6400, 3200, 64])
    base.update(kw)
    for k, v in base.items():
        if isinstance(v, list):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


def _grads(**kw):
    a = tsr._LinearGrads()
    base = dict(dout=1 << 20, x=2 << 20, weight=3 << 20, pre=4 << 20, dx=5 << 20, dweight=6 << 20, dbias=7 << 20,
                dout_stride=[6400, 3200, 64], x_stride=[50 * 128, 0, 128], pre_stride=[6400, 3200, 64],
                dx_stride=[50 * 128, 0, 128])
    base.update(kw)
    for k, v in base.items():
        if isinstance(v, list):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


def _linear_both(L, d, a=None, g=None, ws=1 << 24, size=1 << 40):
    return (L.tsr_linear(ctypes.byref(d), ctypes.byref(a or _args()), ws, size, None),
            L.tsr_linear_backward(ctypes.byref(d), ctypes.byref(g or _grads()), ws, size, None))


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(N=-3), INVALID), (dict(in_heads=0), INVALID), (dict(out_heads=-1), INVALID),
    (dict(in_dim=0), INVALID), (dict(in_dim=12), INVALID), (dict(out_dim=72), INVALID), (dict(out_heads=1, out_dim=4), INVALID),
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(activation=4), INVALID), (dict(activation=-1), INVALID),
    (dict(in_dim=(1 << 20) + 8), UNSUPPORTED), (dict(out_heads=1 << 14, out_dim=128), UNSUPPORTED),
    (dict(B=1 << 12, N=1 << 13), UNSUPPORTED), (dict(B=(1 << 31) - 1, N=(1 << 31) - 1), UNSUPPORTED),
])
def test_linear_refuses_bad_shapes(L, kw, code):
    assert _linear_both(L, _linear(**kw)) == (code, code)
    n = ctypes.c_size_t(0)
    for f in (L.tsr_linear_workspace, L.tsr_linear_backward_workspace):
        assert f(ctypes.byref(_linear(**kw)), ctypes.byref(n)) == code
    assert len(L.tsr_last_error()) > 0


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(weight=0), dict(out=0), dict(x=(1 << 20) + 8), dict(weight=(2 << 20) + 2), dict(bias=(3 << 20) + 8),
    dict(residual=(4 << 20) + 8), dict(out=(5 << 20) + 4), dict(pre=(6 << 20) + 8), dict(x_stride=[6400, 0, 0]),
    dict(x_stride=[6400, 0, 124]), dict(x_stride=[-6400, 0, 128]), dict(out_stride=[6400, 3200, 32]),
    dict(out_stride=[6400, 3136, 64]), dict(out_stride=[0, 3200, 64]), dict(residual_stride=[6400, 0, 64]),
    dict(pre_stride=[6400, 64, 64]), dict(residual=5 << 20, residual_stride=[6400, 64, 128]), dict(pre=5 << 20),
    dict(pre=4 << 20), dict(out=1 << 20), dict(out=2 << 20), dict(pre=3 << 20),
])
def test_linear_refuses_bad_tensors(L, kw):
    assert _linear_both(L, _linear(), _args(**kw))[0] == INVALID
    assert len(L.tsr_last_error()) > 0


@pytest.mark.parametrize("kw", [
    dict(dx=0, dweight=0, dbias=0), dict(dout=0), dict(x=0), dict(weight=0), dict(pre=0), dict(dout=(1 << 20) + 8),
    dict(dx=(5 << 20) + 8), dict(dweight=(6 << 20) + 8), dict(dbias=(7 << 20) + 8), dict(dout_stride=[6400, 3200, 0]),
    dict(pre_stride=[6400, 3200, 4]), dict(dx_stride=[6400, 0, 64]), dict(dx=1 << 20), dict(dweight=3 << 20),
    dict(dbias=2 << 20), dict(dx=4 << 20), dict(dweight=5 << 20),
])
def test_linear_backward_refuses_bad_tensors(L, kw):
    assert _linear_both(L, _linear(activation=1), None, _grads(**kw))[1] == INVALID
    assert len(L.tsr_last_error()) > 0


def test_linear_refuses_strides_beyond_the_tensor_maps(L):
    a = _args(x_stride=[1 << 38, 0, 128])
    assert _linear_both(L, _linear(), a)[0] == UNSUPPORTED


def test_linear_refuses_bad_workspaces(L):
    d, n = _linear(activation=3, N=4000, in_dim=4096, out_dim=128), ctypes.c_size_t(0)
    g = _grads(x_stride=[4000 * 4096, 0, 4096], dx_stride=[4000 * 4096, 0, 4096], dout_stride=[4000 * 256, 4000 * 128, 128],
               pre_stride=[4000 * 256, 4000 * 128, 128])
    assert L.tsr_linear_backward_workspace(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value >= 2 * 4000 * 256 * 2
    for ws, size in ((None, n.value), ((1 << 24) + 64, n.value), (1 << 24, n.value - 1)):
        assert L.tsr_linear_backward(ctypes.byref(d), ctypes.byref(g), ws, size, None) == INVALID
    assert b"too small" in L.tsr_last_error()
    assert L.tsr_linear_workspace(None, ctypes.byref(n)) == INVALID
    assert L.tsr_linear_workspace(ctypes.byref(d), None) == INVALID
    assert L.tsr_linear_backward_workspace(ctypes.byref(d), None) == INVALID
    assert L.tsr_linear(ctypes.byref(d), None, None, 0, None) == INVALID
    assert L.tsr_linear(None, ctypes.byref(_args()), None, 0, None) == INVALID
    assert L.tsr_linear_backward(ctypes.byref(d), None, None, 0, None) == INVALID


def test_linear_workspaces_cover_both_ways_to_take_the_batches(L):
    """The tokens of a batch are one row of tokens where the strides allow it, a tile of each
    batch's own otherwise: one size serves both."""
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert L.tsr_linear_workspace(ctypes.byref(_linear(B=3, N=700, in_dim=4096, out_heads=1, out_dim=8)), ctypes.byref(a)) == 0
    assert L.tsr_linear_workspace(ctypes.byref(_linear(B=1, N=2100, in_dim=4096, out_heads=1, out_dim=8)), ctypes.byref(b)) == 0
    assert a.value >= b.value


def test_calls_go_through_the_public_initialisation(monkeypatch):
    """The current device is asked for in the way that sets CUDA up first, and says so where
    that is refused (in a forked child, without a driver)."""
    import torch

    def refuse():
        raise RuntimeError("Cannot re-initialize CUDA in forked subprocess")

    monkeypatch.setattr(torch.cuda, "current_device", refuse)
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((8, 64), dtype=torch.bfloat16)
    heads, norm = torch.zeros((1, 2, 4, 16), dtype=torch.bfloat16), torch.zeros(16, dtype=torch.bfloat16)
    for call in (lambda: tsr.tsr_linear(x, w), lambda: tsr.tsr_linear_backward(x[:, :8], x, w),
                 lambda: tsr.tsr_norm_rope(heads, norm, (8, 8), grid=(2, 2)),
                 lambda: tsr.tsr_norm_rope_backward(heads, heads, norm, (8, 8), grid=(2, 2)),
                 lambda: tsr.tsr_rope(heads, (8, 8), grid=(2, 2)), lambda: tsr._stream_ptr(None)):
        with pytest.raises(RuntimeError, match="re-initialize"):
            call()


def test_entry_points_are_named_once():
    assert len(set(tsr.EXPORTS)) == len(tsr.EXPORTS) and len(set(tsr.__all__)) == len(tsr.__all__)
