"""Argument checks of a layer's operators (norm with rotation), on the host, before
anything is launched."""
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
