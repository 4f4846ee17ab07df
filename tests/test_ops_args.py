"""Argument checks of the operators beside the attention forward (position
rotation, block selection), on the host, before anything is launched."""
import ctypes

import pytest

import block_sparse_attention_tsr_gb300 as tsr

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def L():
    tsr.build()
    return tsr.lib()


def _rope(**kw):
    d = tsr._RopeDesc()
    base = dict(B=1, N=64, d=64, dtype=0, n_axes=2, axis_dim=[32, 32], theta=1e4, grid=[8, 8])
    base.update(kw)
    for k, v in base.items():
        if isinstance(v, list):
            getattr(d, k)[:len(v)] = v
        else:
            setattr(d, k, v)
    return d


def _tensors(n=1, **kw):
    arr = (tsr._RopeTensor * 5)()
    for i in range(5):
        a = arr[i]
        a.x, a.out, a.H = 4096 * (2 * i + 1), 4096 * (2 * i + 2), 2
        a.x_stride[:] = a.out_stride[:] = [2 * 64 * 64, 64 * 64, 64]
    for k, v in kw.items():
        if isinstance(v, list):
            getattr(arr[0], k)[:] = v
        else:
            setattr(arr[0], k, v)
    return arr


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(d=63), INVALID), (dict(d=258), INVALID),
    (dict(d=0), INVALID), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(n_axes=0), INVALID),
    (dict(n_axes=5), INVALID), (dict(axis_dim=[32, 31]), INVALID), (dict(axis_dim=[0, 32]), INVALID),
    (dict(axis_dim=[-2, 32]), INVALID), (dict(axis_dim=[32, 34]), INVALID), (dict(grid=[8, 9]), INVALID),
    (dict(grid=[0, 8]), INVALID), (dict(grid=[-8, -8]), INVALID), (dict(theta=0.0), INVALID),
    (dict(theta=float("nan")), INVALID), (dict(theta=float("inf")), INVALID), (dict(theta=-1.0), INVALID),
    (dict(N=(1 << 24) + 2, grid=[2, (1 << 23) + 1]), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
    (dict(positions=4098), INVALID),
])
def test_rope_refuses_bad_shapes(L, kw, code):
    d, t = _rope(**kw), _tensors()
    assert L.tsr_rope(ctypes.byref(d), ctypes.cast(t, ctypes.c_void_p), 1, None) == code
    assert len(L.tsr_last_error()) > 0


@pytest.mark.parametrize("n,kw", [
    (0, {}), (5, {}), (1, dict(x=0)), (1, dict(out=0)), (1, dict(x=4097)), (1, dict(out=8193)),
    (1, dict(H=0)), (1, dict(x_stride=[8192, -1, 64])), (1, dict(out_stride=[8192, 4096, 32])),
    (1, dict(out_stride=[8192, 0, 64])), (1, dict(out=4096, out_stride=[8192, 64, 128])),
    (1, dict(out_stride=[8192, 64, 64])), (1, dict(out_stride=[8192, 4032, 64])),
    (1, dict(x_stride=[8192, 4096, 1 << 60])), (2, dict(out=4096 * 3)), (2, dict(out=4096 * 4)),
])
def test_rope_refuses_bad_tensors(L, n, kw):
    d, t = _rope(), _tensors(**kw)
    assert L.tsr_rope(ctypes.byref(d), ctypes.cast(t, ctypes.c_void_p), n, None) == INVALID
    assert len(L.tsr_last_error()) > 0


def test_rope_refuses_null(L):
    d, t = _rope(), _tensors()
    assert L.tsr_rope(None, ctypes.cast(t, ctypes.c_void_p), 1, None) == INVALID
    assert L.tsr_rope(ctypes.byref(d), None, 1, None) == INVALID


def _select(**kw):
    d = tsr._SelectDesc()
    base = dict(B=1, H=2, N=1000, d=64, bq=64, bk=64, keep=3)
    base.update(kw)
    for k, v in base.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(H=-1), INVALID), (dict(N=0), INVALID), (dict(d=96), INVALID),
    (dict(bq=15), INVALID), (dict(bk=8), INVALID), (dict(keep=0), INVALID), (dict(first=-1), INVALID),
    (dict(N=(1 << 24) + 1), UNSUPPORTED), (dict(B=1 << 11, H=1 << 10), UNSUPPORTED),
])
def test_select_refuses_bad_shapes(L, kw, code):
    d, n = _select(**kw), ctypes.c_size_t(0)
    assert L.tsr_block_select_workspace(ctypes.byref(d), ctypes.byref(n)) == code
    assert L.tsr_block_select(ctypes.byref(d), 4096, 8192, 12288, 16384, 1 << 40, None) == code
    assert len(L.tsr_last_error()) > 0


def test_select_refuses_bad_pointers(L):
    d, n = _select(), ctypes.c_size_t(0)
    assert L.tsr_block_select_workspace(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    call = lambda *a: L.tsr_block_select(ctypes.byref(d), *a, None)
    assert call(0, 8192, 12288, 16384, n.value) == INVALID
    assert call(4096, 8200, 12288, 16384, n.value) == INVALID
    assert call(4096, 8192, 0, 16384, n.value) == INVALID
    assert call(4096, 8192, 12288, 0, n.value) == INVALID
    assert call(4096, 8192, 12288, 16400, n.value) == INVALID
    assert call(4096, 8192, 12288, 16384, n.value - 1) == INVALID
    assert b"too small" in L.tsr_last_error()
    assert L.tsr_block_select_workspace(None, ctypes.byref(n)) == INVALID
    big, m = _select(bq=2 ** 31 - 1, bk=2 ** 31 - 1), ctypes.c_size_t(0)
    assert L.tsr_block_select_workspace(ctypes.byref(big), ctypes.byref(m)) == 0 and 0 < m.value < n.value
    assert L.tsr_block_select_workspace(ctypes.byref(d), None) == INVALID


def _mask(**kw):
    m = tsr._Mask()
    base = dict(kind=0, B=1, H=1, N=128, d=64, bq=64, bk=64, blocks=16)
    base.update(kw)
    for k, v in base.items():
        setattr(m, k, v)
    return m


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), INVALID), (dict(bq=8), INVALID), (dict(blocks=0), INVALID), (dict(N=0), INVALID),
    (dict(kind=9), INVALID), (dict(kind=2, n_frames=4, frame_size=32, head_kind=16), UNSUPPORTED),
    (dict(kind=3, slice_m=64, indptr=16), UNSUPPORTED),
])
def test_backward_plan_refuses_bad_masks(L, kw, code):
    h, m = ctypes.c_void_p(0), _mask(**kw)
    assert L.tsr_backward_plan(ctypes.byref(m), ctypes.byref(h), None) == code
    assert not h.value and len(L.tsr_last_error()) > 0


def test_backward_refuses_null(L):
    h, n = ctypes.c_void_p(0), ctypes.c_size_t(0)
    assert L.tsr_backward_plan(None, ctypes.byref(h), None) == INVALID
    assert L.tsr_backward_plan(ctypes.byref(_mask()), None, None) == INVALID
    assert L.tsr_backward_plan_update(None, ctypes.byref(_mask()), None) == INVALID
    assert L.tsr_bsa_backward_workspace(None, ctypes.byref(n)) == INVALID
    assert L.tsr_backward_plan_device_status(None, None) == INVALID
    assert L.tsr_bsa_backward(*([4096] * 6), None, 4096, 4096, 4096, 4096, 1 << 20, None) == INVALID
    assert L.tsr_backward_plan_destroy(None) == 0
