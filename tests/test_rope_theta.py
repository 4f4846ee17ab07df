"""Values of theta at the end of the doubles' range: a frequency that is not finite is
refused on the host."""
import ctypes

import pytest

import block_sparse_attention_tsr_gb300 as tsr


@pytest.fixture(scope="module")
def L():
    tsr.build()
    return tsr.lib()


def call(L, theta, dims):
    d, t = tsr._RopeDesc(), tsr._RopeTensor()
    d.B, d.N, d.d, d.dtype, d.n_axes, d.theta = 1, 64, 64, 0, len(dims), theta
    d.axis_dim[:len(dims)] = dims
    d.grid[:len(dims)] = [64] + [1] * (len(dims) - 1)
    t.x, t.out, t.H = 4096, 1 << 20, 2
    t.x_stride[:] = t.out_stride[:] = [2 * 64 * 64, 64 * 64, 64]
    return L.tsr_rope(ctypes.byref(d), ctypes.byref(t), 1, None)


@pytest.mark.parametrize("dims", [(64,), (2, 62), (62, 2)])
def test_a_frequency_that_is_not_finite(L, dims):
    assert call(L, 5e-324, dims) == 1
    assert b"frequency" in L.tsr_last_error()
