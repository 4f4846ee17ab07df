"""The gradient oracle against differences of its own forward, in fp64."""
import numpy as np
import pytest

import workloads as W
from oracle import backward as ob


@pytest.mark.parametrize("segments", [False, True])
def test_gradients_against_differences(segments):
    N, d = 70, 5
    spec = (W.segment_mask(3, 1, 1, N, lo=16, hi=30) if segments else
            W.MaskSpec(W.MASK_UNIFORM, 1, 1, N, bq=16, bk=24,
                       blocks=W.bernoulli_blocks(1, 1, 5, 3, 0.6, 4, zero_rows=1, diag=False)))
    ok = ob.allowed(spec, 0, 0)
    r = np.random.default_rng(0)
    x = [r.standard_normal((N, d)) for _ in range(3)]
    do = r.standard_normal((N, d))
    grads = ob.head(ok, *x, do)[2:5]
    h = 1e-5
    for i in range(3):
        t = r.standard_normal((N, d))
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + h * t, x[i] - h * t
        diff = ((ob.head(ok, *up, do)[0] - ob.head(ok, *down, do)[0]) * do).sum() / (2 * h)
        # central differences: h^2 times a third derivative of order 10 at these sizes
        assert abs(diff - (grads[i] * t).sum()) <= 1e-6


def test_rows_and_columns_without_pairs():
    N, d = 64, 4
    blocks = np.ones((1, 1, 4, 4), np.uint8)
    blocks[0, 0, 1] = 0
    blocks[0, 0, :, 2] = 0
    ok = ob.allowed(W.MaskSpec(W.MASK_UNIFORM, 1, 1, N, bq=16, bk=16, blocks=blocks), 0, 0)
    r = np.random.default_rng(1)
    q, k, v, do = (r.standard_normal((N, d)) for _ in range(4))
    o, lse, dq, dk, dv, p, ds = ob.head(ok, q, k, v, do)
    assert np.all(o[16:32] == 0) and np.all(lse[16:32] == -np.inf) and np.all(dq[16:32] == 0)
    assert np.all(dk[32:48] == 0) and np.all(dv[32:48] == 0)
    assert np.allclose(ds.sum(1), 0, atol=1e-13)       # rows of dS sum to zero
