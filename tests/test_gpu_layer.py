"""A layer's training step, each of its results against fp64 on the inputs it got."""
import numpy as np
import pytest
import torch

import block_sparse_attention_tsr_gb300 as tsr
import workloads as W
from oracle import backward as ob
from oracle import layer

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("d,grid,dims", [(128, (4, 11, 17), (44, 42, 42)), (64, (3, 13, 10), (16, 24, 24))])
def test_rotate_select_attend_and_back(d, grid, dims, halves):
    B, H, N = 1, 2, int(np.prod(grid))
    kw = dict(grid=grid, halves=halves)
    q0, k0, v = (t.cuda() for t in W.qkv(B, H, N, d, 31))
    do = W.qkv(B, H, N, d, 32)[0].cuda()
    pos = layer.coordinates(grid)
    q, k = tsr.tsr_rope([t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q0, k0)], dims, **kw)
    for got, x in ((q, q0), (k, k0)):
        want, size = layer.rotate(f64(x), pos, dims, halves=halves)
        assert np.all(np.abs(f64(got) - want) <= layer.rotation_bound(want, size, U))
    blocks = tsr.tsr_block_select(q, k, 4, bq=64, bk=64, first=1, diagonal=True)
    assert np.array_equal(blocks.cpu().numpy(), layer.select(f64(q), f64(k), 4, 64, 64, 1, True))
    mask = tsr.make_mask(tsr.UNIFORM, B, H, N, d, bq=64, bk=64, blocks=blocks)
    out, lse = tsr.tsr_bsa_forward(q, k, v, tsr.tsr_plan(mask))
    plan = tsr.tsr_backward_plan(mask)
    grads = tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan)
    plan.device_status()
    spec = W.MaskSpec(W.MASK_UNIFORM, B, H, N, bq=64, bk=64, blocks=blocks.cpu().numpy())
    for h in range(H):
        x = [f64(t[0, h]) for t in (q, k, v, do)]
        o, _, dq, dk, dv, p, ds = ob.head(ob.allowed(spec, 0, h), *x)
        for g, want, bound in zip(grads, (dq, dk, dv), ob.head_bounds(*x, o, dq, dk, dv, p, ds)):
            assert np.all(np.abs(f64(g[0, h]) - want) <= bound)
    for got, x in zip(tsr.tsr_rope_backward(list(grads[:2]), dims, **kw), grads):
        want, size = layer.rotate(f64(x), pos, dims, halves=halves, inverse=True)
        assert np.all(np.abs(f64(got) - want) <= layer.rotation_bound(want, size, U))
