"""The attention backward on the GPU against fp64 gradients: element by element
within the bound that the computation's roundings give (oracle/backward.py), and in
the 2-norm within half of it (each rounding is uniform in its range, 1 / sqrt(3) of
its bound in the mean square, and they are independent)."""
import numpy as np
import pytest
import torch

import block_sparse_attention_tsr_gb300 as tsr
import workloads as W
from oracle import backward as ob

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tsr.build()
    tsr.lib()


def uniform(B, H, N, bq, bk, p, seed, zero_rows=0, zero_cols=0, diag=False):
    nq, nk = W.cdiv(N, bq), W.cdiv(N, bk)
    blocks = W.bernoulli_blocks(B, H, nq, nk, p, seed, diag=diag, zero_rows=zero_rows)
    if zero_cols:
        blocks[:, :, :, np.random.default_rng(seed).choice(nk, zero_cols, replace=False)] = 0
    return W.MaskSpec(W.MASK_UNIFORM, B, H, N, bq=bq, bk=bk, blocks=blocks)


def gpu_mask(spec, d):
    return tsr.make_mask(spec.kind, spec.B, spec.H, spec.N, d, **W.mask_tensors(spec))


def inputs(spec, d, seed, scale=1.0):
    q, k, v = W.qkv(spec.B, spec.H, spec.N, d, seed)
    do = W.qkv(spec.B, spec.H, spec.N, d, seed + 1000)[0]
    if scale != 1.0:
        q, k = ((t.float() * scale).bfloat16() for t in (q, k))
    return [t.cuda() for t in (q, k, v, do)]


def compare(spec, x, grads):
    q, k, v, do = (t.double().cpu().numpy() for t in x)
    got = [g.double().cpu().numpy() for g in grads]
    for b in range(spec.B):
        for h in range(spec.H):
            hd = [t[b, h] for t in (q, k, v, do)]
            o, lse, dq, dk, dv, p, ds = ob.head(ob.allowed(spec, b, h), *hd)
            bounds = ob.head_bounds(*hd, o, dq, dk, dv, p, ds)
            pairs = (p.sum(1), p.sum(0), p.sum(0))
            for name, g, want, bound, any_pair in zip(("dq", "dk", "dv"), (t[b, h] for t in got), (dq, dk, dv),
                                                      bounds, pairs):
                err = np.abs(g - want)
                assert np.all(err <= bound), f"{name} {b},{h}: {np.max(err / bound):.3f} of the bound"
                if spec.N >= 63:
                    assert np.linalg.norm(err) <= 0.5 * np.linalg.norm(bound), name
                assert np.all(g[any_pair == 0] == 0), name      # no allowed pair: exactly 0


def run(spec, d, seed, scale=1.0):
    x = inputs(spec, d, seed, scale)
    q, k, v, do = x
    mask = gpu_mask(spec, d)
    out, lse = tsr.tsr_bsa_forward(q, k, v, tsr.tsr_plan(mask))
    plan = tsr.tsr_backward_plan(mask)
    ws = torch.full((plan.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")
    g = [torch.full_like(q, float("nan")) for _ in range(3)]
    tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan, *g, workspace=ws)
    torch.cuda.synchronize()
    plan.device_status()
    compare(spec, x, g)
    return x, out, lse, plan, g


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 127, 128, 129, 191, 256, 333, 1000])
def test_dense_lengths(N, d):
    run(uniform(1, 2, N, 64, 64, 1.1, N), d, N)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,N,bq,bk,p", [
    (1, 2, 1024, 64, 64, 0.3), (2, 3, 700, 32, 32, 0.2), (1, 1, 1500, 128, 128, 0.5),
    (1, 2, 900, 16, 16, 0.1), (1, 2, 1111, 64, 256, 0.4), (1, 2, 1111, 256, 64, 0.4),
    (1, 3, 640, 19, 23, 0.3), (1, 1, 2050, 300, 48, 0.3), (3, 1, 400, 4096, 64, 0.6)])
def test_block_masks(B, H, N, bq, bk, p, d):
    nq, nk = W.cdiv(N, bq), W.cdiv(N, bk)
    run(uniform(B, H, N, bq, bk, p, 7, zero_rows=int(nq > 3), zero_cols=int(nk > 3)), d, 11)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,lo,hi", [(700, 16, 40), (1500, 16, 300), (130, 16, 100)])
def test_segment_masks(N, lo, hi, d):
    run(W.segment_mask(5, 1, 2, N, lo=lo, hi=hi), d, 13)


@pytest.mark.parametrize("d", [64, 128])
def test_nothing_allowed(d):
    spec = uniform(1, 2, 300, 64, 64, 0.0, 1)
    spec.blocks[0, 1, 2, 3] = 1
    _, out, lse, _, g = run(spec, d, 1)
    assert all(torch.all(t[0, 0] == 0) for t in g)


@pytest.mark.parametrize("scale", [4.0, 0.01])
def test_sharp_and_flat_softmax(scale):
    run(uniform(1, 2, 777, 64, 64, 0.4, 3, diag=True), 128, 17, scale)


def test_one_key_per_row():
    """A 16 x 16 diagonal: short lists, every tile a boundary tile."""
    spec = uniform(1, 1, 1000, 16, 16, 0.0, 1, diag=True)
    run(spec, 128, 19)


def test_many_items_and_same_bits():
    """More work items than SMs; twice the same bits; the forward's tensors unchanged."""
    spec = uniform(2, 8, 2100, 64, 64, 0.25, 9, zero_rows=1, zero_cols=1)
    x, out, lse, plan, g = run(spec, 128, 23)
    keep = [t.clone() for t in (*x, out, lse)]
    again = tsr.tsr_bsa_backward(*x[:3], out, lse, x[3], plan)
    assert all(torch.equal(a, b) for a, b in zip(g, again))
    assert all(torch.equal(a, b) for a, b in zip(keep, (*x, out, lse)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,p", [(1030, 0.5), (2100, 1.1), (4200, 0.5), (4200, 0.02)])
def test_few_items_in_parts(N, p, d):
    """One head: items with long lists (the second and third case) are cut in two
    parts that the later one adds up, in order: the same bits every time, from any
    workspace."""
    spec = uniform(1, 1, N, 64, 64, p, 12, zero_rows=1, zero_cols=1)
    x, out, lse, plan, g = run(spec, d, 29)
    ws = torch.full((plan.workspace_bytes,), 7, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        again = tsr.tsr_bsa_backward(*x[:3], out, lse, x[3], plan, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(g, again))


def test_update_streams_and_overlapping_calls():
    a, b = uniform(1, 3, 900, 64, 64, 0.2, 1, zero_rows=1), uniform(1, 3, 900, 32, 128, 0.6, 2, zero_cols=1)
    x = inputs(a, 64, 3)
    q, k, v, do = x
    fwd, plan = tsr.tsr_plan(gpu_mask(a, 64)), tsr.tsr_backward_plan(gpu_mask(a, 64))
    out, lse = tsr.tsr_bsa_forward(q, k, v, fwd)
    first = tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan)
    compare(a, x, first)
    # two calls of one plan at the same time, each with its own workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    both = [tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(t, u) for g in both for t, u in zip(g, first))
    fwd.update(gpu_mask(b, 64))
    plan.update(gpu_mask(b, 64))
    out, lse = tsr.tsr_bsa_forward(q, k, v, fwd)
    compare(b, x, tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan))
    plan.device_status()


def test_graph_capture():
    spec = uniform(1, 2, 600, 64, 64, 0.4, 4, zero_rows=1)
    q, k, v, do = inputs(spec, 128, 5)
    mask = gpu_mask(spec, 128)
    fwd, plan = tsr.tsr_plan(mask), tsr.tsr_backward_plan(mask)
    out, lse = tsr.tsr_bsa_forward(q, k, v, fwd)
    g = [torch.empty_like(q) for _ in range(3)]
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan, *g, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tsr.tsr_bsa_forward(q, k, v, fwd, out, lse)
        tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan, *g, workspace=ws)
    do.copy_(do.flip(2))
    v.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    compare(spec, (q, k, v, do), g)


def test_a_layer_together():
    """Rotate Q and K, select blocks, attend, and back through all of it."""
    B, H, grid, d, dims = 1, 2, (4, 11, 17), 128, (44, 42, 42)
    N = 4 * 11 * 17
    q0, k0, v, do = inputs(W.MaskSpec(W.MASK_UNIFORM, B, H, N), d, 31)
    token_major = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q0, k0)]
    q, k = tsr.tsr_rope(token_major, dims, grid=grid)
    blocks = tsr.tsr_block_select(q, k, 4, bq=64, bk=64, first=1, diagonal=True)
    mask = tsr.make_mask(tsr.UNIFORM, B, H, N, d, bq=64, bk=64, blocks=blocks)
    out, lse = tsr.tsr_bsa_forward(q, k, v, tsr.tsr_plan(mask))
    plan = tsr.tsr_backward_plan(mask)
    dq, dk, dv = tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan)
    spec = W.MaskSpec(W.MASK_UNIFORM, B, H, N, bq=64, bk=64, blocks=blocks.cpu().numpy())
    compare(spec, (q, k, v, do), (dq, dk, dv))
    g = tsr.tsr_rope_backward([dq, dk], dims, grid=grid)
    # orthogonal: norms stay, up to the rounding of each value
    for a, b in zip(g, (dq, dk)):
        assert abs(a.double().norm() / b.double().norm() - 1) <= 2.0 ** -8
    plan.device_status()


def test_svg_heads_as_block_masks():
    """An SVG layer's gradients through UNIFORM masks: spatial heads by frame, temporal
    heads of radius 0 in temporal-major order by spatial position."""
    F, S, d = 18, 40, 64
    N = F * S
    svg = W.svg_mask(1, 2, n_frames=F, frame_size=S, kinds=np.array([0, 1], np.int8))
    x = inputs(svg, d, 41)
    q, k, v, do = x
    out, lse = tsr.tsr_bsa_forward(q, k, v, tsr.tsr_plan(gpu_mask(svg, d)))
    by_frame = np.zeros((1, 1, F, F), np.uint8)
    by_frame[0, 0, np.arange(F), np.arange(F)] = by_frame[0, 0, :, 0] = 1
    by_place = np.eye(S, dtype=np.uint8)[None, None]
    for h, (blocks, b) in enumerate(((by_frame, S), (by_place, F))):
        spec = W.MaskSpec(W.MASK_UNIFORM, 1, 1, N, bq=b, bk=b, blocks=blocks)
        one = [t[:, h:h + 1].contiguous() for t in (q, k, v, out, do)]
        if h == 1:
            one = [tsr.tsr_temporal_permute(t, torch.empty_like(t), F, S) for t in one]
        o, l = tsr.tsr_bsa_forward(*one[:3], tsr.tsr_plan(gpu_mask(spec, d)))
        lse_h = lse[:, h:h + 1].contiguous()
        if h == 1:
            lse_h = lse_h.view(1, 1, F, S).transpose(2, 3).reshape(1, 1, N).contiguous()
        assert (o.float() - one[3].float()).abs().max() <= 2e-2 and (l - lse_h).abs().max() <= 1e-3 * l.abs().max()
        g = tsr.tsr_bsa_backward(*one[:3], one[3], lse_h, one[4], tsr.tsr_backward_plan(gpu_mask(spec, d)))
        compare(spec, (*one[:3], one[4]), g)


def test_a_failed_update_is_refused_until_one_succeeds():
    spec = uniform(1, 1, 640, 64, 64, 0.4, 1, diag=True)
    x = inputs(spec, 64, 2)
    q, k, v, do = x
    plan = tsr.tsr_backward_plan(gpu_mask(spec, 64))
    out, lse = tsr.tsr_bsa_forward(q, k, v, tsr.tsr_plan(gpu_mask(spec, 64)))
    with pytest.raises(tsr.TsrError) as e:
        plan.update(gpu_mask(uniform(1, 1, 640, 64, 17, 0.3, 7), 64))     # the key side is too fine
    assert e.value.status == 2
    with pytest.raises(tsr.TsrError) as e:
        tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan)
    assert e.value.status == 1
    plan.update(gpu_mask(spec, 64))
    compare(spec, x, tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan))


def test_same_tensor_for_several_inputs():
    """Q, K, V (and dO) may be one tensor."""
    spec = uniform(1, 2, 500, 64, 64, 0.5, 6, diag=True)
    q = inputs(spec, 128, 8)[0]
    mask = gpu_mask(spec, 128)
    out, lse = tsr.tsr_bsa_forward(q, q, q, tsr.tsr_plan(mask))
    g = tsr.tsr_bsa_backward(q, q, q, out, lse, q, tsr.tsr_backward_plan(mask))
    compare(spec, (q, q, q, q), g)


def test_refusals():
    svg = W.svg_mask(1, 2, n_frames=4, frame_size=32)
    keys = W.random_keylist(1, 1, 2, 128, slice_m=64)
    for spec in (svg, keys):
        with pytest.raises(tsr.TsrError) as e:
            tsr.tsr_backward_plan(gpu_mask(spec, 64))
        assert e.value.status == 2
    # a 128-token tile over more than 8 blocks, of queries (the forward's limit) or keys
    for bq, bk in ((17, 64), (64, 17)):
        with pytest.raises(tsr.TsrError) as e:
            tsr.tsr_backward_plan(gpu_mask(uniform(1, 1, 640, bq, bk, 0.3, 7), 64))
        assert e.value.status == 2
    spec = uniform(1, 2, 200, 64, 64, 0.5, 1, diag=True)
    q, k, v, do = inputs(spec, 64, 1)
    plan = tsr.tsr_backward_plan(gpu_mask(spec, 64))
    out, lse = tsr.tsr_bsa_forward(q, k, v, tsr.tsr_plan(gpu_mask(spec, 64)))
    with pytest.raises(tsr.TsrError):
        plan.update(gpu_mask(uniform(1, 2, 201, 64, 64, 0.5, 1), 64))
    tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan)            # the refused update left it as it was
    for kw in (dict(dq=q), dict(dq=out), dict(dv=do)):
        with pytest.raises(tsr.TsrError):
            tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan, **kw)
    g = torch.empty_like(q)
    with pytest.raises(tsr.TsrError):
        tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan, dq=g, dk=g)
    with pytest.raises(tsr.TsrError):
        tsr.tsr_bsa_backward(q, k, v, out, lse, do, plan, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    for bad in (dict(lse=lse.double()), dict(dout=do.float()), dict(q=q[:, :1]), dict(k=k.transpose(1, 2))):
        args = dict(q=q, k=k, v=v, out=out, lse=lse, dout=do)
        args.update(bad)
        with pytest.raises(ValueError):
            tsr.tsr_bsa_backward(plan=plan, **args)
