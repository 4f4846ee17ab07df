"""Gradients of masked attention in fp64 NumPy, written from the definition, with a
bound of what a bf16 implementation may be off by.  Test infrastructure only."""
import math

import numpy as np

import workloads as W

U = 2.0 ** -8           # half a step of bf16, relative


def allowed(spec, b, h):
    """Element mask [N, N] of one head of a UNIFORM or SEGMENTS mask."""
    t = np.arange(spec.N)
    if spec.kind == W.MASK_UNIFORM:
        i, j = t // spec.bq, t // spec.bk
    else:
        i = np.searchsorted(spec.q_bounds, t, side="right") - 1
        j = np.searchsorted(spec.k_bounds, t, side="right") - 1
    return spec.blocks[b, h][np.ix_(i, j)] != 0


def head(ok, q, k, v, do):
    """One head: O, lse, dQ, dK, dV (fp64), rows with nothing allowed: O = 0, lse = -inf."""
    scale = 1 / math.sqrt(q.shape[1])
    s = np.where(ok, q @ k.T * scale, -np.inf)
    m = s.max(1, keepdims=True)
    e = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    l = e.sum(1, keepdims=True)
    p = e / np.where(l > 0, l, 1.0)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0]
    o = p @ v
    dp = do @ v.T
    delta = (do * o).sum(1, keepdims=True)
    ds = p * (dp - delta) * scale
    return o, lse, ds @ k, ds.T @ q, p.T @ do, p, ds


def head_bounds(q, k, v, do, o, dq, dk, dv, p, ds):
    """Elementwise bounds on the error of dQ, dK, dV, from the roundings of the
    computation: S (fp32 sums of d exact products), P and dS (bf16), O (bf16, from
    bf16 P) inside delta, and the gradients themselves (bf16)."""
    d = q.shape[1]
    scale = 1 / math.sqrt(d)
    a = np.abs
    # relative error of P before its rounding: S and lse are each off by at most
    # d 2^-23 of the sum of magnitudes; 2^-18 covers the exponential and logarithm
    eps_p = 2 * d * 2.0 ** -23 * (a(q) @ a(k).T).max() * scale + 2.0 ** -18
    e_dv = (U + eps_p) * (p.T @ a(do))
    e_dp = d * 2.0 ** -23 * (a(do) @ a(v).T)
    e_delta = (a(do) * ((U + 2 * eps_p) * (p @ a(v)) + U * a(o))).sum(1, keepdims=True)
    e_ds = (U + eps_p) * a(ds) + p * (e_dp + e_delta) * scale * (1 + U)
    e_dq, e_dk = e_ds @ a(k), e_ds.T @ a(q)
    n = p.shape[0]
    acc = n * 2.0 ** -23                       # the fp32 sums over the sequence
    e_dv += acc * (p.T @ a(do))
    e_dq += acc * (a(ds) @ a(k))
    e_dk += acc * (a(ds).T @ a(q))
    tiny = 1e-30
    return [e * (1 + U) + U * a(g) + tiny for e, g in ((e_dq, dq), (e_dk, dk), (e_dv, dv))]
