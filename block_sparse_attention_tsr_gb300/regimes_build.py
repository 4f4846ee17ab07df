"""Offline profiling that fills the regime table (Tessera abstract:
profile-guided regime selection through a lookup table built by offline
profiling).

For every mask class -- logical block shape, density bucket, sequence-length
bucket, head dimension -- a few seeded synthetic masks of that class are planned
and run with every kernel variant (tile orientation: 128-row query tiles or
key-major 64-query tiles; for 128-row tiles the tile width, pipeline depth and
CTAs per SM); the fastest variant (geometric mean of the forward's time over the
bucket's lengths, head counts and masks) becomes the row of that class.  Block masks alternate between banded-plus-random
ones, whose neighbouring rows of blocks resemble each other, and independently
random ones, which fill 128-row tiles least: a selection by scores lies between
the two.  Run on the target GPU:

    python -m block_sparse_attention_tsr_gb300.regimes_build [--out PATH] [--quick]

and commit the written table (``regimes_gb300.txt`` next to this file), which
the binding loads at start-up.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import block_sparse_attention_tsr_gb300 as tsr  # noqa: E402
import workloads as W  # noqa: E402

SHAPES = ((32, 32), (64, 64), (128, 128), (64, 256), (256, 64))
DENSITY_EDGES = (0.0, 0.15, 0.30, 0.45, 0.60, 1.01)
# (n_min, n_max, (N, heads) profiled).  Long sequences are timed with all the heads of
# a request and long enough to reach the power limit, as in use: at 64 x 64 blocks of
# density 0.15 - 0.30 the 128-row tiles, 0.57 full, win by 1% with 8 heads and a few
# calls, and lose by 1% (8% at 75,600 tokens) with 24 heads kept busy.  Short sequences
# differ with the number of work items (64 x 64 blocks, density 0.35, 128-row against
# key-major tiles: 20 against 18 us and 38 against 20 us with 64 items, where the former
# are split, 49 against 57 with 384, 181 against 137 with 504), so several are timed.
N_BUCKETS = ((0, 8191, ((1024, 8), (1024, 24), (2048, 4), (2048, 24), (4096, 8), (8000, 8), (8000, 24))),
             (8192, 1 << 24, ((32760, 24),)))
# (bn, stages, ctas per SM, orientation): 1 = 128-row query tiles, 2 = the
# key-major kernel (d = 128 only; its ring shape is fixed)
ROWS, KEYS = 1, 2
VARIANTS = {128: ((128, 3, 1, ROWS), (128, 2, 1, ROWS), (64, 4, 1, ROWS), (64, 2, 2, ROWS),
                  (64, 2, 1, KEYS)),
            64: ((128, 4, 1, ROWS), (64, 4, 1, ROWS), (64, 3, 2, ROWS))}
# key-list (M x 1 slice) masks: classes by slice height and listed-key fraction;
# the gathered kernel variants
KEYLIST_M = (64, 128)
KEYLIST_EDGES = (0.0, 0.10, 0.20, 0.35, 0.60, 1.01)
VARIANTS_GATHERED = {128: ((128, 3, 1, ROWS), (64, 2, 2, ROWS), (64, 2, 1, KEYS)),
                     64: ((128, 4, 1, ROWS), (64, 3, 2, ROWS))}


def keylist_spec(N, M, frac, heads, seed):
    """A key-list mask of one head's lists (clustered runs), repeated for every
    head: the generator is slow at high densities, and identical heads time the
    same as distinct ones of the same class."""
    one = W.keylist_mask(seed=seed, B=1, H=1, N=N, slice_m=M, frac=frac)
    indptr = np.concatenate([[0]] + [one.indptr[1:] + h * one.indptr[-1] for h in range(heads)])
    return W.MaskSpec(W.MASK_KEYLIST, 1, heads, N, slice_m=M, indptr=indptr.astype(np.int64),
                      indices=np.tile(one.indices, heads))


def block_mask(r, heads, N, bq, bk, dens, banded):
    nq, nk = W.cdiv(N, bq), W.cdiv(N, bk)
    if banded:
        return W.banded_blocks(1, heads, nq, nk, dens, r)
    return (r.random((1, heads, nq, nk)) < dens[..., None, None]).astype(np.uint8)


def time_variant(mask, q, k, v, out, lse, variant, reps):
    """The forward's time in ms, the plan made before."""
    bn, stages, ctas, orient = variant
    plan = tsr.tsr_plan(mask, {"bn": bn, "stages": stages, "ctas_per_sm": ctas, "orient": orient})
    stream = torch.cuda.current_stream()
    for _ in range(3):
        tsr.tsr_bsa_forward(q, k, v, plan, out, lse)
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record(stream)
    for _ in range(reps):
        tsr.tsr_bsa_forward(q, k, v, plan, out, lse)
    b.record(stream)
    torch.cuda.synchronize()
    tsr.tsr_plan_device_status(plan)
    plan.destroy()
    return a.elapsed_time(b) / reps


class Inputs:
    """q, k, v, out and lse of one (N, heads)."""

    def __init__(self, N, heads, d):
        self.N, self.heads = N, heads
        self.qkv = [x.cuda() for x in W.qkv(1, heads, N, d, seed=5)]
        self.out = torch.empty_like(self.qkv[0])
        self.lse = torch.empty((1, heads, N), device="cuda")

    def time(self, spec, d, variants, reps):
        mask = tsr.make_mask(spec.kind, 1, self.heads, self.N, d, **W.mask_tensors(spec))
        return {vv: time_variant(mask, *self.qkv, self.out, self.lse, vv, reps) for vv in variants}


def best_of(times, what):
    """The variant of the least geometric mean of `times`, a list of {variant: ms}."""
    mean = {vv: float(np.exp(np.mean([np.log(t[vv]) for t in times]))) for vv in times[0]}
    best = min(mean, key=mean.get)
    print(f"{what} -> {best}  " + " ".join(f"{vv}:{t:.4f}ms" for vv, t in mean.items()), flush=True)
    return best


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--out", default=os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                  "regimes_gb300.txt"))
    ap.add_argument("--masks", type=int, default=4, help="seeded masks per class, length and head count")
    ap.add_argument("--reps", type=int, default=40)
    ap.add_argument("--quick", action="store_true", help="d = 128, long sequences only")
    args = ap.parse_args()
    tsr.build()
    tsr.lib()
    tsr.tsr_regime_load(None)
    rows = []
    t0 = time.time()
    dims = (128,) if args.quick else (128, 64)
    nbs = N_BUCKETS[1:] if args.quick else N_BUCKETS
    for d in dims:
        for n_min, n_max, points in nbs:
            inputs = [Inputs(N, heads, d) for N, heads in points]
            for bq, bk in SHAPES:
                for lo, hi in zip(DENSITY_EDGES[:-1], DENSITY_EDGES[1:]):
                    times = []
                    for x in inputs:
                        for m in range(args.masks):
                            r = np.random.Generator(np.random.PCG64(1000 * bq + bk + 7919 * m))
                            dens = np.clip(r.uniform(lo, min(hi, 1.0), size=(1, x.heads)), 0.01, 1.0)
                            blocks = block_mask(r, x.heads, x.N, bq, bk, dens, m % 2 == 0)
                            spec = W.MaskSpec(W.MASK_UNIFORM, 1, x.heads, x.N, bq=bq, bk=bk, blocks=blocks)
                            times.append(x.time(spec, d, VARIANTS[d], args.reps))
                    best = best_of(times, f"d={d} N<={n_max} {bq}x{bk} dens[{lo:.2f},{hi:.2f})")
                    rows.append((W.MASK_UNIFORM, bq, bk, n_min, n_max, lo, hi, d) + best)
            # key-list masks (listed keys drawn in clustered runs, mean length 8)
            for M in KEYLIST_M:
                for lo, hi in zip(KEYLIST_EDGES[:-1], KEYLIST_EDGES[1:]):
                    times = []
                    for x in inputs:
                        for m in range(args.masks):
                            spec = keylist_spec(x.N, M, 0.5 * (lo + min(hi, 1.0)), x.heads,
                                                seed=31 * M + 7 * m + int(100 * lo))
                            times.append(x.time(spec, d, VARIANTS_GATHERED[d], args.reps))
                    best = best_of(times, f"d={d} N<={n_max} keylist M={M} frac[{lo:.2f},{hi:.2f})")
                    rows.append((W.MASK_KEYLIST, M, 1, n_min, n_max, lo, hi, d) + best)
            # head-routed (SVG) masks: one row per length bucket
            F = 21 if n_min >= 8192 else 16     # >= 16 frames: at most 8 segments per tile
            times = []
            for x in inputs:
                y = x if x.N % F == 0 else Inputs(x.N // F * F, x.heads, d)
                times.append(y.time(W.svg_mask(1, y.heads, n_frames=F, frame_size=y.N // F), d, VARIANTS[d],
                                    args.reps))
            rows.append((W.MASK_SVG, "*", "*", n_min, n_max, "*", "*", d) + best_of(times, f"d={d} N<={n_max} svg"))
    # anything else: one default row per head dimension
    rows.append(("*", "*", "*", "*", "*", "*", "*", 128, 64, 2, 2, ROWS))
    rows.append(("*", "*", "*", "*", "*", "*", "*", 64, 64, 3, 2, ROWS))
    with open(args.out, "w") as f:
        f.write("# Regime table for GB300 (sm_103a), written by regimes_build.py\n")
        f.write(f"# {time.strftime('%Y-%m-%d')}: {args.masks} seeded masks per class (banded-plus-"
                f"random and random blocks; clustered key lists, one head's repeated; SVG routing), "
                f"4 to 24 heads of 1,024 to 8,000 tokens (short sequences) and 24 of 32,760 (long), "
                f"geometric mean of the forward's time\n")
        f.write("# kind bq bk n_min n_max dens_min dens_max d bn stages ctas orient\n")
        for r in rows:
            f.write(" ".join(f"{x:.2f}" if isinstance(x, float) else str(x) for x in r) + "\n")
    print(f"wrote {len(rows)} rows to {args.out} in {time.time() - t0:.0f} s")


if __name__ == "__main__":
    main()
