// bwd.cu -- the backward pass of block-sparse attention on tcgen05 tensor cores.
//
// With P = exp(S / sqrt(d) - lse) on the allowed pairs (S = Q K^T), O = P V and
// the gradient dO of O:
//     dV = P^T dO,   dP = dO V^T,   delta_i = sum_c dO_ic O_ic,
//     dS = P o (dP - delta),   dQ = dS K / sqrt(d),   dK = dS^T Q / sqrt(d).
//
// Two kinds of work item share one launch, each owning its output rows, so every
// gradient is summed in registers of the tensor core in a fixed order: no atomics,
// the same bits every run.
//   key items    128 keys with the list of query tiles that see them: dK and dV
//   query items  128 queries with the list of key tiles they see: dQ
// Both recompute S and dP, so a pair costs 7 products (4 + 3) of 2 d flops where one
// pass with atomics on dQ would take 5.  The lists come from two plans of the
// forward's planner: the mask's own and its transpose's, 128-row tiles 64 wide.
//
// Both kinds work alike: 128 stationary rows X1, X2 in shared memory (K, V or Q, dO)
// against a stream of 128-row steps Y1, Y2 (Q, dO or K, V), a step being two tiles of
// the list, not necessarily neighbours:
//     S = X1 Y1^T, dP = X2 Y2^T;   acc1 += dS Y1;   key items: acc2 += P Y2
// so the softmax sees S with the stationary rows on the TMEM lanes.  P and dS are
// rounded to bf16, the operand type of the second products, and written over S
// and dP in TMEM; delta is taken from the bf16 O that the forward stored.  In the 2-norm
// of a small dQ dS's rounding is 0.0018, delta's 0.0010 and the output's own 0.0017.
// The remainder of dS as another operand would be 2 products more on 7, delta from P and
// dP another pass over S and dP.
//
// Two threads issue MMAs, because the pipe runs dry while a lone issuer waits on a
// barrier (a step took 3,635 clocks against 2,240 of MMAs): one S and acc2, the other
// dP and acc1.  MMAs of one thread run in issue order, so a product may overwrite
// columns that the thread's previous product reads.  The issuers run as whole warps
// (elect_lane, ptx.cuh): 2.55 -> 2.05 ms at 8 heads of 16,384 tokens, all blocks on.
//
// The 512 TMEM columns decide how far S and dP run ahead of the softmax:
//   query items         S is free once the softmax holds it in registers; two dP
//   key items, d = 64   two S (acc2 has to read P before an S may overwrite it), one dP
//   key items, d = 128  the accumulators leave 256: one S, one dP
// Where there is one of each, acc1 and the next dP wait for the next S: issued as they
// come, the two threads' products fall together and then wait for the softmax
// together (3,600 clocks a step, 3,460 in turn; 2,460 with whole-warp issuers).  S and
// dP in 64-wide slots, or S alone in two halves, did not pay when one-lane issuers ran
// them (3,526 and 3,634 clocks; a 64-wide product then took as long as a 128-wide one);
// they have not been timed since.
// Few items with long lists (short sequences of few heads): each list is cut in two
// parts with a CTA each, whose fp32 accumulators go to the workspace; the part that
// finishes last adds them up, in the parts' order.
// Warps: 16 softmax (row = TMEM lane, 32 columns each), which also store the
// gradients, a producer (TMA tiles, the rows' statistics) and the two issuers.  Every
// wait is bounded: on expiry the error word is set and the kernel winds down.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "fwd_kernel.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace tsr {

namespace bwd {

constexpr int kSoftmaxWarps = 16, kThreads = (kSoftmaxWarps + 3) * 32;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  CUtensorMap tq, tk, tv, tdo;     // 3-D {d, N, B*H}, 64 x 64 boxes
  const int4 *items_k, *items_q;   // tsr_plan_item, key items (transposed plan), query items
  const int2 *entries_k, *entries_q;
  const uint4 *descs_k, *descs_q;
  const float* nlse2;              // [B*H][Np] -lse * log2(e), -inf for rows with no key and past N
  const float* ndelta;             // [B*H][Np] -delta
  __nv_bfloat16 *dq, *dk, *dv;
  uint32_t* err;
  float4* part;                    // split items: [item * split + part][acc (2)][d / 4][128 rows]
  int32_t* arrived;                // split items: parts finished, [key items, query items]
  int32_t n_key_items, N, Np, split;
  float scale_log2, scale;
  int32_t stall;                   // test only: TSR_BACKWARD_STALL_* bits
  uint64_t timeout_ns;             // bound of every wait
};

// Shared memory and TMEM of an item.
template <int D, bool KEYS>
struct Cfg {
  // Y1 is read by the first product of a step and again by the last, one step later,
  // so it gets a stage more than Y2 where shared memory is short
  static constexpr int S1 = D == 128 ? 3 : 4, S2 = D == 128 ? 2 : 4;
  static constexpr int TILE = 128 * D * 2;          // one 128-row operand
  static constexpr int STAT = 2 * 128 * 4;          // -lse2 and -delta of a step's rows
  static constexpr int X1 = 0, X2 = TILE, Y1 = 2 * TILE, Y2 = Y1 + S1 * TILE, ST = Y2 + S2 * TILE;
  static constexpr int CTRL = ST + 2 * STAT;
  static constexpr int SMEM = CTRL + 512;
  // TMEM: S and dP buffers, then the accumulators
  static constexpr int N_S = KEYS && D == 64 ? 2 : 1, N_DP = KEYS ? 1 : 2;
  static constexpr int S_COL = 0, DP_COL = N_S * 128, A1_COL = DP_COL + N_DP * 128, A2_COL = A1_COL + D;
  static_assert((KEYS ? A2_COL : A1_COL) + D <= 512, "TMEM");
  static constexpr uint32_t IDESC_S = idesc_bf16(128, 128, false, false);
  static constexpr uint32_t IDESC_A = idesc_bf16(128, D, false, true);
  static_assert(SMEM <= 227 * 1024, "shared memory");
  // more than half an SM: one CTA per SM, so the 512 TMEM columns are free at launch
  static_assert(SMEM > 114 * 1024, "one CTA per SM");
};
constexpr int kTmemCols = 512;

struct alignas(8) Ctrl {
  uint64_t x1_full, x2_full;
  uint64_t y1_full[4], y1_empty[4], y2_full[4], y2_empty[4];
  uint64_t st_full[2], st_empty[2];
  uint64_t s_full[2], p_full[2], dp_full[2], ds_full[2], acc_full, final_bar;
  uint64_t never;              // never signalled (stall test)
  uint32_t tmem_base;
  int32_t abort_flag;
  int32_t last;                // split items: this CTA's part was the last of its item
};
static_assert(sizeof(Ctrl) <= 512, "Ctrl");

// Untiled copy global -> shared (16-byte aligned, completion on an mbarrier).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ float4 lds128(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

// (y0, y1) = (x0, x1) * s + (b0, b1)
__device__ __forceinline__ void fma2b(float& y0, float& y1, float x0, float x1, float s, float b0, float b1) {
  asm("{\n\t.reg .b64 xa, sa, ba;\n\tmov.b64 xa, {%2, %3};\n\tmov.b64 sa, {%4, %4};\n\t"
      "mov.b64 ba, {%5, %6};\n\tfma.rn.f32x2 xa, xa, sa, ba;\n\tmov.b64 {%0, %1}, xa;\n\t}"
      : "=f"(y0), "=f"(y1)
      : "f"(x0), "f"(x1), "f"(s), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void mul2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %3};\n\t"
      "mul.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

// Allowed columns [32 sub, 32 sub + 32) of row r of a 64-wide boundary tile (grid
// descriptor).  The segment counts are the same for the whole warp, so the loops
// end early; most tiles have one column segment and need no ranges.
__device__ __forceinline__ uint32_t row_mask(const uint4& d0, const uint4& d1, int r, int sub) {
  const int n_r = d0.x & 0xFF, n_c = (d0.x >> 8) & 0xFF;
  int rs = 0;
#pragma unroll
  for (int k = 1; k < 8; ++k) {
    if (k >= n_r) break;
    if (static_cast<int>(fwd::desc_byte(d0, d1, 2 + k)) <= r) rs = k;
  }
  const uint64_t bits = (static_cast<uint64_t>(d1.w) << 32) | d1.z;
  const uint32_t all = (1u << n_c) - 1u;
  const uint32_t rb = static_cast<uint32_t>(bits >> (rs * 8)) & all;
  if (rb == all && fwd::desc_byte(d0, d1, 10 + n_c) >= 64u) return 0xFFFFFFFFu;
  uint32_t word = 0u;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    if (c >= n_c) break;
    if ((rb >> c) & 1u) {
      const int lo = max(static_cast<int>(fwd::desc_byte(d0, d1, 10 + c)) - 32 * sub, 0);
      const int hi = min(static_cast<int>(fwd::desc_byte(d0, d1, 11 + c)) - 32 * sub, 32);
      if (lo < hi) word |= (hi == 32 ? 0xFFFFFFFFu : (1u << hi) - 1u) & ~((1u << lo) - 1u);
    }
  }
  return word;
}

// 32 lanes x 16 consecutive 32-bit TMEM columns <- 16 registers per thread.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Softmax warps.  A warp takes 32 rows and 32 columns of every step.
template <int D, bool KEYS>
__device__ __forceinline__ void softmax_role(const Params& p, Ctrl& ctrl, uint32_t base, uint32_t tmem, int4 it,
                                             const int2* entries, const uint4* descs, int warp, int lane) {
  using C = Cfg<D, KEYS>;
  volatile int32_t* abort_flag = &ctrl.abort_flag;
  grid_wait();                             // the rows' statistics; the first tiles load meanwhile
  const int grp = warp >> 2;               // columns [32 grp, +32) of the step
  const int part = grp >> 1, sub = grp & 1;
  const int r = (warp & 3) * 32 + lane;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const int32_t n = it.w - it.z, steps = (n + 1) / 2;
  const int64_t row = static_cast<int64_t>(it.y) * 128 + r;
  const bool valid = row < p.N;
  float nlse = 0.f, ndelta = 0.f;
  if (!KEYS) {
    // plain loads: this kernel is resident while bwd_stats_kernel writes them, and
    // __ldg is for data that stays as it is for a kernel's whole life
    nlse = valid ? p.nlse2[static_cast<int64_t>(it.x) * p.Np + row] : -INFINITY;
    ndelta = valid ? p.ndelta[static_cast<int64_t>(it.x) * p.Np + row] : 0.f;
  }
  // The tile's descriptor is loaded one step ahead, its index two, so that no load is
  // waited for where it is issued.
  auto index_of = [&](int32_t j) -> int32_t {
    const int32_t e = 2 * j + part;
    return e < n ? __ldg(&entries[it.z + e]).y : -1;
  };
  int32_t desc_next = index_of(0), desc_after = index_of(1);
  uint4 n0 = make_uint4(0u, 0u, 0u, 0u), n1 = n0;
  auto fetch = [&]() {
    if (desc_next >= 0) {
      n0 = __ldg(&descs[2 * desc_next]);
      n1 = __ldg(&descs[2 * desc_next + 1]);
    }
  };
  fetch();
  bool ok = true;
  for (int32_t j = 0; j < steps; ++j) {
    const bool on = 2 * j + part < n;        // the last step may hold one tile
    const uint32_t allowed = !on ? 0u : desc_next >= 0 ? row_mask(n0, n1, r, sub) : 0xFFFFFFFFu;
    desc_next = desc_after;
    fetch();
    desc_after = index_of(j + 2);
    // a warp whose rows all see nothing here (half of a tile whose other half does)
    // has no arithmetic to do, one whose rows see everything no masking
    const bool none = __all_sync(0xFFFFFFFFu, allowed == 0u);
    const bool mixed = !__all_sync(0xFFFFFFFFu, allowed == 0xFFFFFFFFu);
    const int ab = j & 1;                    // barriers alternate
    const uint32_t phase = (j >> 1) & 1;
    const uint32_t s_col = tmem + lanes + C::S_COL + 32 * grp + (C::N_S == 2 ? 128 * (j & 1) : 0);
    const uint32_t dp_col = tmem + lanes + C::DP_COL + 32 * grp + (C::N_DP == 2 ? 128 * (j & 1) : 0);
    const uint32_t st = base + C::ST + (j & 1) * C::STAT + grp * 128;   // [-lse2 128][-delta 128]
    if (KEYS) {
      if (!mbar_wait_warp(smem_u32(&ctrl.st_full[ab]), phase, abort_flag, p.err, p.timeout_ns)) { ok = false; break; }
    }
    if (!mbar_wait_warp(smem_u32(&ctrl.s_full[ab]), phase, abort_flag, p.err, p.timeout_ns)) { ok = false; break; }
    tc_fence_after();
    uint32_t x[32];                          // S, then P, as float bits
    if (!none) {
      tmem_ld32(s_col, x);
      tc_wait_ld();
    }
    if (!KEYS) {
      // S is in registers: its columns are free for the next product
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctrl.p_full[ab]));
    }
    if (!none) {
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        float4 l = make_float4(nlse, nlse, nlse, nlse);
        if (KEYS) l = lds128(st + i * 4);
        float y[4];
        fma2b(y[0], y[1], __uint_as_float(x[i]), __uint_as_float(x[i + 1]), p.scale_log2, l.x, l.y);
        fma2b(y[2], y[3], __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]), p.scale_log2, l.z, l.w);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i + k] = __float_as_uint(ex2_approx(y[k]));
      }
      if (mixed) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!((allowed >> i) & 1u)) x[i] = 0u;
      }
    }
    if (KEYS) {
      if (on) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          pk[i] = none ? 0u : pack_bf16x2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
        tmem_st16(s_col, pk);
        tc_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctrl.p_full[ab]));
    }
    if (!mbar_wait_warp(smem_u32(&ctrl.dp_full[ab]), phase, abort_flag, p.err, p.timeout_ns)) { ok = false; break; }
    tc_fence_after();
    if (on) {
      uint32_t pk[16];
      if (none) {
#pragma unroll
        for (int i = 0; i < 16; ++i) pk[i] = 0u;
      } else {
        uint32_t a[32];
        tmem_ld32(dp_col, a);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float4 dl = make_float4(ndelta, ndelta, ndelta, ndelta);
          if (KEYS) dl = lds128(st + 512 + i * 4);
          float x0 = __uint_as_float(a[i]), x1 = __uint_as_float(a[i + 1]);
          float x2 = __uint_as_float(a[i + 2]), x3 = __uint_as_float(a[i + 3]);
          fwd::add2(x0, x1, dl.x, dl.y);
          fwd::add2(x2, x3, dl.z, dl.w);
          mul2(x0, x1, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
          mul2(x2, x3, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
          pk[i / 2] = pack_bf16x2(x0, x1);
          pk[i / 2 + 1] = pack_bf16x2(x2, x3);
        }
        if (mixed) {
          // masked pairs: 0 whatever dP holds (P is 0 there, but dP need not be finite)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t two = (allowed >> (2 * i)) & 3u;
            pk[i] &= (two & 1u ? 0xFFFFu : 0u) | (two & 2u ? 0xFFFF0000u : 0u);
          }
        }
      }
      tmem_st16(dp_col, pk);
      tc_wait_st();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(smem_u32(&ctrl.ds_full[ab]));
      if (KEYS) mbar_arrive(smem_u32(&ctrl.st_empty[ab]));
    }
  }
  // ---- epilogue: a quarter of the columns of each accumulator
  constexpr int W = D / 4;
  if (p.split > 1) {
    if (ok && (n == 0 || mbar_wait_warp(smem_u32(&ctrl.acc_full), 0, abort_flag, p.err, p.timeout_ns))) {
      tc_fence_after();
#pragma unroll
      for (int w = 0; w < (KEYS ? 2 : 1); ++w) {
        const uint32_t col = tmem + lanes + (w ? C::A2_COL : C::A1_COL) + grp * W;
        float4* dst = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + w) * (D / 4) * 128 + grp * (W / 4) * 128 + r;
#pragma unroll
        for (int c = 0; c < W; c += 16) {
          uint32_t a[16] = {};
          if (n > 0) {
            tmem_ld16(col + c, a);
            tc_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[(c / 4 + i) * 128] = make_float4(__uint_as_float(a[4 * i]), __uint_as_float(a[4 * i + 1]),
                                                 __uint_as_float(a[4 * i + 2]), __uint_as_float(a[4 * i + 3]));
        }
      }
      __threadfence();
    }
  } else if (ok && n > 0) {
    if (mbar_wait_warp(smem_u32(&ctrl.acc_full), 0, abort_flag, p.err, p.timeout_ns)) {
      tc_fence_after();
#pragma unroll
      for (int w = 0; w < (KEYS ? 2 : 1); ++w) {
        __nv_bfloat16* out = KEYS ? (w ? p.dv : p.dk) : p.dq;
        const float f = w ? 1.f : p.scale;
        const uint32_t col = tmem + lanes + (w ? C::A2_COL : C::A1_COL) + grp * W;
        uint4* dst =
            reinterpret_cast<uint4*>(out + (static_cast<int64_t>(it.x) * p.N + (valid ? row : 0)) * D + grp * W);
#pragma unroll
        for (int c = 0; c < W; c += 16) {
          uint32_t a[16];
          tmem_ld16(col + c, a);
          tc_wait_ld();
          if (valid) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              dst[c / 8 + i] = make_uint4(
                  pack_bf16x2(__uint_as_float(a[8 * i]) * f, __uint_as_float(a[8 * i + 1]) * f),
                  pack_bf16x2(__uint_as_float(a[8 * i + 2]) * f, __uint_as_float(a[8 * i + 3]) * f),
                  pack_bf16x2(__uint_as_float(a[8 * i + 4]) * f, __uint_as_float(a[8 * i + 5]) * f),
                  pack_bf16x2(__uint_as_float(a[8 * i + 6]) * f, __uint_as_float(a[8 * i + 7]) * f));
          }
        }
      }
    }
  } else if (ok && valid) {
#pragma unroll
    for (int w = 0; w < (KEYS ? 2 : 1); ++w) {
      __nv_bfloat16* out = KEYS ? (w ? p.dv : p.dk) : p.dq;
      uint4* dst = reinterpret_cast<uint4*>(out + (static_cast<int64_t>(it.x) * p.N + row) * D + grp * W);
#pragma unroll
      for (int i = 0; i < W / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

template <int D, bool KEYS>
__device__ __forceinline__ void producer_role(const Params& p, Ctrl& ctrl, uint32_t base, int4 it,
                                              const int2* entries) {
  using C = Cfg<D, KEYS>;
  volatile int32_t* abort_flag = &ctrl.abort_flag;
  const int32_t n = it.w - it.z, steps = (n + 1) / 2, bh = it.x;
  const CUtensorMap *x1 = KEYS ? &p.tk : &p.tq, *x2 = KEYS ? &p.tv : &p.tdo;
  const CUtensorMap *y1 = KEYS ? &p.tq : &p.tk, *y2 = KEYS ? &p.tdo : &p.tv;
  if (steps == 0) return;
  // one 64-row tile into rows [64 * part, +64) of a 128-row operand
  auto tile = [&](const CUtensorMap* map, uint32_t dst, int part, int32_t row, uint32_t bar) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * 128 * 128 + part * 64 * 128, map, bar, c * 64, row, bh);
  };
  auto stationary = [&](const CUtensorMap* map, uint32_t dst, uint64_t* bar) {
    mbar_arrive_expect_tx(smem_u32(bar), C::TILE);
    tile(map, dst, 0, it.y * 128, smem_u32(bar));
    tile(map, dst, 1, it.y * 128 + 64, smem_u32(bar));
  };
  int32_t i1 = 0, i2 = 0, is = 0;       // stages filled, for the drain
  bool x2_issued = false;
  stationary(x1, base + C::X1, &ctrl.x1_full);
  for (int32_t j = 0; j < steps; ++j) {
    const int parts = 2 * j + 1 < n ? 2 : 1;
    const int32_t k0 = __ldg(&entries[it.z + 2 * j]).x;
    const int32_t k1 = parts == 2 ? __ldg(&entries[it.z + 2 * j + 1]).x : 0;
    const int a = j % C::S1, b = j % C::S2;
    auto stream = [&](const CUtensorMap* map, uint32_t dst, uint64_t* bar) {
      mbar_arrive_expect_tx(smem_u32(bar), parts * (C::TILE / 2));
      tile(map, dst, 0, k0, smem_u32(bar));
      if (parts == 2) tile(map, dst, 1, k1, smem_u32(bar));
    };
    if (!mbar_wait(smem_u32(&ctrl.y1_empty[a]), ((j / C::S1) & 1) ^ 1, abort_flag, p.err, p.timeout_ns)) break;
    stream(y1, base + C::Y1 + a * C::TILE, &ctrl.y1_full[a]);
    ++i1;
    if (KEYS) {
      const uint32_t bar = smem_u32(&ctrl.st_full[j & 1]), dst = base + C::ST + (j & 1) * C::STAT;
      if (!mbar_wait(smem_u32(&ctrl.st_empty[j & 1]), ((j >> 1) & 1) ^ 1, abort_flag, p.err, p.timeout_ns)) break;
      if (j == 0) grid_wait();
      mbar_arrive_expect_tx(bar, parts * 512);
      const int64_t o = static_cast<int64_t>(bh) * p.Np;
      bulk_load(dst, p.nlse2 + o + k0, 256, bar);
      bulk_load(dst + 512, p.ndelta + o + k0, 256, bar);
      if (parts == 2) {
        bulk_load(dst + 256, p.nlse2 + o + k1, 256, bar);
        bulk_load(dst + 768, p.ndelta + o + k1, 256, bar);
      }
      ++is;
    }
    if (j == 0) {
      stationary(x2, base + C::X2, &ctrl.x2_full);
      x2_issued = true;
    }
    if (!mbar_wait(smem_u32(&ctrl.y2_empty[b]), ((j / C::S2) & 1) ^ 1, abort_flag, p.err, p.timeout_ns)) break;
    stream(y2, base + C::Y2 + b * C::TILE, &ctrl.y2_full[b]);
    ++i2;
  }
  if (*abort_flag) {
    // let the copies in flight land before the CTA ends
    volatile int32_t no = 0;
    mbar_wait(smem_u32(&ctrl.x1_full), 0, &no, p.err);
    if (x2_issued) mbar_wait(smem_u32(&ctrl.x2_full), 0, &no, p.err);
    for (int32_t k = max(0, i1 - C::S1); k < i1; ++k)
      mbar_wait(smem_u32(&ctrl.y1_full[k % C::S1]), (k / C::S1) & 1, &no, p.err);
    for (int32_t k = max(0, i2 - C::S2); k < i2; ++k)
      mbar_wait(smem_u32(&ctrl.y2_full[k % C::S2]), (k / C::S2) & 1, &no, p.err);
    for (int32_t k = max(0, is - 2); k < is; ++k)
      mbar_wait(smem_u32(&ctrl.st_full[k & 1]), (k >> 1) & 1, &no, p.err);
  }
}

// The two MMA issuers.  FIRST owns S's columns: S, and acc2 (which reads P there).
// The other owns dP's: dP, and acc1 (which reads dS there).
template <int D, bool KEYS, bool FIRST>
__device__ __forceinline__ void mma_role(const Params& p, Ctrl& ctrl, uint32_t base, uint32_t tmem, int4 it) {
  using C = Cfg<D, KEYS>;
  volatile int32_t* abort_flag = &ctrl.abort_flag;
  const int32_t n = it.w - it.z, steps = (n + 1) / 2;
  const uint32_t elect = elect_lane();
  // test only: this issuer does one step, then waits for a barrier that nobody signals
  const int32_t last = (p.stall & (FIRST ? 1 : 2) << (KEYS ? 0 : 2)) ? min(steps, 1) : steps;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return mbar_wait_warp(smem_u32(bar), parity, abort_flag, p.err, p.timeout_ns);
  };
  // barriers of step j alternate, so that no phase runs two ahead of a waiter
  auto done = [&](uint64_t (&b)[2], int32_t j) { return wait(&b[j & 1], (j >> 1) & 1); };
  // D[128 x 128] = X Y^T over d
  auto outer = [&](uint32_t col, uint32_t sx, uint32_t sy) {
    tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t o = (kk >> 2) * 128 * 128 + (kk & 3) * 32;
      mma_bf16_ss(elect, tmem + col, sdesc_sw128(sx + o, 16, 1024), sdesc_sw128(sy + o, 16, 1024), C::IDESC_S, kk > 0);
    }
  };
  // acc[128 x D] += A (bf16, TMEM) Y over the step's rows; P and dS lie 16 columns
  // (32 rows of Y) per softmax warp, 32 apart
  auto inner = [&](uint32_t acc, uint32_t col, uint32_t sy, int32_t j) {
    tc_fence_after();
    const int kks = 2 * j + 1 < n ? 8 : 4;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      if (kk < kks)
        mma_bf16_ts(elect, tmem + acc, tmem + col + (kk >> 1) * 32 + (kk & 1) * 8,
                    sdesc_sw128(sy + kk * 16 * 128, 128 * 128, 1024), C::IDESC_A, (j > 0 || kk > 0) ? 1u : 0u);
  };
  auto y1 = [&](int32_t j) { return base + C::Y1 + (j % C::S1) * C::TILE; };
  auto y2 = [&](int32_t j) { return base + C::Y2 + (j % C::S2) * C::TILE; };
  auto y2_full = [&](int32_t j) { return wait(&ctrl.y2_full[j % C::S2], (j / C::S2) & 1); };
  int32_t j = 0;                               // steps whose products are issued
  if constexpr (FIRST) {
    auto s_col = [&](int32_t j) { return static_cast<uint32_t>(C::S_COL + (C::N_S == 2 ? 128 * (j & 1) : 0)); };
    auto do_s = [&](int32_t j) -> bool {
      if (!wait(&ctrl.y1_full[j % C::S1], (j / C::S1) & 1)) return false;
      outer(s_col(j), base + C::X1, y1(j));
      mma_commit(elect, smem_u32(&ctrl.s_full[j & 1]));
      return true;
    };
    const bool ok = steps > 0 && wait(&ctrl.x1_full, 0) && do_s(0) && (C::N_S == 1 || steps == 1 || do_s(1));
    for (; ok && j < last; ++j) {
      if (KEYS && !y2_full(j)) break;
      if (!done(ctrl.p_full, j)) break;
      if (KEYS) {
        inner(C::A2_COL, s_col(j), y2(j), j);
        mma_commit(elect, smem_u32(&ctrl.y2_empty[j % C::S2]));
      }
      if (j + C::N_S < steps && !do_s(j + C::N_S)) break;
    }
  } else {
    auto dp_col = [&](int32_t j) { return static_cast<uint32_t>(C::DP_COL + (C::N_DP == 2 ? 128 * (j & 1) : 0)); };
    auto do_dp = [&](int32_t j) -> bool {
      if (!y2_full(j)) return false;
      outer(dp_col(j), base + C::X2, y2(j));
      mma_commit(elect, smem_u32(&ctrl.dp_full[j & 1]));
      mma_commit(elect, smem_u32(&ctrl.y2_empty[j % C::S2]));
      return true;
    };
    const bool ok = steps > 0 && wait(&ctrl.x2_full, 0) && do_dp(0) && (C::N_DP == 1 || steps == 1 || do_dp(1));
    for (; ok && j < last; ++j) {
      if (!done(ctrl.ds_full, j)) break;
      // one S and one dP: acc1 and dP(j+1) wait for S(j+1), so that the pipe works on
      // them while the softmax has S(j+1) to work on, and on acc2 and S while it has dP
      if (KEYS && C::N_S == 1 && j + 1 < steps && !done(ctrl.s_full, j + 1)) break;
      // Y1 has landed: S of this step was computed from it
      inner(C::A1_COL, dp_col(j), y1(j), j);
      mma_commit(elect, smem_u32(&ctrl.y1_empty[j % C::S1]));
      if (j + C::N_DP < steps && !do_dp(j + C::N_DP)) break;
    }
  }
  // the accumulators are whole once all that both threads issued has completed; after
  // an abort they are not, and only TMEM can be released
  if (last < steps) wait(&ctrl.never, 0);
  if (j == steps) mma_commit(elect, smem_u32(&ctrl.acc_full));
  mma_commit(elect, smem_u32(&ctrl.final_bar));
  volatile int32_t no = 0;
  mbar_wait(smem_u32(&ctrl.final_bar), 0, &no, p.err);
}

// The sum of a split item's parts, by the warps that store the accumulators.
template <int D, bool KEYS>
__device__ __forceinline__ void merge_parts(const Params& p, int4 it, int64_t unit0, int warp, int lane) {
  constexpr int W = D / 4;
  const int grp = warp >> 2, r = (warp & 3) * 32 + lane;
  const int64_t row = static_cast<int64_t>(it.y) * 128 + r;
  if (row >= p.N) return;
#pragma unroll
  for (int w = 0; w < (KEYS ? 2 : 1); ++w) {
    __nv_bfloat16* out = KEYS ? (w ? p.dv : p.dk) : p.dq;
    const float f = w ? 1.f : p.scale;
    uint4* dst = reinterpret_cast<uint4*>(out + (static_cast<int64_t>(it.x) * p.N + row) * D + grp * W);
#pragma unroll
    for (int c = 0; c < W / 8; ++c) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
      for (int q = 0; q < p.split; ++q) {
        const float4* src = p.part + ((unit0 + q) * 2 + w) * (D / 4) * 128 + (grp * (W / 4) + 2 * c) * 128 + r;
        const float4 x = __ldcg(src), y = __ldcg(src + 128);
        a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
        b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
      }
      dst[c] = make_uint4(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f),
                          pack_bf16x2(b.x * f, b.y * f), pack_bf16x2(b.z * f, b.w * f));
    }
  }
}

// A work item, or its part `part` of p.split: whole steps, in near-equal shares.
template <bool KEYS>
__device__ __forceinline__ int4 item_of(const Params& p, int32_t item, int32_t part) {
  int4 it = __ldg((KEYS ? p.items_k : p.items_q) + 2 * static_cast<int64_t>(item));
  if (p.split > 1) {
    const int32_t n = it.w - it.z, steps = (n + 1) / 2;
    const int32_t a = static_cast<int32_t>(static_cast<int64_t>(steps) * part / p.split);
    const int32_t b = static_cast<int32_t>(static_cast<int64_t>(steps) * (part + 1) / p.split);
    it.w = it.z + min(n, 2 * b);
    it.z += 2 * a;
  }
  return it;
}

template <int D, bool KEYS>
__device__ __forceinline__ void roles(const Params& p, Ctrl& ctrl, uint32_t base, uint32_t tmem, int4 it,
                                      int warp, int lane) {
  const int2* entries = KEYS ? p.entries_k : p.entries_q;
  if (warp < kSoftmaxWarps) {
    softmax_role<D, KEYS>(p, ctrl, base, tmem, it, entries, KEYS ? p.descs_k : p.descs_q, warp, lane);
  } else if (warp == kSoftmaxWarps) {
    if (lane == 0) producer_role<D, KEYS>(p, ctrl, base, it, entries);
  } else if (warp == kSoftmaxWarps + 1) {
    mma_role<D, KEYS, true>(p, ctrl, base, tmem, it);
  } else {
    mma_role<D, KEYS, false>(p, ctrl, base, tmem, it);
  }
  __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) bsa_bwd_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  Ctrl& ctrl = *reinterpret_cast<Ctrl*>(smem + Cfg<D, true>::CTRL);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int32_t part = p.split > 1 ? blockIdx.x % p.split : 0, item = p.split > 1 ? blockIdx.x / p.split : blockIdx.x;
  const bool keys = item < p.n_key_items;
  if (base & 1023u) {       // swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(p.err, DEV_ERR_INTERNAL);
    return;
  }
  if (threadIdx.x == 0) {
    for (uint64_t* b : {&ctrl.x1_full, &ctrl.x2_full}) mbar_init(smem_u32(b), 1);
    mbar_init(smem_u32(&ctrl.acc_full), 2);
    mbar_init(smem_u32(&ctrl.final_bar), 2);
    mbar_init(smem_u32(&ctrl.never), 1);
    for (int i = 0; i < 4; ++i) {
      for (uint64_t* b : {&ctrl.y1_full[i], &ctrl.y1_empty[i], &ctrl.y2_full[i]}) mbar_init(smem_u32(b), 1);
      mbar_init(smem_u32(&ctrl.y2_empty[i]), keys ? 2 : 1);     // dP, and acc2 of key items
    }
    for (int i = 0; i < 2; ++i) {
      for (uint64_t* b : {&ctrl.s_full[i], &ctrl.dp_full[i], &ctrl.st_full[i]}) mbar_init(smem_u32(b), 1);
      for (uint64_t* b : {&ctrl.p_full[i], &ctrl.ds_full[i], &ctrl.st_empty[i]}) mbar_init(smem_u32(b), kSoftmaxWarps);
    }
    ctrl.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kSoftmaxWarps + 1) {
    tmem_alloc(smem_u32(&ctrl.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, ctrl.tmem_base, 0);
  const int4 it = keys ? item_of<true>(p, item, part) : item_of<false>(p, item - p.n_key_items, part);
  if (keys) roles<D, true>(p, ctrl, base, tmem, it, warp, lane);
  else roles<D, false>(p, ctrl, base, tmem, it, warp, lane);
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (p.split > 1) {
    // every warp's part is written (and fenced): count it; the last CTA adds them up
    if (threadIdx.x == 0) ctrl.last = !ctrl.abort_flag && atomicAdd(p.arrived + item, 1) == p.split - 1;
    __syncthreads();
    if (ctrl.last && warp < kSoftmaxWarps) {
      __threadfence();
      const int64_t unit0 = static_cast<int64_t>(item) * p.split;
      if (keys) merge_parts<D, true>(p, it, unit0, warp, lane);
      else merge_parts<D, false>(p, it, unit0, warp, lane);
    }
  }
}

// Per query row: -lse in base 2 and -delta, delta = sum dO o O (fp32), one row per D / 8
// lanes; rows past N of the padded arrays get P = 0.  Also clears the counters of
// split items.  HBM-bound: reads O and dO.
template <int D>
__global__ void __launch_bounds__(256) bwd_stats_kernel(const uint4* __restrict__ o, const uint4* __restrict__ g,
                                                        const float* __restrict__ lse, float* __restrict__ nlse2,
                                                        float* __restrict__ ndelta, int64_t rows_p, int32_t N,
                                                        int32_t Np, int32_t* __restrict__ arrived, int32_t n_arrived) {
  constexpr int VR = D / 8;
  const int64_t row = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) / VR;
  const int v = threadIdx.x % VR;
  grid_launch_dependents();
  if (blockIdx.x == 0)
    for (int k = threadIdx.x; k < n_arrived; k += blockDim.x) arrived[k] = 0;
  if (row >= rows_p) return;       // whole groups of VR lanes leave together
  const int64_t bh = row / Np;
  const int32_t i = static_cast<int32_t>(row - bh * Np);
  float s = 0.f;
  float l = -INFINITY;
  if (i < N) {
    const int64_t src = (bh * N + i) * VR + v;
    const uint4 a = __ldg(o + src), b = __ldg(g + src);
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s = fmaf(__uint_as_float(x[k] << 16), __uint_as_float(y[k] << 16), s);
      s = fmaf(__uint_as_float(x[k] & 0xFFFF0000u), __uint_as_float(y[k] & 0xFFFF0000u), s);
    }
    l = -__ldg(lse + bh * N + i) * kLog2e;
    if (l == INFINITY) l = -INFINITY;        // no allowed key: P = 2^(s - inf) = 0
  }
  const uint32_t grp = VR == 32 ? 0xFFFFFFFFu : ((1u << VR) - 1u) << ((threadIdx.x & 31) / VR * VR);
#pragma unroll
  for (int m = VR / 2; m; m >>= 1) s += __shfl_xor_sync(grp, s, m);
  if (v == 0) {
    nlse2[row] = l;
    ndelta[row] = -s;
  }
}

// blocks [heads][nq][nk] -> [heads][nk][nq]
__global__ void transpose_blocks_kernel(const uint8_t* __restrict__ src, uint8_t* __restrict__ dst, int32_t nq,
                                        int32_t nk, int32_t tiles_k) {
  __shared__ uint8_t t[32][33];
  const int64_t base = static_cast<int64_t>(blockIdx.y) * nq * nk;
  const int q0 = (blockIdx.x / tiles_k) * 32, k0 = (blockIdx.x % tiles_k) * 32;
  for (int y = threadIdx.y; y < 32; y += 8) {
    const int q = q0 + y, k = k0 + threadIdx.x;
    if (q < nq && k < nk) t[y][threadIdx.x] = src[base + static_cast<int64_t>(q) * nk + k];
  }
  __syncthreads();
  for (int y = threadIdx.y; y < 32; y += 8) {
    const int k = k0 + y, q = q0 + threadIdx.x;
    if (q < nq && k < nk) dst[base + static_cast<int64_t>(k) * nq + q] = t[threadIdx.x][y];
  }
}

template <int D>
tsr_status launch(const Params& prm, int64_t ctas, int device, cudaStream_t st) {
  auto kern = bsa_bwd_kernel<D>;
  static OncePerDevice once;
  if (tsr_status e = allow_smem(kern, Cfg<D, true>::SMEM, device, once)) return e;
  TSR_CUDA(launch_dependent(kern, static_cast<unsigned>(ctas), kThreads, Cfg<D, true>::SMEM, st, prm));
  return TSR_OK;
}

}  // namespace bwd

tsr_status launch_transpose_blocks(const uint8_t* src, uint8_t* dst, int64_t heads, int32_t nq, int32_t nk,
                                   cudaStream_t st) {
  const int32_t tq = (nq + 31) / 32, tk = (nk + 31) / 32;
  if (static_cast<int64_t>(tq) * tk >= (int64_t{1} << 31)) return fail(TSR_ERR_UNSUPPORTED, "too many blocks");
  for (int64_t h0 = 0; h0 < heads; h0 += 65535) {     // the grid's y limit
    const int64_t n = std::min<int64_t>(65535, heads - h0), o = h0 * nq * nk;
    bwd::transpose_blocks_kernel<<<dim3(static_cast<unsigned>(tq * tk), static_cast<unsigned>(n)), dim3(32, 8), 0,
                                   st>>>(src + o, dst + o, nq, nk, tk);
    TSR_CUDA(cudaGetLastError());
  }
  return TSR_OK;
}

namespace {

// Parts per item that the workspace has room for: two where that still leaves an SM
// for each.
int32_t max_split(const tsr_plan_impl* Q, const tsr_plan_impl* K) {
  return (Q->n_items + K->n_items) * 2 <= num_sms(Q->device) ? 2 : 1;
}

struct BwdLayout {
  size_t stats, arrived, part, total;
  int32_t split;
};
BwdLayout backward_layout(const tsr_plan_impl* Q, const tsr_plan_impl* K) {
  BwdLayout l;
  const int64_t items = Q->n_items + K->n_items;
  l.split = max_split(Q, K);
  auto round = [](size_t b) { return (b + 255) / 256 * 256; };
  l.stats = 0;
  l.arrived = round(static_cast<size_t>(2) * Q->B * Q->H * ((Q->N + 63) / 64 * 64) * sizeof(float));
  l.part = l.arrived + (l.split > 1 ? round(sizeof(int32_t) * items) : 0);
  l.total = l.part + (l.split > 1 ? static_cast<size_t>(items) * l.split * 2 * 128 * Q->d * sizeof(float) : 0);
  return l;
}

}  // namespace

size_t backward_workspace(const tsr_plan_impl* plan_q, const tsr_plan_impl* plan_k) {
  return backward_layout(plan_q, plan_k).total;
}

tsr_status launch_backward(const BwdArgs& a, cudaStream_t st) {
  const tsr_plan_impl *Q = a.plan_q, *K = a.plan_k;
  const int32_t N = Q->N, D = Q->d, Np = (N + 63) / 64 * 64;
  const int64_t BH = static_cast<int64_t>(Q->B) * Q->H;
  bwd::Params p;
  memset(&p, 0, sizeof p);
  const uint64_t d = D, n = N, bh = BH;
  if (!encode_tmap_3d(&p.tq, a.q, d, n, bh, 64, 64) || !encode_tmap_3d(&p.tk, a.k, d, n, bh, 64, 64) ||
      !encode_tmap_3d(&p.tv, a.v, d, n, bh, 64, 64) || !encode_tmap_3d(&p.tdo, a.dout, d, n, bh, 64, 64))
    return fail(TSR_ERR_CUDA, "cuTensorMapEncodeTiled failed (pointer alignment or shape)");
  p.items_k = static_cast<const int4*>(K->items);
  p.items_q = static_cast<const int4*>(Q->items);
  p.entries_k = static_cast<const int2*>(K->entries);
  p.entries_q = static_cast<const int2*>(Q->entries);
  p.descs_k = static_cast<const uint4*>(K->descs);
  p.descs_q = static_cast<const uint4*>(Q->descs);
  float* nlse2 = static_cast<float*>(a.workspace);
  float* ndelta = nlse2 + BH * Np;
  p.nlse2 = nlse2;
  p.ndelta = ndelta;
  p.dq = static_cast<__nv_bfloat16*>(a.dq);
  p.dk = static_cast<__nv_bfloat16*>(a.dk);
  p.dv = static_cast<__nv_bfloat16*>(a.dv);
  p.err = Q->err;
  p.n_key_items = static_cast<int32_t>(K->n_items);
  p.N = N;
  p.Np = Np;
  p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
  // Items are cut in two where the longest list leaves 16 tiles to a part.  One head,
  // d = 128, density 0.3: 4,096 tokens 42 -> 36 us; with 11 tiles to a part (2,048
  // tokens) 26 -> 27 us, the partial sums costing what the shorter lists save.
  const BwdLayout l = backward_layout(Q, K);
  p.stall = a.stall;
  p.timeout_ns = a.stall ? 100000000ull : kWaitTimeoutNs;
  p.split = std::max(Q->max_item_len, K->max_item_len) >= 16 * l.split ? l.split : 1;
  p.part = reinterpret_cast<float4*>(static_cast<uint8_t*>(a.workspace) + l.part);
  p.arrived = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(a.workspace) + l.arrived);
  const int64_t items = K->n_items + Q->n_items, ctas = items * p.split;
  const int32_t n_arrived = p.split > 1 ? static_cast<int32_t>(items) : 0;
  const int64_t rows = BH * Np;
  const int64_t stat_blocks = (rows * (D / 8) + 255) / 256;
  if (stat_blocks >= (int64_t{1} << 31)) return fail(TSR_ERR_UNSUPPORTED, "too many rows");
  const uint4 *o = static_cast<const uint4*>(a.out), *g = static_cast<const uint4*>(a.dout);
  if (D == 64)
    bwd::bwd_stats_kernel<64><<<static_cast<unsigned>(stat_blocks), 256, 0, st>>>(o, g, a.lse, nlse2, ndelta, rows, N, Np,
                                                                           p.arrived, n_arrived);
  else
    bwd::bwd_stats_kernel<128><<<static_cast<unsigned>(stat_blocks), 256, 0, st>>>(o, g, a.lse, nlse2, ndelta, rows, N, Np,
                                                                           p.arrived, n_arrived);
  TSR_CUDA(cudaGetLastError());
  return D == 64 ? bwd::launch<64>(p, ctas, Q->device, st) : bwd::launch<128>(p, ctas, Q->device, st);
}

}  // namespace tsr
