// select.cu -- block selection: for each block of queries the key blocks whose
// block means score highest, as the uint8 block mask that tsr_plan takes.
//
//   qm_i = mean of q over block i,  km_j = mean of k over block j,  s_ij = qm_i . km_j
//   kept(i) = forced(i) + the highest s_ij of the others, ties to the lowest j
//
// Two kernels.  pool_kernel reads Q and K once (the bound: HBM) and writes the
// block means; select_kernel computes the scores of a strip of 16 query blocks and
// picks from them.  The scores stay in shared memory, for rows of more than 1,632
// blocks in a slot per CTA of the workspace.
//
// Resolution.  Which block is kept last turns on differences between scores that
// fp32 sums do not resolve, so the selection is made in two steps.  The
// means are sums with a running error term (two-sum), about 48 bits.  The scores
// come from the tensor cores with each mean split into two bf16 terms (three
// products; error about 3e-5 |qm_i| |km_j|, below), and any block whose score
// is within twice that error of the last kept one is scored again from the 48-bit
// means with error terms (about 2^-46 |qm_i| |km_j|); the order of those decides.  A row has two or so such
// blocks, where scoring everything in fp64 would cost 1.3 ms for a 480p layer at
// the 1.25 TFLOP/s of fp64.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace tsr {

namespace {

// Fast scores.  A mean x is split as x = h + l + r, h = bf16(x), l = bf16(x - h).
// The tensor cores sum h h', h l' and l h' in fp32, so a score is off by at most
//     |r| |x'| + |x| |r'| + |l| |l'|                (Cauchy-Schwarz over d)
//     + kSumErr |x| |x'|
// with the norms of both blocks' parts, which pool_kernel takes.  The last term rests
// on an assumption about the hardware: an MMA adds 16 products and the sum so far,
// each cut no higher than 2^-23 of the largest.  Then the 8 MMAs of h h' are off by
// 8 * 17 * 2^-23 = 1.6e-5 at most, and the other chain's terms are 2^-8 of these.
// Measured over 15 million sums of 128 products, of even and uneven magnitudes:
// 1.1e-6 |x| |x'| at most.
constexpr float kSumErr = 2e-5f;

constexpr int kPoolThreads = 128;
constexpr int kSelThreads = 256;
constexpr int kStrip = 16;            // query blocks per CTA of select_kernel
// A strip's scores in shared memory: two CTAs per SM, each with the 8 KB of fragments,
// the largest norms and 1 KB of the system's beside them (1,632 blocks a row).
constexpr int kStripBytes = 104 * 1024;
// Strips of longer rows have their scores in the workspace, one slot per CTA that is
// resident (152 SMs x 3); each CTA takes strip after strip.
constexpr int kScoreSlots = 456;

struct PoolParams {
  const uint4* x[2];            // Q and K
  float* hi[2];                 // block means [B*H][blocks][d], high and low parts
  float* lo[2];
  float4* norm[2];              // |x|, |l|, |r| of the means [B*H][blocks]
  // the means' two bf16 terms in the order of the MMA fragments: [B*H][blocks / 8]
  // [d / 16][32] of {hi(c, c+1), lo(c, c+1), hi(c+2, c+3), lo(c+2, c+3)}, lane 4 g + t
  // holding row g's channels c = 16 kk + 4 t.  (Which channels make a k index is free
  // as long as A and B agree; so a lane's four lie together.)
  uint4* frag[2];
  int32_t frag_rows[2];         // blocks rounded up to 8
  int32_t block[2], n_blocks[2];
  int64_t first_k, n_units;     // blocks of Q, then those of K
  int32_t N;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two neighbouring values as two bf16 terms each: hi = bf16(x), lo = bf16(x - hi).
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x.x, x.y);
  lo = pack_bf16x2(x.x - bf16_lo(hi), x.y - bf16_hi(hi));
}

// (s, e) += x on two channels at once: s + e grows by exactly x up to the rounding
// of e (Knuth's two-sum, seven packed adds).
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {      // a - b, rounded once
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(b), "l"(0xBF800000BF800000ull), "l"(a));
  return d;
}
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  return (static_cast<uint64_t>(__float_as_uint(hi)) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ float lane2(uint64_t v, int i) {
  return __uint_as_float(static_cast<uint32_t>(i ? v >> 32 : v));
}
__device__ __forceinline__ void two_sum(uint64_t& s, uint64_t& e, uint64_t x) {
  const uint64_t t = add2(s, x);
  const uint64_t z = sub2(t, s);
  e = add2(e, add2(sub2(s, sub2(t, z)), sub2(x, z)));
  s = t;
}

__device__ __forceinline__ void two_sum1(float& s, float& e, float x) {
  const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
  s = t;
}

// Block means: one warp per block of rows of one head, or (SHARED: blocks of many
// rows) the four warps of a CTA.  D / 8 lanes across a row, eight loads of 16 bytes
// in flight per lane, no barrier between blocks.  Everything is fp32 pairs: fp64
// sums, at two lanes a clock per SM, took 320 us for a 480p layer, one CTA per block
// (whose loads wait out its barriers) 104 us, a warp per block 65.
template <int D, bool SHARED>
__device__ __forceinline__ void pool_block(const PoolParams& p, int64_t unit, int warp, int lane) {
  constexpr int VR = D / 8, RPW = 32 / VR, WARPS = kPoolThreads / 32;   // RPW rows per warp load
  const int w = unit >= p.first_k ? 1 : 0;
  const int64_t u = unit - (w ? p.first_k : 0);
  const int64_t bh = u / p.n_blocks[w];
  const int blk = static_cast<int>(u - bh * p.n_blocks[w]);
  const int row0 = static_cast<int>(static_cast<int64_t>(blk) * p.block[w]);
  const int rows = min(p.block[w], p.N - row0);
  const uint4* src = p.x[w] + (bh * p.N + row0) * VR + lane % VR;
  uint64_t s[4] = {0, 0, 0, 0}, e[4] = {0, 0, 0, 0};
  constexpr int U = 8, STEP = RPW * (SHARED ? WARPS : 1);
  for (int r = lane / VR + (SHARED ? warp * RPW : 0); r < rows; r += STEP * U) {
    uint4 x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int rr = r + k * STEP;
      x[k] = rr < rows ? __ldg(src + static_cast<int64_t>(rr) * VR) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const uint32_t wd[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) two_sum(s[i], e[i], pair2(bf16_lo(wd[i]), bf16_hi(wd[i])));
    }
  }
  // rows of a warp's other lanes
#pragma unroll
  for (int m = 16; m >= VR; m >>= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t os = __shfl_xor_sync(0xFFFFFFFFu, s[i], m), oe = __shfl_xor_sync(0xFFFFFFFFu, e[i], m);
      two_sum(s[i], e[i], os);
      e[i] = add2(e[i], oe);
    }
  }
  if constexpr (SHARED) {
    __shared__ uint64_t part[WARPS - 1][2][4][32];
    if (warp > 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        part[warp - 1][0][i][lane] = s[i];
        part[warp - 1][1][i][lane] = e[i];
      }
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int k = 0; k < WARPS - 1; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        two_sum(s[i], e[i], part[k][0][i][lane]);
        e[i] = add2(e[i], part[k][1][i][lane]);
      }
    }
  }
  // every lane of a column holds its 8 channels; lane group g finishes 8 / RPW of them
  constexpr int CH = 8 / RPW;
  const int g = lane / VR;
  const float n = static_cast<float>(rows);
  const bool exact = (rows & (rows - 1)) == 0;
  const float inv = 1.f / n;
  float hi[CH], lo[CH], m = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float ts = 0.f, te = 0.f;
#pragma unroll
    for (int k = 0; k < RPW; ++k)
      if (g == k) {
        ts = lane2(s[(k * CH + c) / 2], (k * CH + c) & 1);
        te = lane2(e[(k * CH + c) / 2], (k * CH + c) & 1);
      }
    // the pair made unique (ts the sum rounded, te the rest): how the sum was split
    // between them depends on the rows' order, and equal sums have to give equal means
    const float rest = te;
    te = 0.f;
    two_sum1(ts, te, rest);
    float q, q2;
    if (exact) {                 // a power of two: exact
      q = ts * inv;
      q2 = te * inv;
    } else {                     // the quotient of ts, then that of its exact remainder
      q = __fdiv_rn(ts, n);
      q2 = __fdiv_rn(__fadd_rn(__fmaf_rn(-q, n, ts), te), n);
    }
    hi[c] = __fadd_rn(q, q2);
    lo[c] = __fadd_rn(__fsub_rn(q, hi[c]), q2);
    m = fmaxf(m, fabsf(hi[c]));
  }
  const int64_t o = u * D + (lane % VR) * 8 + g * CH;
  if constexpr (CH == 4) {
    *reinterpret_cast<float4*>(p.hi[w] + o) = make_float4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<float4*>(p.lo[w] + o) = make_float4(lo[0], lo[1], lo[2], lo[3]);
  } else {
    *reinterpret_cast<float2*>(p.hi[w] + o) = make_float2(hi[0], hi[1]);
    *reinterpret_cast<float2*>(p.lo[w] + o) = make_float2(lo[0], lo[1]);
  }
  // the two bf16 terms; l and r for the norms
  const int c0 = (lane % VR) * 8 + g * CH;      // 4 (d = 128) or 2 (d = 64) of a fragment's channels
  const int64_t at = ((bh * (p.frag_rows[w] / 8) + blk / 8) * (D / 16) + c0 / 16) * 32 + (blk % 8) * 4 + (c0 % 16) / 4;
  uint2 t[CH / 2];
  float ll[CH], rr[CH];
#pragma unroll
  for (int i = 0; i < CH / 2; ++i) {
    split2(make_float2(hi[2 * i], hi[2 * i + 1]), t[i].x, t[i].y);
    ll[2 * i] = bf16_lo(t[i].y);
    ll[2 * i + 1] = bf16_hi(t[i].y);
    rr[2 * i] = hi[2 * i] - bf16_lo(t[i].x) - ll[2 * i] + lo[2 * i];
    rr[2 * i + 1] = hi[2 * i + 1] - bf16_hi(t[i].x) - ll[2 * i + 1] + lo[2 * i + 1];
  }
  if constexpr (CH == 4) p.frag[w][at] = make_uint4(t[0].x, t[0].y, t[CH / 2 - 1].x, t[CH / 2 - 1].y);
  else reinterpret_cast<uint2*>(p.frag[w] + at)[(c0 % 4) / 2] = t[0];
  // norms over the largest component, so that small means do not vanish squared
#pragma unroll
  for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
  m = fmaxf(m, FLT_MIN);
  const float over = 1.f / m;
  float n2 = 0.f, l2 = 0.f, r2 = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    n2 = fmaf(hi[c] * over, hi[c] * over, n2);
    l2 = fmaf(ll[c] * over, ll[c] * over, l2);
    r2 = fmaf(rr[c] * over, rr[c] * over, r2);
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) {
    n2 += __shfl_xor_sync(0xFFFFFFFFu, n2, x);
    l2 += __shfl_xor_sync(0xFFFFFFFFu, l2, x);
    r2 += __shfl_xor_sync(0xFFFFFFFFu, r2, x);
  }
  if (lane == 0) {                              // NaN where a mean is
    const float f = m * 1.0001f;
    p.norm[w][u] = make_float4(sqrtf(n2) * f, sqrtf(l2) * f, sqrtf(r2) * f, 0.f);
  }
}

template <int D, bool SHARED>
__global__ void __launch_bounds__(kPoolThreads, 8) pool_kernel(const __grid_constant__ PoolParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = SHARED ? blockIdx.x : blockIdx.x * static_cast<int64_t>(kPoolThreads / 32) + warp;
  grid_launch_dependents();      // select_kernel's blocks take the room of the last of these
  if (unit < p.n_units) pool_block<D, SHARED>(p, unit, warp, lane);
}

// What pool_kernel writes is read with plain loads: select_kernel is resident while it
// still writes, and __ldg is for data that stays as it is for a kernel's whole life.
struct SelParams {
  const float *q_hi, *q_lo, *k_hi, *k_lo;
  const float4 *q_norm, *k_norm;
  const uint4 *q_frag, *k_frag;
  int32_t q_frag_rows, k_frag_rows;
  float* scores;        // [CTA][kStrip][pitch] where a strip does not fit shared memory
  uint8_t* blocks;
  int64_t n_strips;     // of all heads
  int32_t N, bq, bk, nq, nk, strips, pitch;
  int32_t keep, first, diagonal;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Order-preserving integer of a score: a larger score has a larger key, equal
// scores (-0 and 0 too) equal ones, NaN the lowest, 0.
__device__ __forceinline__ uint32_t key32(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unkey32(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ uint64_t key64(double x) {
  if (x != x) return 0ull;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return (u & 0x8000000000000000ull) ? ~u : (u | 0x8000000000000000ull);
}

// A power of two that brings a mean of this norm near 1, and its inverse.
__device__ __forceinline__ float scale_of(float norm, double& back) {
  const int e = min(max(static_cast<int>((__float_as_uint(norm) >> 23) & 255u), 1), 253);
  back = __longlong_as_double(static_cast<int64_t>(e - 127 + 1023) << 52);
  return __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
}

// The order keys of four scores from the 48-bit means, by one warp: lanes 8 c .. 8 c
// + 7 take key block j of their own (all eight get the key; j < 0: 0).  Products with
// their error terms (fma) summed with theirs (two-sum), in fp32 on means scaled to 1
// by powers of two, so that nothing leaves fp32's range; about 2^-46 of |qm| |km|.
// (fp64 runs at two lanes a clock per SM here.)
template <int D>
__device__ __forceinline__ uint64_t exact_keys(const float* qh, const float* ql, float q_norm, const float* kh,
                                               const float* kl, const float4* k_norm, int j, int lane) {
  double q_back, k_back;
  const bool on = j >= 0;
  const int64_t o = static_cast<int64_t>(on ? j : 0);
  const float q_scale = scale_of(q_norm, q_back), k_scale = scale_of(k_norm[o].x, k_back);
  float s = 0.f, e = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int c = i * 8 + (lane & 7);           // float4 of channels
    const float4 a = reinterpret_cast<const float4*>(qh)[c], b = reinterpret_cast<const float4*>(ql)[c];
    const float4 x = reinterpret_cast<const float4*>(kh + o * D)[c];
    const float4 y = reinterpret_cast<const float4*>(kl + o * D)[c];
    const float ah[4] = {a.x, a.y, a.z, a.w}, al[4] = {b.x, b.y, b.z, b.w};
    const float xh[4] = {x.x, x.y, x.z, x.w}, xl[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float u = ah[k] * q_scale, ul = al[k] * q_scale, v = xh[k] * k_scale, vl = xl[k] * k_scale;
      const float p = __fmul_rn(u, v);
      e = __fadd_rn(e, __fmaf_rn(ul, v, __fmaf_rn(u, vl, __fmaf_rn(u, v, -p))));
      two_sum1(s, e, p);
    }
  }
#pragma unroll
  for (int m = 4; m; m >>= 1) {
    // lane i and lane i ^ m add in the same order, the lower lane's sum first
    const float os = __shfl_xor_sync(0xFFFFFFFFu, s, m), oe = __shfl_xor_sync(0xFFFFFFFFu, e, m);
    const bool low = (lane & m) == 0;
    float a = low ? s : os, b = low ? e : oe;
    two_sum1(a, b, low ? os : s);
    s = a;
    e = __fadd_rn(b, low ? oe : e);
  }
  return on ? key64((static_cast<double>(s) + static_cast<double>(e)) * (q_back * k_back)) : 0ull;
}

// The largest key T such that at least `want` of the n keys that `in` admits are
// >= T (there are at least `want` of them).  in(j) and key(j) are evaluated by lane
// j % 32.
template <typename In, typename Key>
__device__ __forceinline__ uint32_t kth_key(int n, int want, int lane, In in, Key key) {
  uint32_t lo = 0u, hi = 0xFFFFFFFFu;
  while (lo < hi) {      // count(>= lo) >= want, count(>= hi + 1) < want
    const uint32_t mid = lo + ((hi - lo) >> 1) + 1u;
    int c = 0;
    for (int j = lane; j < n; j += 32) c += (in(j) && key(j) >= mid) ? 1 : 0;
    c = __reduce_add_sync(0xFFFFFFFFu, c);
    if (c >= want) lo = mid;
    else hi = mid - 1u;
  }
  return lo;
}

// Selection of one row by one warp, its scores row[0 .. nk) (used as scratch).
// KPL > 0: nk <= 32 KPL, the scores in registers, score m * 32 + lane in v[m];
// KPL = 0: any nk, read again where needed.
template <int D, int KPL>
__device__ __forceinline__ void select_row(const SelParams& p, int64_t bh, int i, float* row, float3 k_max, int lane) {
  uint8_t* out = p.blocks + (bh * p.nq + i) * p.nk;
  // forced blocks: [0, first) and, with `diagonal`, [d_lo, d_hi), the key blocks
  // that share a token with the query block
  const int first = min(p.first, p.nk);
  int d_lo = 0, d_hi = 0;
  if (p.diagonal) {
    const int64_t a = static_cast<int64_t>(i) * p.bq;
    const int64_t b = min(a + p.bq, static_cast<int64_t>(p.N)) - 1;
    d_lo = max(static_cast<int>(a / p.bk), first);
    d_hi = max(static_cast<int>(b / p.bk) + 1, d_lo);
  }
  auto forced = [&](int j) -> bool { return j < first || (j >= d_lo && j < d_hi); };
  const int n_forced = first + (d_hi - d_lo), others = p.nk - n_forced;
  const int want = min(p.keep - n_forced, others);
  if (want <= 0 || want == others) {
    const bool all = want == others && want > 0;
    for (int j = lane; j < p.nk; j += 32) out[j] = (all || forced(j)) ? 1 : 0;
    return;
  }
  // the last two terms cover values that the bf16 terms or their products flush
  const float4 qn = p.q_norm[bh * p.nq + i];
  const float q_norm = qn.x;
  const float err2 = 2.002f * (kSumErr * (q_norm * k_max.x) + qn.z * k_max.x + q_norm * k_max.z + qn.y * k_max.y +
                               4e-37f * (q_norm + k_max.x) + 1e-36f);
  bool finite = q_norm * k_max.x <= FLT_MAX && err2 <= FLT_MAX;
  // with finite norms every score is finite; forced blocks and those past nk hold
  // -inf and are never counted (a row has room for whole chunks of 32)
  constexpr int REGS = KPL > 0 ? KPL : 1;
  const int chunks = KPL > 0 ? KPL : (p.nk + 31) / 32;
  for (int j = lane; j < first; j += 32) row[j] = -INFINITY;
  for (int j = d_lo + lane; j < d_hi; j += 32) row[j] = -INFINITY;
  for (int j = p.nk + lane; j < chunks * 32; j += 32) row[j] = -INFINITY;
  __syncwarp();
  float v[REGS];
  if (KPL > 0) {
#pragma unroll
    for (int m = 0; m < REGS; ++m) v[m] = row[m * 32 + lane];
  }
  auto load = [&](int m) -> float { return row[m * 32 + lane]; };
  auto val = [&](int m) -> float { return KPL > 0 ? v[KPL > 0 ? m : 0] : load(m); };
  float above = INFINITY, below = -INFINITY;    // kept for sure above, dropped for sure below
  if (finite) {
    float vmin = INFINITY, vmax = -INFINITY, s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int m = 0; m < chunks; ++m) {
      const float x = val(m);
      const bool real = x != -INFINITY;
      vmax = fmaxf(vmax, x);
      vmin = fminf(vmin, real ? x : INFINITY);
      const float y = real ? x : 0.f;
      s1 += y;
      s2 = fmaf(y, y, s2);
    }
    const uint32_t kmin = __reduce_min_sync(0xFFFFFFFFu, key32(vmin));
    const uint32_t kmax = __reduce_max_sync(0xFFFFFFFFu, key32(vmax));
    // the want-th largest lies in [lo, hi]: c_lo = count(>= lo) >= want, c_hi =
    // count(> hi) < want.  Narrowed until the bracket is inside the fast bound or
    // exactly `want` are above (then it is the smallest of those): first at the
    // quantile of a normal distribution with the row's mean and deviation, then a
    // step by its density there, then by interpolating the counts and every third
    // time by halving, which ends for any distribution.
    float lo = unkey32(kmin), hi = unkey32(kmax);
    float c_lo = static_cast<float>(others), c_hi = 0.f;
    const float n_want = static_cast<float>(want);
#pragma unroll
    for (int x = 16; x; x >>= 1) {
      s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, x);
      s2 += __shfl_xor_sync(0xFFFFFFFFu, s2, x);
    }
    const float mean = s1 / c_lo, dev = sqrtf(fmaxf(s2 / c_lo - mean * mean, 0.f));
    const float z = normcdfinvf(1.f - (n_want - 0.5f) / c_lo);
    float guess = mean + z * dev;
    const float per_count = dev * 2.5066283f * __expf(0.5f * z * z) / c_lo;   // 1 / density
    for (int turn = 0; hi - lo > 0.25f * err2; turn = turn == 4 ? 2 : turn + 1) {
      float mid = guess;
      if (turn >= 2)
        mid = lo + (turn == 4 ? 0.5f : __fdividef(c_lo - n_want + 0.5f, c_lo - c_hi)) * (hi - lo);
      if (!(mid > lo && mid < hi)) mid = lo + 0.5f * (hi - lo);
      if (!(mid > lo && mid < hi)) break;
      int c = 0;
#pragma unroll
      for (int m = 0; m < chunks; ++m) c += val(m) > mid ? 1 : 0;
      c = __reduce_add_sync(0xFFFFFFFFu, c);
      if (c == want) {
        float low = INFINITY;
#pragma unroll
        for (int m = 0; m < chunks; ++m) low = val(m) > mid ? fminf(low, val(m)) : low;
        lo = hi = unkey32(__reduce_min_sync(0xFFFFFFFFu, key32(low)));
        break;
      }
      guess = mid + (static_cast<float>(c) - n_want + 0.5f) * per_count;
      if (c > want) {
        lo = mid;
        c_lo = static_cast<float>(c);
      } else {
        hi = mid;
        c_hi = static_cast<float>(c);
      }
    }
    above = hi + err2;
    below = lo - err2;
    finite = above <= FLT_MAX && below >= -FLT_MAX;
  }
  if (!finite) above = INFINITY;
  // without finite scores and bounds every block that is not forced is scored exactly
  auto sure = [&](float x) -> bool { return finite && x > above; };
  auto near = [&](int m, float x) -> bool {
    return finite ? x >= below && x <= above : m * 32 + lane < p.nk && !forced(m * 32 + lane);
  };
  // the sure ones' bytes, and the number of the near ones
  int n_sure = 0, n_near = 0;
  uint64_t near_bits = 0;                       // KPL > 0: bit m
#pragma unroll
  for (int m = 0; m < chunks; ++m) {
    const int j = m * 32 + lane;
    const float x = val(m);
    const bool in = sure(x), nr = near(m, x);
    n_sure += in ? 1 : 0;
    if (KPL > 0) near_bits |= nr ? 1ull << (m & 63) : 0ull;
    else n_near += nr ? 1 : 0;
    if (j < p.nk) out[j] = in ? 1 : 0;
  }
  if (KPL > 0) n_near = __popcll(near_bits);
  // lanes store the bytes of their own j, so a forced block's 1 comes after its 0
  for (int j = lane; j < first; j += 32) out[j] = 1;
  for (int j = d_lo + ((lane - d_lo) & 31); j < d_hi; j += 32) out[j] = 1;
  n_sure = __reduce_add_sync(0xFFFFFFFFu, n_sure);
  n_near = __reduce_add_sync(0xFFFFFFFFu, n_near);
  const int left = want - n_sure;               // of the near ones, 1 <= left <= n_near
  if (left == n_near) {
    if (KPL > 0) {
      for (; near_bits; near_bits &= near_bits - 1) out[(__ffsll(near_bits) - 1) * 32 + lane] = 1;
    } else {
      for (int m = 0; m < chunks; ++m)
        if (near(m, val(m))) out[m * 32 + lane] = 1;
    }
    return;
  }
  auto keys_of = [&](int j) -> uint64_t {
    const int64_t qo = (bh * p.nq + i) * D, ko = bh * p.nk;
    return exact_keys<D>(p.q_hi + qo, p.q_lo + qo, q_norm, p.k_hi + ko * D, p.k_lo + ko * D, p.k_norm + ko, j, lane);
  };
  if (n_near <= 32) {
    // lane c takes near block c (in any order): its exact key, then its rank
    int my_j = -1, c = 0;
    auto list = [&](int m0, uint32_t bits) {    // bits: this lane's near blocks of chunks m0 ..
      for (uint32_t any; (any = __ballot_sync(0xFFFFFFFFu, bits != 0u)) != 0u; ++c) {
        const int from = __ffs(any) - 1;
        const int m = __ffs(__shfl_sync(0xFFFFFFFFu, bits, from)) - 1;
        if (lane == c) my_j = (m0 + m) * 32 + from;
        if (lane == from) bits &= bits - 1;
      }
    };
    if (KPL > 0) {
      list(0, static_cast<uint32_t>(near_bits));
      if (KPL > 32) list(32, static_cast<uint32_t>(near_bits >> 32));
    } else {
      for (int m0 = 0; m0 < chunks; m0 += 32) {
        uint32_t bits = 0u;
        for (int m = m0; m < min(m0 + 32, chunks); ++m) bits |= near(m, val(m)) ? 1u << (m - m0) : 0u;
        list(m0, bits);
      }
    }
    uint64_t mine = 0;
    for (int o = 0; o < n_near; o += 4) {
      const uint64_t key = keys_of(__shfl_sync(0xFFFFFFFFu, my_j, o + (lane >> 3)));   // o + 3 < 32
      const uint64_t got = __shfl_sync(0xFFFFFFFFu, key, ((lane - o) & 3) * 8);
      if (lane >= o && lane < o + 4) mine = got;
    }
    int rank = 0;
    for (int o = 0; o < n_near; ++o) {
      const uint64_t other = __shfl_sync(0xFFFFFFFFu, mine, o);
      const int other_j = __shfl_sync(0xFFFFFFFFu, my_j, o);
      rank += (other > mine || (other == mine && other_j < my_j)) ? 1 : 0;
    }
    __syncwarp();                               // after the owners' zeros
    if (my_j >= 0 && rank < left) out[my_j] = 1;
    return;
  }
  // Many near blocks (a query block of zeros, equal key blocks, infinities):
  // order them by the upper, then the lower 32 bits of the exact key, which
  // take the place of their scores.  out[j] holds the state meanwhile.
  enum : uint8_t { kOut = 0, kIn = 1, kNear = 2 };
#pragma unroll
  for (int m = 0; m < chunks; ++m) {
    const int j = m * 32 + lane;
    if (j < p.nk) out[j] = near(m, val(m)) ? kNear : (forced(j) || sure(val(m))) ? kIn : kOut;
  }
  __syncwarp();
  auto is_near = [&](int j) { return out[j] == kNear; };
  auto word = [&](int j) { return __float_as_uint(row[j]); };
  int open = left;                              // places left among the kNear
  for (int half = 0; half < 2; ++half) {
    for (int j0 = 0; j0 < p.nk; j0 += 32) {
      const int j = j0 + lane;
      uint32_t b = __ballot_sync(0xFFFFFFFFu, j < p.nk && is_near(j));
      while (b) {                               // four at a time
        int jj = -1;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (b && lane >> 3 == c) jj = j0 + __ffs(b) - 1;
          b &= b - 1;
        }
        const uint64_t key = keys_of(jj);
        if (jj >= 0 && (lane & 7) == 0) row[jj] = __uint_as_float(static_cast<uint32_t>(half ? key : key >> 32));
      }
    }
    __syncwarp();
    const uint32_t t = kth_key(p.nk, open, lane, is_near, word);
    int in = 0;
    for (int j = lane; j < p.nk; j += 32) {
      if (!is_near(j)) continue;
      const uint32_t w = word(j);
      if (w != t) out[j] = w > t ? kIn : kOut;
      in += w > t ? 1 : 0;
    }
    open -= __reduce_add_sync(0xFFFFFFFFu, in);
    __syncwarp();
  }
  // equal exact scores: the lowest j
  for (int j0 = 0; j0 < p.nk; j0 += 32) {
    const int j = j0 + lane;
    const bool tie = j < p.nk && is_near(j);
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, tie);
    if (tie) out[j] = __popc(b & ((1u << lane) - 1u)) < open ? kIn : kOut;
    open -= min(open, __popc(b));
  }
}

// A CTA's strip of kStrip query blocks of one head.
template <int D, int KPL>
__device__ __forceinline__ void select_strip(const SelParams& p, int64_t strip, float* smem) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t bh = strip / p.strips;
  const int i0 = static_cast<int>(strip - bh * p.strips) * kStrip;
  float* sc = KPL == 0 && p.scores ? p.scores + static_cast<int64_t>(blockIdx.x) * kStrip * p.pitch : smem;
  __shared__ float3 k_max_w[kSelThreads / 32];

  // the head's largest norms of the key blocks' parts (NaN counts as infinite)
  float3 km = make_float3(0.f, 0.f, 0.f);
  for (int j = threadIdx.x; j < p.nk; j += kSelThreads) {
    const float4 x = p.k_norm[bh * p.nk + j];
    km.x = x.x <= FLT_MAX ? fmaxf(km.x, x.x) : INFINITY;
    if (km.x > FLT_MAX) break;
    km.y = fmaxf(km.y, x.y);
    km.z = fmaxf(km.z, x.z);
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    km.x = fmaxf(km.x, __shfl_xor_sync(0xFFFFFFFFu, km.x, m));
    km.y = fmaxf(km.y, __shfl_xor_sync(0xFFFFFFFFu, km.y, m));
    km.z = fmaxf(km.z, __shfl_xor_sync(0xFFFFFFFFu, km.z, m));
  }
  if (lane == 0) k_max_w[warp] = km;

  // ---- scores: every warp takes the strip's 16 query blocks, whose A fragments
  // (both bf16 terms) are copied to shared memory, and every eighth pair of groups of
  // 8 key blocks, whose B fragments are read 512 bytes in a row
  {
    constexpr int KK = D / 16;
    __shared__ uint4 frag[2][KK][32];
    const int g = lane >> 2, t = lane & 3;
    for (int x = threadIdx.x; x < 2 * KK * 32; x += kSelThreads) {
      const int group = i0 / 8 + x / (KK * 32);
      frag[x / (KK * 32)][x / 32 % KK][lane] =
          group < p.q_frag_rows / 8 ? p.q_frag[(bh * (p.q_frag_rows / 8) + group) * KK * 32 + x % (KK * 32)]
                                    : make_uint4(0u, 0u, 0u, 0u);
    }
    __syncthreads();
    const uint4* kf = p.k_frag + bh * (p.k_frag_rows / 8) * KK * 32 + lane;
    const int groups = p.k_frag_rows / 8;
    for (int j = warp * 2; j < groups; j += 2 * (kSelThreads / 32)) {
      const int j1 = min(j + 1, groups - 1);
      float c0[2][4] = {}, c1[2][4] = {};
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        const uint4 b0 = kf[(j * KK + kk) * 32], b1 = kf[(j1 * KK + kk) * 32];
        const uint4 a0 = frag[0][kk][lane], a1 = frag[1][kk][lane];
        const uint4 ah = make_uint4(a0.x, a1.x, a0.z, a1.z), al = make_uint4(a0.y, a1.y, a0.w, a1.w);
        mma_16816(c0[0], ah, b0.x, b0.z);
        mma_16816(c0[1], ah, b1.x, b1.z);
        mma_16816(c1[0], ah, b0.y, b0.w);
        mma_16816(c1[1], ah, b1.y, b1.w);
        mma_16816(c1[0], al, b0.x, b0.z);
        mma_16816(c1[1], al, b1.x, b1.z);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int col = (j + n) * 8 + t * 2;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int cc = col + (e & 1), rr = g + ((e & 2) ? 8 : 0);
          if (cc < p.nk) sc[rr * p.pitch + cc] = c0[n][e] + c1[n][e];
        }
      }
    }
  }
  __syncthreads();
  float3 k_max = k_max_w[0];
#pragma unroll
  for (int w = 1; w < kSelThreads / 32; ++w)
    k_max = make_float3(fmaxf(k_max.x, k_max_w[w].x), fmaxf(k_max.y, k_max_w[w].y), fmaxf(k_max.z, k_max_w[w].z));
  for (int rr = warp; rr < kStrip && i0 + rr < p.nq; rr += kSelThreads / 32)
    select_row<D, KPL>(p, bh, i0 + rr, sc + rr * p.pitch, k_max, lane);
}

// CTAs per SM (registers against warps to hide latency): with both kernels, 24 heads
// at 480p, 64 x 64, and 720p, 128 x 128: two 135 / 219 us, three 129 / 211, four 133 / 216.
// At three, 80 registers, the d = 128 variants of 8 to 20 scores a lane spill 4 to 40 bytes.
template <int D, int KPL>
__global__ void __launch_bounds__(kSelThreads, KPL > 20 ? 2 : 3) select_kernel(const __grid_constant__ SelParams p) {
  extern __shared__ float smem[];
  grid_wait();
  if constexpr (KPL > 0) {
    select_strip<D, KPL>(p, blockIdx.x, smem);
  } else {
    for (int64_t strip = blockIdx.x; strip < p.n_strips; strip += gridDim.x) {
      select_strip<D, KPL>(p, strip, smem);
      __syncthreads();                          // before its scores and fragments are overwritten
    }
  }
}

// Scores per lane that the variants of select_kernel hold in registers.
constexpr int kRowRegs[] = {2, 8, 16, 20, 40};

struct Layout {
  int32_t nq, nk, strips, pitch;
  bool in_smem;
  int32_t q_frag_rows, k_frag_rows;          // blocks rounded up to 8
  size_t q_hi, q_lo, k_hi, k_lo, q_norm, k_norm, q_frag, k_frag, scores, total;
};

Layout layout_of(const tsr_select_desc& s) {
  Layout l;
  l.nq = n_blocks(s.N, s.bq);
  l.nk = n_blocks(s.N, s.bk);
  l.strips = (l.nq + kStrip - 1) / kStrip;
  l.pitch = (l.nk + 31) / 32 * 32;           // whole chunks of 32,
  for (int kpl : kRowRegs)                   // as many as the kernel takes,
    if (l.nk <= 32 * kpl) {
      l.pitch = 32 * kpl;
      break;
    }
  l.pitch += 4;                              // rows of a strip starting in different banks
  l.in_smem = static_cast<size_t>(kStrip) * l.pitch * 4 <= kStripBytes;   // else in the workspace
  const size_t BH = static_cast<size_t>(s.B) * s.H;
  size_t at = 0;
  auto take = [&](size_t floats) {
    const size_t o = at;
    at += (floats * 4 + 255) / 256 * 256;
    return o;
  };
  l.q_hi = take(BH * l.nq * s.d);
  l.q_lo = take(BH * l.nq * s.d);
  l.k_hi = take(BH * l.nk * s.d);
  l.k_lo = take(BH * l.nk * s.d);
  l.q_norm = take(BH * l.nq * 4);
  l.k_norm = take(BH * l.nk * 4);
  l.q_frag_rows = (l.nq + 7) / 8 * 8;
  l.k_frag_rows = (l.nk + 7) / 8 * 8;
  l.q_frag = take(BH * l.q_frag_rows * s.d);
  l.k_frag = take(BH * l.k_frag_rows * s.d);
  l.scores = take(l.in_smem ? 0 : std::min<size_t>(kScoreSlots, BH * l.strips) * kStrip * l.pitch);
  l.total = at;
  return l;
}

template <typename Kern>
tsr_status allow_smem(Kern kern, bool (&set)[64]) {
  int dev = 0;
  TSR_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64 || !set[dev]) {
    TSR_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kStripBytes));
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  return TSR_OK;
}

template <int D, int KPL>
tsr_status launch_variant(const PoolParams& pp, const SelParams& sp, size_t smem, bool big_blocks, cudaStream_t st) {
  constexpr int kWarps = kPoolThreads / 32;
  // a CTA per block where a block holds more rows than a warp should read alone
  // (256 rows are 64 kB at d = 128), or where there are too few blocks to fill the GPU
  if (big_blocks || pp.n_units < 2048)
    pool_kernel<D, true><<<static_cast<unsigned>(pp.n_units), kPoolThreads, 0, st>>>(pp);
  else
    pool_kernel<D, false><<<static_cast<unsigned>((pp.n_units + kWarps - 1) / kWarps), kPoolThreads, 0, st>>>(pp);
  TSR_CUDA(cudaGetLastError());
  const unsigned ctas =
      static_cast<unsigned>(sp.scores ? std::min<int64_t>(kScoreSlots, sp.n_strips) : sp.n_strips);
  static bool set[64] = {false};
  if (tsr_status e = allow_smem(select_kernel<D, KPL>, set)) return e;
  TSR_CUDA(launch_dependent(select_kernel<D, KPL>, ctas, kSelThreads, smem, st, sp));
  return TSR_OK;
}

template <int D>
tsr_status launch(const tsr_select_desc& s, const Layout& l, const void* q, const void* k, uint8_t* blocks,
                  uint8_t* ws, cudaStream_t st) {
  const int64_t BH = static_cast<int64_t>(s.B) * s.H;
  auto f = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  PoolParams pp;
  pp.x[0] = static_cast<const uint4*>(q);
  pp.x[1] = static_cast<const uint4*>(k);
  pp.hi[0] = f(l.q_hi);
  pp.lo[0] = f(l.q_lo);
  pp.norm[0] = reinterpret_cast<float4*>(ws + l.q_norm);
  pp.hi[1] = f(l.k_hi);
  pp.lo[1] = f(l.k_lo);
  pp.norm[1] = reinterpret_cast<float4*>(ws + l.k_norm);
  pp.frag[0] = reinterpret_cast<uint4*>(ws + l.q_frag);
  pp.frag[1] = reinterpret_cast<uint4*>(ws + l.k_frag);
  pp.frag_rows[0] = l.q_frag_rows;
  pp.frag_rows[1] = l.k_frag_rows;
  pp.block[0] = s.bq;
  pp.block[1] = s.bk;
  pp.n_blocks[0] = l.nq;
  pp.n_blocks[1] = l.nk;
  pp.first_k = BH * l.nq;
  pp.N = s.N;
  pp.n_units = BH * (static_cast<int64_t>(l.nq) + l.nk);
  SelParams sp;
  sp.q_hi = pp.hi[0];
  sp.q_lo = pp.lo[0];
  sp.k_hi = pp.hi[1];
  sp.k_lo = pp.lo[1];
  sp.q_frag = pp.frag[0];
  sp.k_frag = pp.frag[1];
  sp.q_frag_rows = l.q_frag_rows;
  sp.k_frag_rows = l.k_frag_rows;
  sp.q_norm = pp.norm[0];
  sp.k_norm = pp.norm[1];
  sp.scores = l.in_smem ? nullptr : f(l.scores);
  sp.blocks = blocks;
  sp.N = s.N;
  sp.bq = s.bq;
  sp.bk = s.bk;
  sp.nq = l.nq;
  sp.nk = l.nk;
  sp.strips = l.strips;
  sp.n_strips = BH * l.strips;
  sp.pitch = l.pitch;
  sp.keep = s.keep;
  sp.first = s.first;
  sp.diagonal = s.diagonal;
  const size_t smem = l.in_smem ? static_cast<size_t>(kStrip) * l.pitch * 4 : 0;
  const bool big = std::max(s.bq, s.bk) > 256;
  // scores per lane held in registers: as many as a row has, up to 40
  if (l.nk <= 64) return launch_variant<D, 2>(pp, sp, smem, big, st);
  if (l.nk <= 256) return launch_variant<D, 8>(pp, sp, smem, big, st);
  if (l.nk <= 512) return launch_variant<D, 16>(pp, sp, smem, big, st);
  if (l.nk <= 640) return launch_variant<D, 20>(pp, sp, smem, big, st);
  if (l.nk <= 1280) return launch_variant<D, 40>(pp, sp, smem, big, st);
  return launch_variant<D, 0>(pp, sp, smem, big, st);
}

}  // namespace

size_t select_workspace(const tsr_select_desc& s) { return layout_of(s).total; }

// (Running one part of the heads' selection beside the next part's means, as stages
// of a chain of dependent launches, measured 125 -> 144 us with two parts and 163
// with four at 480p: a strip takes some 50 us in company, and each stage waits for
// the last strips of the one before.)
//
// The arguments have been checked (api_ops.cu).
tsr_status launch_select(const tsr_select_desc& s, const void* q, const void* k, uint8_t* blocks, void* ws,
                         cudaStream_t st) {
  const Layout l = layout_of(s);
  if (s.d == 64) return launch<64>(s, l, q, k, blocks, static_cast<uint8_t*>(ws), st);
  return launch<128>(s, l, q, k, blocks, static_cast<uint8_t*>(ws), st);
}

}  // namespace tsr
