// select.cu -- block selection: for each block of queries the key blocks whose
// block means score highest, as the uint8 block mask that tsr_plan takes.
//
//   qm_i = mean of q over block i,  km_j = mean of k over block j,  s_ij = qm_i . km_j
//   kept(i) = forced(i) + the highest s_ij of the others, ties to the lowest j
//
// Two kernels.  pool_kernel reads Q and K once (the bound: HBM) and writes the
// block means; select_kernel computes a strip of scores and picks from it, the
// scores never leaving shared memory.
//
// Exactness.  Which block is kept last turns on differences between scores that
// fp32 sums do not resolve, so the selection is made exact in two steps.  The
// means are sums with a running error term (two-sum), about 48 bits.  The scores
// come from the tensor cores with each mean split into two bf16 terms (three
// products; error at most kScoreErr * |qm_i| |km_j|), and any block whose score
// is within twice that error of the last kept one is scored again in fp64 from
// the 48-bit means; the order of those decides.  A row has a handful of such
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

// |approximate score - score| <= kScoreErr |qm| |km| (Cauchy-Schwarz over d):
// a bf16 term is off by 2^-8 of its value at most, two terms by 2^-16, so the
// dropped products are at most 3 * 2^-16; 24 accumulations of 16 products in
// fp32, truncating, add less than 24 * 2^-22.  Together 5.2e-5.
constexpr float kScoreErr = 1e-4f;

constexpr int kPoolThreads = 128;
constexpr int kSelThreads = 256;
constexpr int kStrip = 16;            // query blocks per CTA of select_kernel
constexpr int kStripBytes = 112 * 1024;   // a strip's scores, two CTAs per SM

struct PoolParams {
  const uint4* x[2];            // Q and K
  float* hi[2];                 // block means [B*H][blocks][d], high and low parts
  float* lo[2];
  float* norm[2];               // |mean| [B*H][blocks]
  int32_t block[2], n_blocks[2];
  int64_t first_k, n_units;     // blocks of Q, then those of K
  int32_t N;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

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

// Block means: one warp per block of rows of one head, or (SHARED: blocks of many
// rows) the four warps of a CTA.  D / 8 lanes across a row, eight loads of 16 bytes
// in flight per lane, no barrier between blocks.  Everything is fp32 pairs: fp64
// sums, at two lanes a clock per SM, took 320 us for a 480p layer, one CTA per block
// (whose loads wait out its barriers) 104 us.
template <int D, bool SHARED>
__global__ void __launch_bounds__(kPoolThreads, 8) pool_kernel(const __grid_constant__ PoolParams p) {
  constexpr int VR = D / 8, RPW = 32 / VR, WARPS = kPoolThreads / 32;   // RPW rows per warp load
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = SHARED ? blockIdx.x : blockIdx.x * static_cast<int64_t>(WARPS) + warp;
  if (unit >= p.n_units) return;
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
  // |mean|, over the largest component so that small means do not vanish squared
#pragma unroll
  for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
  m = fmaxf(m, FLT_MIN);
  const float over = 1.f / m;
  float n2 = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) n2 = fmaf(hi[c] * over, hi[c] * over, n2);
#pragma unroll
  for (int x = 16; x; x >>= 1) n2 += __shfl_xor_sync(0xFFFFFFFFu, n2, x);
  if (lane == 0) p.norm[w][u] = sqrtf(n2) * m * 1.0001f;     // NaN where a mean is
}

struct SelParams {
  const float *q_hi, *q_lo, *k_hi, *k_lo, *q_norm, *k_norm;
  float* scores;        // [CTA][kStrip][pitch] when the strip does not fit shared memory
  uint8_t* blocks;
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

// Two neighbouring values as two bf16 terms each: hi = bf16(x), lo = bf16(x - hi).
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x.x, x.y);
  lo = pack_bf16x2(x.x - bf16_lo(hi), x.y - bf16_hi(hi));
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

// The score in fp64 from the 48-bit means, by one warp (every lane gets it).
template <int D>
__device__ __forceinline__ double exact_score(const double (&q)[D / 32], const float* kh, const float* kl, int lane) {
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int c = i * 32 + lane;
    t = fma(q[i], static_cast<double>(__ldg(kh + c)) + static_cast<double>(__ldg(kl + c)), t);
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, m);
  return t;
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
__device__ __forceinline__ void select_row(const SelParams& p, int64_t bh, int i, float* row, float k_max, int lane) {
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
  const float q_norm = __ldg(p.q_norm + bh * p.nq + i);
  const float err2 = 2.f * (kScoreErr * (q_norm * k_max) + 4e-37f * (q_norm + k_max) + 1e-36f);
  bool finite = q_norm * k_max <= FLT_MAX && err2 <= FLT_MAX;
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
    float vmin = INFINITY, vmax = -INFINITY;
#pragma unroll
    for (int m = 0; m < chunks; ++m) {
      const float x = val(m);
      vmax = fmaxf(vmax, x);
      vmin = fminf(vmin, x == -INFINITY ? INFINITY : x);
    }
    const uint32_t kmin = __reduce_min_sync(0xFFFFFFFFu, key32(vmin));
    const uint32_t kmax = __reduce_max_sync(0xFFFFFFFFu, key32(vmax));
    // the want-th largest lies in [lo, hi]: c_lo = count(>= lo) >= want, c_hi =
    // count(> hi) < want.  Narrowed, by interpolating the counts and every third
    // time by halving, until the bracket is inside the fast bound or exactly `want`
    // are above (then it is the smallest of those).
    float lo = unkey32(kmin), hi = unkey32(kmax);
    float c_lo = static_cast<float>(others), c_hi = 0.f;
    for (int turn = 0; hi - lo > 0.25f * err2; ++turn) {
      const float f = turn % 3 == 2 ? 0.5f : (c_lo - static_cast<float>(want) + 0.5f) / (c_lo - c_hi);
      float mid = lo + f * (hi - lo);
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
  // lanes store the bytes of their own j, so a forced block's 1 comes after its 0
  auto keep_forced = [&]() {
    for (int j = lane; j < first; j += 32) out[j] = 1;
    for (int j = d_lo + ((lane - d_lo) & 31); j < d_hi; j += 32) out[j] = 1;
  };
  int n_sure = 0, n_near = 0;
#pragma unroll
  for (int m = 0; m < chunks; ++m) {
    n_sure += sure(val(m)) ? 1 : 0;
    n_near += near(m, val(m)) ? 1 : 0;
  }
  n_sure = __reduce_add_sync(0xFFFFFFFFu, n_sure);
  n_near = __reduce_add_sync(0xFFFFFFFFu, n_near);
  const int left = want - n_sure;               // of the near ones, 1 <= left <= n_near
  if (left == n_near) {
#pragma unroll
    for (int m = 0; m < chunks; ++m) {
      const int j = m * 32 + lane;
      if (j < p.nk) out[j] = sure(val(m)) || near(m, val(m)) ? 1 : 0;
    }
    keep_forced();
    return;
  }
  double q[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const int64_t o = (bh * p.nq + i) * D + c * 32 + lane;
    q[c] = static_cast<double>(__ldg(p.q_hi + o)) + static_cast<double>(__ldg(p.q_lo + o));
  }
  const float* kh = p.k_hi + bh * p.nk * D;
  const float* kl = p.k_lo + bh * p.nk * D;
  auto exact_key = [&](int j) -> uint64_t {
    return key64(exact_score<D>(q, kh + static_cast<int64_t>(j) * D, kl + static_cast<int64_t>(j) * D, lane));
  };
  if (n_near <= 32) {
    // lane c holds near block c (ascending j): its exact key, then its rank
    int my_j = -1, c = 0;
#pragma unroll
    for (int m = 0; m < chunks; ++m) {
      const int j = m * 32 + lane;
      const float x = val(m);
      const bool nr = near(m, x);
      if (j < p.nk && !nr) out[j] = sure(x) ? 1 : 0;
      uint32_t b = __ballot_sync(0xFFFFFFFFu, nr);
      while (b) {
        if (lane == c++) my_j = m * 32 + __ffs(b) - 1;
        b &= b - 1;
      }
    }
    keep_forced();
    uint64_t mine = 0;
#pragma unroll 2
    for (int o = 0; o < n_near; ++o) {
      const uint64_t key = exact_key(__shfl_sync(0xFFFFFFFFu, my_j, o));
      if (lane == o) mine = key;
    }
    int rank = 0;
    for (int o = 0; o < n_near; ++o) {
      const uint64_t other = __shfl_sync(0xFFFFFFFFu, mine, o);
      rank += (other > mine || (other == mine && o < lane)) ? 1 : 0;
    }
    if (my_j >= 0) out[my_j] = rank < left ? 1 : 0;
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
      while (b) {
        const int jj = j0 + __ffs(b) - 1;
        b &= b - 1;
        const uint64_t key = exact_key(jj);
        if (lane == 0) row[jj] = __uint_as_float(static_cast<uint32_t>(half ? key : key >> 32));
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

// One CTA: a strip of kStrip query blocks of one head.
template <int D, int KPL>
__global__ void __launch_bounds__(kSelThreads, KPL > 20 ? 2 : 3) select_kernel(const __grid_constant__ SelParams p) {
  extern __shared__ float smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t bh = blockIdx.x / p.strips;
  const int i0 = static_cast<int>(blockIdx.x - bh * p.strips) * kStrip;
  float* sc = p.scores ? p.scores + static_cast<int64_t>(blockIdx.x) * kStrip * p.pitch : smem;
  __shared__ float k_max_w[kSelThreads / 32];

  // the largest |km| of the head (NaN counts as infinite)
  float km = 0.f;
  for (int j = threadIdx.x; j < p.nk; j += kSelThreads) {
    const float x = __ldg(p.k_norm + bh * p.nk + j);
    km = x <= FLT_MAX ? fmaxf(km, x) : INFINITY;
    if (km > FLT_MAX) break;
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) km = fmaxf(km, __shfl_xor_sync(0xFFFFFFFFu, km, m));
  if (lane == 0) k_max_w[warp] = km;

  // ---- scores: every warp takes the strip's 16 query blocks, whose A fragments
  // (both bf16 terms) lie in shared memory in the order of their use, and every
  // eighth group of 8 key blocks
  {
    __shared__ uint4 frag[2][D / 16][32];
    const int g = lane >> 2, t = lane & 3;
    if (warp < D / 16) {
      uint32_t ah[4], al[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int r = i0 + g + ((f & 1) ? 8 : 0), c = warp * 16 + t * 2 + ((f & 2) ? 8 : 0);
        const float2 x = r < p.nq ? __ldg(reinterpret_cast<const float2*>(p.q_hi + (bh * p.nq + r) * D + c))
                                  : make_float2(0.f, 0.f);
        split2(x, ah[f], al[f]);
      }
      frag[0][warp][lane] = make_uint4(ah[0], ah[1], ah[2], ah[3]);
      frag[1][warp][lane] = make_uint4(al[0], al[1], al[2], al[3]);
    }
    __syncthreads();
    for (int j0 = warp * 8; j0 < p.nk; j0 += 8 * (kSelThreads / 32)) {
      const int j = j0 + g;
      const float* kr = p.k_hi + (bh * p.nk + (j < p.nk ? j : p.nk - 1)) * D + t * 2;
      float2 x[D / 8];
#pragma unroll
      for (int kk = 0; kk < D / 8; ++kk) x[kk] = __ldg(reinterpret_cast<const float2*>(kr + kk * 8));
      float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t bh0, bl0, bh1, bl1;
        split2(x[2 * kk], bh0, bl0);
        split2(x[2 * kk + 1], bh1, bl1);
        const uint4 ah = frag[0][kk][lane], al = frag[1][kk][lane];
        mma_16816(c0, ah, bh0, bh1);
        mma_16816(c1, ah, bl0, bl1);
        mma_16816(c1, al, bh0, bh1);
      }
      const int col = j0 + t * 2;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int cc = col + (e & 1), rr = g + ((e & 2) ? 8 : 0);
        if (cc < p.nk) sc[rr * p.pitch + cc] = c0[e] + c1[e];
      }
    }
  }
  __syncthreads();
  float k_max = k_max_w[0];
#pragma unroll
  for (int w = 1; w < kSelThreads / 32; ++w) k_max = fmaxf(k_max, k_max_w[w]);
  for (int rr = warp; rr < kStrip && i0 + rr < p.nq; rr += kSelThreads / 32)
    select_row<D, KPL>(p, bh, i0 + rr, sc + rr * p.pitch, k_max, lane);
}

// Scores per lane that the variants of select_kernel hold in registers.
constexpr int kRowRegs[] = {2, 8, 16, 20, 32};

struct Layout {
  int32_t nq, nk, strips, pitch;
  bool in_smem;
  size_t q_hi, q_lo, k_hi, k_lo, q_norm, k_norm, scores, total;
};

Layout layout_of(const tsr_select_desc& s) {
  Layout l;
  l.nq = (s.N + s.bq - 1) / s.bq;
  l.nk = (s.N + s.bk - 1) / s.bk;
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
  l.q_norm = take(BH * l.nq);
  l.k_norm = take(BH * l.nk);
  l.scores = take(l.in_smem ? 0 : BH * l.strips * kStrip * l.pitch);
  l.total = at;
  return l;
}

template <int D, int KPL>
tsr_status launch_strips(const SelParams& sp, unsigned ctas, size_t smem, cudaStream_t st) {
  auto kern = select_kernel<D, KPL>;
  int dev = 0;
  TSR_CUDA(cudaGetDevice(&dev));
  static bool attr_set[64] = {false};
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    TSR_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kStripBytes));
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  kern<<<ctas, kSelThreads, smem, st>>>(sp);
  TSR_CUDA(cudaGetLastError());
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
  pp.norm[0] = f(l.q_norm);
  pp.hi[1] = f(l.k_hi);
  pp.lo[1] = f(l.k_lo);
  pp.norm[1] = f(l.k_norm);
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
  sp.pitch = l.pitch;
  sp.keep = s.keep;
  sp.first = s.first;
  sp.diagonal = s.diagonal;
  const size_t smem = l.in_smem ? static_cast<size_t>(kStrip) * l.pitch * 4 : 0;
  // a CTA per block where a block holds more rows than a warp should read alone
  // (256 rows are 64 kB at d = 128), or where there are too few blocks to fill the GPU
  constexpr int kWarps = kPoolThreads / 32;
  if (std::max(s.bq, s.bk) > 256 || pp.n_units < 2048)
    pool_kernel<D, true><<<static_cast<unsigned>(pp.n_units), kPoolThreads, 0, st>>>(pp);
  else
    pool_kernel<D, false><<<static_cast<unsigned>((pp.n_units + kWarps - 1) / kWarps), kPoolThreads, 0, st>>>(pp);
  TSR_CUDA(cudaGetLastError());
  // scores per lane held in registers: as many as a row has, up to 32
  const unsigned ctas = static_cast<unsigned>(BH * l.strips);
  if (l.nk <= 64) return launch_strips<D, 2>(sp, ctas, smem, st);
  if (l.nk <= 256) return launch_strips<D, 8>(sp, ctas, smem, st);
  if (l.nk <= 512) return launch_strips<D, 16>(sp, ctas, smem, st);
  if (l.nk <= 640) return launch_strips<D, 20>(sp, ctas, smem, st);
  if (l.nk <= 1024) return launch_strips<D, 32>(sp, ctas, smem, st);
  return launch_strips<D, 0>(sp, ctas, smem, st);
}

}  // namespace

size_t select_workspace(const tsr_select_desc& s) { return layout_of(s).total; }

// The arguments have been checked (api_ops.cu).
tsr_status launch_select(const tsr_select_desc& s, const void* q, const void* k, uint8_t* blocks, void* ws,
                         cudaStream_t st) {
  const Layout l = layout_of(s);
  const int64_t BH = static_cast<int64_t>(s.B) * s.H;
  if (BH * (static_cast<int64_t>(l.nq) + l.nk) >= (int64_t{1} << 31))
    return fail(TSR_ERR_UNSUPPORTED, "more than 2^31 blocks");
  if (s.d == 64) return launch<64>(s, l, q, k, blocks, static_cast<uint8_t*>(ws), st);
  return launch<128>(s, l, q, k, blocks, static_cast<uint8_t*>(ws), st);
}

}  // namespace tsr
