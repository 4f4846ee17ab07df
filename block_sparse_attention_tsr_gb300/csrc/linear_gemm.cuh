// linear_gemm.cuh -- the matrix products of a linear layer on tcgen05 tensor cores:
//     D[r][c] = sum_k A(r, k) B(c, k)
// with A and B 16-bit (bf16 or fp16), D in fp32 in TMEM and an epilogue on its way out.
//
//   forward   A = x (rows: tokens),           B = weight (rows: out features), k: in features
//   dx        A = dz (rows: tokens),          B = weight^T (rows: in features), k: out features
//   dweight   A = dz^T (rows: out features),  B = x^T (rows: in features),     k: tokens
//
// An operand whose k is contiguous in memory is K-major, one whose rows are contiguous
// MN-major; the tensor cores take both, so nothing is transposed.  Every tensor is seen by
// TMA as {channel, token, head, batch} with free strides: the attention's head-major
// [B][H][N][d] is read and written in place.
//
// Bound: the tensor pipe for many tokens.  Two CTAs (a pair, cta_group::2) compute a tile
// of 256 rows x BN columns; each loads half of A's and half of B's rows, so a step of 64 k
// is 32 KB per SM for 512 clocks of MMAs at BN = 256, 64 bytes a clock, about what an SM
// takes from L2 (a tile of 128 x 256 of one CTA would need 96).  The accumulator has two
// buffers in TMEM: the epilogue of a tile runs beside the MMAs of the next.
//
// Persistent: a CTA pair takes every n-th work unit, whole tiles first.  The tiles that
// would make up a last, part-filled wave are cut along k instead (and all tiles, where
// there are fewer than pairs): their units store fp32 parts that linear_finish_kernel adds
// in their order.
// Warps: TMA producer, MMA issuer (of the pair's first CTA), 8 epilogue warps.  Every wait
// is bounded: on expiry the error word is set and the kernel winds down; what has not been
// computed is not stored.
//
// For few tokens the weight's bytes bound it (linear_few_kernel): the features lie on the
// 128 rows and the tokens on 32 or 128 columns, and a cluster of up to 8 CTAs shares a
// tile's k; each leaves its sums in shared memory and adds up its share of the tile from
// all of them.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace tsr {

namespace linear {

constexpr int kEpiWarps = 8, kThreads = (kEpiWarps + 2) * 32;
constexpr int kMostCtas = 256;         // of a product by pairs
constexpr int BK = 64;                 // k per step: 128 bytes, the swizzle's row

// A tensor's addressing: element strides of batch, head and token; channels contiguous.
struct View {
  int64_t sb, sh, sn;
  int32_t dim;                         // channels per head
};

// Quotients of n < 2^31 by a number that the host knows, by its reciprocal: with 2^(l-1) < d
// <= 2^l and m = floor(2^(31+l) / d) + 1, n m / 2^(31+l) exceeds n / d by less than 1 / d
// (division by invariant integers, Granlund and Montgomery, 1994).  A division costs some 200
// clocks; a tile of few steps waited for five, in every warp.
struct Div {
  uint32_t d, mul, shift;
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return d == 1 ? n : __umulhi(n, mul) >> shift; }
};
inline Div div_by(uint32_t d) {
  uint32_t l = 0;
  while (1ull << l < d) ++l;
  return {d, d == 1 ? 0u : static_cast<uint32_t>((1ull << (31 + l)) / d + 1), d == 1 ? 0u : l - 1};
}

// What happens to a value of D on its way out.
struct Epilogue {
  const void *bias, *res;              // null: none
  void *out, *pre;                     // pre: the value before the activation, null: not kept
  View vout, vres, vpre;
  int32_t act, f16;
};

struct GemmParams {
  CUtensorMap ta, tb;                  // few tokens: the weight, and the tokens
  // out, pre and residual as {channel, token, head, batch} in boxes of 32 tokens x 64 channels
  // (32 where pre is kept), and the parts, fp32, as {column, row, tile, part} in boxes of 32 x 32
  CUtensorMap tout, tpre, tres, tpart;
  Epilogue epi;
  float* part;                         // [splits][tiles - whole][256][BN]
  uint8_t* gave_up;                    // [kMostCtas] behind the parts: 1 of a CTA that gave up
  uint32_t ctas;
  uint32_t whole, units;               // tiles that are not cut along k: the first ones; all work units
  int32_t n_rows;                      // rows per batch (tokens, or features)
  int32_t cols;
  int32_t row_tiles, col_tiles;        // row tiles of all batches
  Div by_batch;                        // row tiles per batch
  Div by_group, by_cut;                // tiles of a group of row tiles (tile_of); tiles that are cut
  uint32_t group_log2;                 // row tiles of a group
  int32_t splits, k_steps;             // k steps of a whole product
  uint32_t k_each, k_more;             // k steps of a part; parts that have one more
  int32_t k_steps_per_batch;           // dweight: steps of one batch's tokens
  Div a_dim, b_dim, out_dim;           // channels per head of A's, B's and out's tensors
  uint32_t idesc;
  int32_t late;                        // what is before on the stream is not an input: waited for at the end
  int32_t pass_on;                     // late, or a late product behind this one reads inputs that this one was shown
  int32_t stall;                       // test only: the issuer waits for ever after its first step
  uint64_t timeout_ns;                 // bound of every wait
};

// Waits that gave up (tsr_linear_device_status): of the device, not of a call.
static __device__ uint32_t g_err;

// ------------------------------------------------------------- the epilogue
// Eight 16-bit values as four pairs, and back.
template <bool F16>
__device__ __forceinline__ void unpack8(uint4 w, F2 (&v)[4]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F16) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
      v[i] = pack2(p.x, p.y);
    } else {
      v[i] = pack2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xFFFF0000u));
    }
  }
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const F2 (&v)[4]) {
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2(v[i]);
    if constexpr (F16) {
      const __half2 h = __floats2half2_rn(p.x, p.y);
      x[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      x[i] = pack_bf16x2(p.x, p.y);
    }
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu0 = 2.f * 0.7978845608028654f, kGelu1 = kGelu0 * 0.044715f;   // 2 sqrt(2 / pi)

__device__ __forceinline__ F2 rcp2(F2 v) {
  const float2 x = unpack2(v);
  float2 y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
  return pack2(y.x, y.y);
}
__device__ __forceinline__ F2 exp2_2(F2 v) {
  const float2 x = unpack2(v);
  return pack2(ex2_approx(x.x), ex2_approx(x.y));
}
// 1 / (1 + 2^x).  The exponential is within about |x| 2^-23 of its value, the reciprocal
// within 2^-23: far inside a 16-bit rounding.
__device__ __forceinline__ F2 logistic_neg(F2 x) { return rcp2(add2(both(1.f), exp2_2(x))); }
// The normal distribution function Phi(z) = erfc(-z / sqrt 2) / 2: with x = |z| / sqrt 2 and
// t = 1 / (1 + x / 2), erfc(x) = t Q(t) e^(-x^2), Q a polynomial of erfc(x) e^(x^2) / t with
// the least relative error (7e-7) for t in [0.2, 1].  Within 2e-6 of itself for z > -5, 1e-5
// for z > -11: no cancellation for negative z.  bell: e^(-z^2 / 2), which the slope takes too
// (with an exponential of its own the column sums of 32,760 x 8,192 took 290 us, not 267).
__device__ __forceinline__ F2 bell(F2 z) { return exp2_2(mul2(mul2(both(-0.5f * kLog2e), z), z)); }
__device__ __forceinline__ F2 normal_cdf(F2 z, F2 bell) {
  const F2 x = mul2(both(0.70710678118654752f), z & 0x7FFFFFFF7FFFFFFFull);
  const F2 t = rcp2(fma2(both(0.5f), x, both(1.f)));
  F2 q = both(0.0921261385f);
  q = fma2(q, t, both(-0.370672017f));
  q = fma2(q, t, both(0.408959091f));
  q = fma2(q, t, both(0.0237065479f));
  q = fma2(q, t, both(0.286929965f));
  q = fma2(q, t, both(0.276539981f));
  q = fma2(q, t, both(0.282409608f));
  const F2 tail = mul2(mul2(mul2(both(0.5f), t), q), bell);
  const float2 s = unpack2(z), low = unpack2(tail), high = unpack2(fma2(tail, both(-1.f), both(1.f)));
  return pack2(s.x < 0.f ? low.x : high.x, s.y < 0.f ? low.y : high.y);
}
// The tanh form is z times the logistic function of 2u, u = sqrt(2 / pi) (z + 0.044715
// z^3): no cancellation there either.
template <int ACT>
__device__ __forceinline__ F2 activate(F2 z) {
  if constexpr (ACT == TSR_ACT_GELU_TANH)
    return mul2(z, logistic_neg(mul2(z, fma2(both(-kLog2e * kGelu1), mul2(z, z), both(-kLog2e * kGelu0)))));
  if constexpr (ACT == TSR_ACT_SILU) return mul2(z, logistic_neg(mul2(both(-kLog2e), z)));
  if constexpr (ACT == TSR_ACT_GELU) return mul2(z, normal_cdf(z, bell(z)));
  return z;
}
// The activation's derivative.  Far out the logistic function is 0 or 1 in fp32 and s (1 - s)
// exactly 0, and so is its product with any finite z (z^2 is cut off where it no longer
// matters); at an infinite z the derivative is NaN, as the formula's inf * 0.
template <int ACT>
__device__ __forceinline__ F2 slope(F2 z) {
  const F2 one = both(1.f), minus = both(-1.f);
  if constexpr (ACT == TSR_ACT_SILU) {
    const F2 s = logistic_neg(mul2(both(-kLog2e), z));
    return mul2(s, fma2(z, fma2(s, minus, one), one));
  } else if constexpr (ACT == TSR_ACT_GELU_TANH) {
    const float2 zz = unpack2(mul2(z, z));
    const F2 q = pack2(fminf(zz.x, 900.f), fminf(zz.y, 900.f));
    const F2 s = logistic_neg(mul2(z, fma2(both(-kLog2e * kGelu1), q, both(-kLog2e * kGelu0))));
    return fma2(mul2(z, mul2(s, fma2(s, minus, one))), fma2(both(3.f * kGelu1), q, both(kGelu0)), s);
  } else if constexpr (ACT == TSR_ACT_GELU) {
    const F2 e = bell(z);
    return fma2(mul2(z, both(0.3989422804014327f)), e, normal_cdf(z, e));
  }
  return one;
}
// f<F16, ACT>() for the call's type and activation: the elements' code has no branches on them.
template <typename F>
__device__ __forceinline__ void by_kind(int f16, int act, F&& f) {
  using std::integral_constant;
  switch (act * 2 + f16) {
    case 0: return f(integral_constant<bool, false>(), integral_constant<int, 0>());
    case 1: return f(integral_constant<bool, true>(), integral_constant<int, 0>());
    case 2: return f(integral_constant<bool, false>(), integral_constant<int, 1>());
    case 3: return f(integral_constant<bool, true>(), integral_constant<int, 1>());
    case 4: return f(integral_constant<bool, false>(), integral_constant<int, 2>());
    case 5: return f(integral_constant<bool, true>(), integral_constant<int, 2>());
    case 6: return f(integral_constant<bool, false>(), integral_constant<int, 3>());
    default: return f(integral_constant<bool, true>(), integral_constant<int, 3>());
  }
}

__device__ __forceinline__ int64_t at(const View& v, int64_t b, int64_t n, int32_t f) {
  const int32_t h = f / v.dim;
  return b * v.sb + h * v.sh + n * v.sn + (f - h * v.dim);
}

// Eight neighbouring features [f, f + 8) of token (b, n), from D's values to the output.
template <bool F16, int ACT>
__device__ __forceinline__ void finish8(const Epilogue& e, F2 (&v)[4], int64_t b, int64_t n, int32_t f) {
  F2 t[4];
  if (e.bias) {
    unpack8<F16>(static_cast<const uint4*>(e.bias)[f / 8], t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = add2(v[i], t[i]);
  }
  if (e.pre) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(e.pre) + at(e.vpre, b, n, f)) = pack8<F16>(v);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = activate<ACT>(v[i]);
  if (e.res) {
    unpack8<F16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(e.res) + at(e.vres, b, n, f)), t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = add2(v[i], t[i]);
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(e.out) + at(e.vout, b, n, f)) = pack8<F16>(v);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// ---------------------------------------------------------------- the kernel
template <int BN>
struct Cfg {
  static constexpr int TM = 256;                          // rows of a tile, half of them in each CTA
  static constexpr int A_BYTES = 128 * BK * 2, B_ROWS = BN / 2, B_BYTES = B_ROWS * BK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  // what leaves through shared memory: for each epilogue warp two pieces of 32 rows x 128
  // bytes (64 columns, of parts 32)
  static constexpr int PIECE = 32 * 128, OUT_BYTES = kEpiWarps * 2 * PIECE;
  static constexpr int FIT = (226 * 1024 - OUT_BYTES) / STAGE, STAGES = FIT < 8 ? FIT : 8;
  static constexpr int OUT = STAGES * STAGE, CTRL = OUT + OUT_BYTES, SMEM = CTRL + 512;
  static constexpr int TMEM = 2 * BN;                     // two accumulators
  static_assert(SMEM > 114 * 1024, "one CTA per SM");
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(TMEM <= 512 && (TMEM & (TMEM - 1)) == 0, "TMEM");
};

struct alignas(8) Ctrl {
  uint64_t full[8], empty[8], acc_full[2], acc_empty[2], final_bar;
  uint64_t never;                      // never signalled (stall test)
  uint64_t res_full[kEpiWarps][2];     // the residual's piece has landed
  uint32_t tmem_base;
  int32_t abort_flag;
  uint32_t gave_up;                    // few tokens: a CTA of the cluster has given up
};
static_assert(sizeof(Ctrl) <= 512, "Ctrl");

// Row and column of tile t: a group of row tiles at a time, their columns one after another,
// so that the CTAs that run together share rows and columns in L2.
__device__ __forceinline__ int2 tile_of(const GemmParams& p, uint32_t t) {
  const uint32_t g = p.by_group(t), in = t - g * p.by_group.d, row = g << p.group_log2, rows = p.row_tiles - row;
  if (rows >> p.group_log2) return make_int2(row + (in & ((1u << p.group_log2) - 1)), in >> p.group_log2);
  const uint32_t col = in / rows;
  return make_int2(row + (in - col * rows), col);
}
// A work unit: a tile and its part of k.
struct Unit {
  int32_t row_tile, col_tile, cut, split, k0, k1;         // cut: the tile's number among the cut ones, or -1
};
__device__ __forceinline__ void steps_of(const GemmParams& p, uint32_t u, Unit& w) {
  w.cut = -1;
  w.split = 0;
  w.k0 = 0;
  w.k1 = p.k_steps;
  if (u >= p.whole) {
    const uint32_t split = p.by_cut(u - p.whole);
    w.split = split;
    w.cut = u - p.whole - split * p.by_cut.d;
    w.k0 = split * p.k_each + min(split, p.k_more);
    w.k1 = w.k0 + p.k_each + (split < p.k_more);
  }
}
__device__ __forceinline__ Unit unit_of(const GemmParams& p, uint32_t u) {
  Unit w;
  steps_of(p, u, w);
  const int2 rc = tile_of(p, w.cut < 0 ? u : p.whole + w.cut);
  w.row_tile = rc.x;
  w.col_tile = rc.y;
  return w;
}

// Where an operand's copies start, step by step: 64 channels of `rows` rows (K-major, one
// box), or G groups of 64 channels of 64 tokens or weight rows (MN-major).
template <bool MN, int G>
struct Walk {
  int32_t dim, c[MN ? G : 1], h[MN ? G : 1], n, b, chunk, chunks;
  // f0: first row (K-major) or channel (MN-major); chunks: k steps of a batch's tokens, 0:
  // k has no batches
  __device__ __forceinline__ Walk(const Div& by, int32_t f0, int32_t k0, int32_t chunks_, int32_t batch)
      : dim(by.d), chunks(chunks_) {
    if constexpr (MN) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        h[g] = by(f0 + 64 * g);
        c[g] = f0 + 64 * g - h[g] * dim;
      }
      b = chunks && k0 >= chunks ? k0 / chunks : 0;
      chunk = k0 - b * chunks;
      n = chunk * BK;
    } else {
      h[0] = by(k0 * BK);
      c[0] = k0 * BK - h[0] * dim;
      n = f0;
      b = batch;
      chunk = 0;
    }
  }
  template <int CG>
  __device__ __forceinline__ void load(uint32_t elect, uint32_t dst, const CUtensorMap* m, uint32_t bar) const {
#pragma unroll
    for (int g = 0; g < (MN ? G : 1); ++g) {
      if constexpr (CG == 2) tma_load_4d_pair(elect, dst + g * 64 * 128, m, bar, c[g], n, h[g], b);
      else tma_load_4d(elect, dst + g * 64 * 128, m, bar, c[g], n, h[g], b);
    }
  }
  __device__ __forceinline__ void advance() {
    if constexpr (MN) {
      n += BK;
      if (chunks && ++chunk == chunks) {
        chunk = 0;
        n = 0;
        ++b;
      }
    } else {
      c[0] += BK;
      if (c[0] >= dim) {
        c[0] -= dim;
        ++h[0];
      }
    }
  }
};

template <int BN, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kThreads, 1) linear_gemm_kernel(const __grid_constant__ GemmParams p) {
  using C = Cfg<BN>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  Ctrl& ctrl = *reinterpret_cast<Ctrl*>(smem + C::CTRL);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  volatile int32_t* abort_flag = &ctrl.abort_flag;
  if (threadIdx.x == 0) {
    if (base & 1023u) atomicOr(&g_err, DEV_ERR_INTERNAL);   // swizzled tiles need 1024-byte alignment
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&ctrl.full[i]), 1);
      mbar_init(smem_u32(&ctrl.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctrl.acc_full[i]), 1);
      mbar_init(smem_u32(&ctrl.acc_empty[i]), kEpiWarps * 2);
    }
    mbar_init(smem_u32(&ctrl.final_bar), 1);
    mbar_init(smem_u32(&ctrl.never), 1);
    for (int i = 0; i < 2 * kEpiWarps; ++i) mbar_init(smem_u32(&ctrl.res_full[0][0] + i), 1);
    ctrl.abort_flag = (base & 1023u) ? 1 : 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane < 2) tma_prefetch_desc(lane ? &p.tb : &p.ta);
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&ctrl.tmem_base), C::TMEM);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, ctrl.tmem_base, 0);
  // what comes before may still run while this CTA sets itself up; where it is no input, till
  // this kernel's end (so that no kernel behind this one starts before it has ended)
  if (!p.late) grid_wait();
  if (p.pass_on) grid_pass_on();
  grid_launch_dependents();
  const uint32_t units = p.units, first = blockIdx.x / 2, stride = gridDim.x / 2;
  // each CTA clears its own, the first those of none (a word of each, stored at the end: 22.6 ->
  // 23.6 us for 2,593 x 1176 -> 1712)
  if (p.gave_up && warp == 2) {
    if (lane == 0) p.gave_up[blockIdx.x] = 0;
    if (blockIdx.x == 0)
      for (uint32_t k = gridDim.x + lane; k < kMostCtas; k += 32) p.gave_up[k] = 0;
  }

  if (warp == 0) {
    // The whole warp runs the loop and one lane acts, so that the copies' addresses and
    // coordinates stay in uniform registers, and the coordinates advance by additions: a
    // step's copies were issued in 360 ns by a single lane that divided for them, while
    // the products of a step take 267 (462 us without copies for 1,728 steps).
    const uint32_t elect = elect_lane();
    int64_t issued = 0;                                   // steps
    int st = 0;
    uint32_t parity = 1u;                                 // of the wait for an empty stage
    bool ok = true;
    for (uint32_t u = first; ok && u < units; u += stride) {
      const Unit w = unit_of(p, u);
      // token rows: tiles of each batch by themselves (dweight: rows are features, k tokens)
      const int32_t b = A_MN ? 0 : p.by_batch(w.row_tile);
      const int32_t row0 = (w.row_tile - b * static_cast<int32_t>(p.by_batch.d)) * C::TM + rank * 128;
      const int32_t col0 = w.col_tile * BN + rank * C::B_ROWS;
      Walk<A_MN, 2> ca(p.a_dim, row0, w.k0, A_MN ? p.k_steps_per_batch : 0, b);
      Walk<B_MN, C::B_ROWS / 64> cb(p.b_dim, col0, w.k0, A_MN ? p.k_steps_per_batch : 0, 0);
      for (int32_t s = w.k0; s < w.k1; ++s) {
        if (!mbar_wait_warp(smem_u32(&ctrl.empty[st]), parity, abort_flag, &g_err, p.timeout_ns)) { ok = false; break; }
        const uint32_t a = base + st * C::STAGE;
        if (rank == 0) mbar_arrive_expect_tx(elect, smem_u32(&ctrl.full[st]), 2 * C::STAGE);
        const uint32_t bar = cluster_addr(smem_u32(&ctrl.full[st]), 0);
        ca.template load<2>(elect, a, &p.ta, bar);
        cb.template load<2>(elect, a + C::A_BYTES, &p.tb, bar);
        ca.advance();
        cb.advance();
        ++issued;
        if (++st == C::STAGES) {
          st = 0;
          parity ^= 1u;
        }
      }
    }
    // the issuer's arrivals on this CTA's empty barriers come before the CTA ends (those of the
    // last steps nobody else waits for; the peer's CTA may be through with its part before)
    for (int64_t k = issued > C::STAGES ? issued - C::STAGES : 0; ok && k < issued; ++k)
      ok = mbar_wait_warp(smem_u32(&ctrl.empty[k % C::STAGES]), static_cast<uint32_t>(k / C::STAGES) & 1u, abort_flag,
                          &g_err, p.timeout_ns);
    if (rank == 0 && !ok) {
      // given up: every copy lands before the CTA ends
      volatile int32_t no = 0;
      for (int64_t k = issued > C::STAGES ? issued - C::STAGES : 0; k < issued; ++k)
        mbar_wait_warp(smem_u32(&ctrl.full[k % C::STAGES]), static_cast<uint32_t>(k / C::STAGES) & 1u, &no, &g_err,
                       p.timeout_ns);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t elect = elect_lane();
      int st = 0;
      uint32_t parity = 0u;
      int32_t tile = 0;
      bool ok = true;
      for (uint32_t u = first; ok && u < units; u += stride, ++tile) {
        Unit w;
        steps_of(p, u, w);
        const int buf = tile & 1;
        if (!mbar_wait_warp(smem_u32(&ctrl.acc_empty[buf]), ((tile >> 1) & 1) ^ 1, abort_flag, &g_err, p.timeout_ns)) break;
        tc_fence_after();
        const uint32_t acc = tmem + buf * BN;
        for (int32_t s = w.k0; s < w.k1; ++s) {
          if (!mbar_wait_warp(smem_u32(&ctrl.full[st]), parity, abort_flag, &g_err, p.timeout_ns)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a = base + st * C::STAGE, b = a + C::A_BYTES;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k) {
            const uint64_t da = A_MN ? sdesc_sw128(a + k * 2048, 64 * 128, 1024) : sdesc_sw128(a + k * 32, 16, 1024);
            const uint64_t db = B_MN ? sdesc_sw128(b + k * 2048, 64 * 128, 1024) : sdesc_sw128(b + k * 32, 16, 1024);
            const uint32_t more = s > w.k0 || k > 0;
            mma_f16_ss_pair(elect, acc, da, db, p.idesc, more);
          }
          mma_commit_pair(elect, smem_u32(&ctrl.empty[st]));
          if (p.stall && !mbar_wait_warp(smem_u32(&ctrl.never), 0, abort_flag, &g_err, p.timeout_ns)) { ok = false; break; }
          if (++st == C::STAGES) {
            st = 0;
            parity ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit_pair(elect, smem_u32(&ctrl.acc_full[buf]));
      }
      if (*abort_flag) {
        // the products in flight end before TMEM is freed
        mma_commit_pair(elect, smem_u32(&ctrl.final_bar));
        volatile int32_t no = 0;
        mbar_wait_warp(smem_u32(&ctrl.final_bar), 0, &no, &g_err, p.timeout_ns);
      }
    }
  } else {
    const int ew = warp - 2, quarter = warp & 3, half = ew >> 2;   // TMEM lanes 32 * quarter of this warp
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t elect = elect_lane();
    uint32_t res_phase = 0u, res_issued = 0u;              // of the residual's pieces
    uint32_t turn = 0u;                                    // pieces take turns, from tile to tile
    int32_t tile = 0;
    for (uint32_t u = first; u < units; u += stride, ++tile) {
      const Unit w = unit_of(p, u);
      const int buf = tile & 1;
      const uint32_t acc = tmem + lanes + buf * BN;
      if (w.cut >= 0) {
        if (!mbar_wait_warp(smem_u32(&ctrl.acc_full[buf]), (tile >> 1) & 1, abort_flag, &g_err, p.timeout_ns)) break;
        tc_fence_after();
      }
      {
        const int32_t b = A_MN ? 0 : p.by_batch(w.row_tile);
        const int32_t n0 = (w.row_tile - b * static_cast<int32_t>(p.by_batch.d)) * C::TM + rank * 128 + quarter * 32;
        constexpr int W = BN / 2;                                   // columns of this warp
        const int32_t f0 = w.col_tile * BN + half * W;
        const bool inside = n0 < p.n_rows;
        const uint32_t pieces = base + C::OUT + ew * 2 * C::PIECE;
        if (w.cut >= 0) {
#pragma unroll 1
          for (int c = 0; c < W; c += 64) {
            if (f0 + c >= p.cols || !inside) break;
            uint32_t v[2][32];
            tmem_ld32(acc + half * W + c, v[0]);
            tmem_ld32(acc + half * W + c + 32, v[1]);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (f0 + c + j * 32 >= p.cols) break;
              const uint32_t q = pieces + (turn++ & 1u) * C::PIECE;
              bulk_wait_read<1>();                                  // the piece before the last has left
              __syncwarp();
              // a lane's row of 128 bytes, 16 each, swizzled as TMA reads it
#pragma unroll
              for (int i = 0; i < 8; ++i)
                sts128(q + lane * 128 + ((i ^ (lane & 7)) << 4),
                       make_uint4(v[j][4 * i], v[j][4 * i + 1], v[j][4 * i + 2], v[j][4 * i + 3]));
              fence_proxy_async_smem();
              __syncwarp();
              tma_store_4d(elect, &p.tpart, q, half * W + c + j * 32, rank * 128 + quarter * 32, w.cut, w.split);
              bulk_commit(elect);
            }
          }
        } else {
          const bool pre = p.epi.pre != nullptr, res = p.epi.res != nullptr, plain = !pre && !res && !p.epi.bias;
          const int dim = p.out_dim.d;
          int32_t h = p.out_dim(f0), ch = f0 - h * dim;
          // a step takes a piece: 64 columns, or with pre 32, pre's in its first half and out's
          // in the second; a residual lands where out's will be
          const int width = pre ? 32 : 64, half_piece = pre ? C::PIECE / 2 : 0;
          const int steps = !inside || f0 >= p.cols ? 0 : (min(W, p.cols - f0) + width - 1) / width;
          auto load_res = [&](int s) {
            const uint32_t k = (turn + s) & 1u, bar = smem_u32(&ctrl.res_full[ew][k]);
            const int32_t f = f0 + s * width, h = p.out_dim(f);
            mbar_arrive_expect_tx(elect, bar, width * 64);
            tma_load_4d(elect, pieces + k * C::PIECE + half_piece, &p.tres, bar, f - h * dim, n0, h, b);
            res_issued |= 1u << k;
          };
          if (res) {
            bulk_wait_read<0>();
            __syncwarp();
            for (int s = 0; s < min(steps, 2); ++s) load_res(s);
          }
          if (!mbar_wait_warp(smem_u32(&ctrl.acc_full[buf]), (tile >> 1) & 1, abort_flag, &g_err, p.timeout_ns)) break;
          tc_fence_after();
          bool ok = true;
          uint32_t v[2][32];
          auto columns = [&](int s) {
            if (s < steps) {
              tmem_ld32(acc + half * W + s * width, v[0]);
              if (!pre) tmem_ld32(acc + half * W + s * width + 32, v[1]);
            }
          };
          columns(0);
#pragma unroll 1
          for (int s = 0; s < steps; ++s) {
            const int n = pre ? 1 : 2;                              // 32 columns each
            const uint32_t k = (turn + s) & 1u;
            uint4 bias[2][4] = {};
            if (p.epi.bias) {
#pragma unroll
              for (int g = 0; g < 8; ++g) {
                const int32_t f = f0 + s * width + g * 8;
                if (f < p.cols && g < 4 * n) bias[g >> 2][g & 3] = static_cast<const uint4*>(p.epi.bias)[f / 8];
              }
            }
            if (res) {
              if (s >= 2) {
                bulk_wait_read<0>();
                __syncwarp();
                load_res(s);
              }
              ok = mbar_wait_warp(smem_u32(&ctrl.res_full[ew][k]), (res_phase >> k) & 1, abort_flag, &g_err, p.timeout_ns);
              if (!ok) break;
              res_phase ^= 1u << k;
              res_issued &= ~(1u << k);
            } else {
              bulk_wait_read<1>();                                  // all but the last step's piece have left
              __syncwarp();
            }
            tc_wait_ld();
            // a lane's row of the piece, 16 bytes each, swizzled as TMA reads it (rows of 128
            // bytes, or of 64)
            const uint32_t q_pre = pieces + k * C::PIECE, q = q_pre + half_piece;
            const uint32_t row = lane * (pre ? 64 : 128), turned = pre ? (lane >> 1) & 3 : lane & 7;
            auto pair = [&](int j, int c) { return pack2(__uint_as_float(v[j][c]), __uint_as_float(v[j][c + 1])); };
            by_kind(p.epi.f16, p.epi.act, [&](auto f16, auto act) {
              if constexpr (act.value == TSR_ACT_NONE) {
                if (plain) {
#pragma unroll
                  for (int g = 0; g < 8; ++g) {
                    F2 x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = pair(g >> 2, 8 * (g & 3) + 2 * i);
                    sts128(q + row + ((g ^ turned) << 4), pack8<f16.value>(x));
                  }
                  return;
                }
              }
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                if (j < n) {
#pragma unroll
                  for (int g = 0; g < 4; ++g) {
                    F2 x[4], t[4];
                    const uint32_t o = row + (((j * 4 + g) ^ turned) << 4);
                    unpack8<f16.value>(bias[j][g], t);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = add2(pair(j, 8 * g + 2 * i), t[i]);
                    if (pre) sts128(q_pre + o, pack8<f16.value>(x));
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = activate<act.value>(x[i]);
                    if (res) {
                      unpack8<f16.value>(lds128(q + o), t);
#pragma unroll
                      for (int i = 0; i < 4; ++i) x[i] = add2(x[i], t[i]);
                    }
                    sts128(q + o, pack8<f16.value>(x));
                  }
                }
              }
            });
            columns(s + 1);                                         // on their way while these leave
            fence_proxy_async_smem();
            __syncwarp();
            if (pre) tma_store_4d(elect, &p.tpre, q_pre, ch, n0, h, b);
            tma_store_4d(elect, &p.tout, q, ch, n0, h, b);
            bulk_commit(elect);
            ch += width;
            if (ch >= dim) {
              ch = 0;
              ++h;
            }
          }
          if (!ok) {
            tc_wait_ld();
            break;
          }
          turn += steps;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        const uint32_t bar = smem_u32(&ctrl.acc_empty[buf]);
        mbar_arrive_cluster(cluster_addr(bar, 0));
      }
    }
    bulk_wait_read<0>();                   // shared memory has been read before the CTA ends
    if (*abort_flag) {
      // a residual's piece in flight lands before the CTA ends
      volatile int32_t no = 0;
      for (int k = 0; k < 2; ++k)
        if ((res_issued >> k) & 1) mbar_wait_warp(smem_u32(&ctrl.res_full[ew][k]), (res_phase >> k) & 1, &no, &g_err, p.timeout_ns);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (p.gave_up && *abort_flag && threadIdx.x == 0) p.gave_up[blockIdx.x] = 1;
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::TMEM);
  }
  if (p.late) grid_wait();
}

// ---------------------------------------------------------------- few tokens
template <int BN>
struct FewCfg {
  static constexpr int A_BYTES = 128 * BK * 2, STAGE = A_BYTES + BN * BK * 2;
  static constexpr int RED = BN * 128 * 4;                // the tile's sums, [token][feature]
  // 32 tokens: two CTAs per SM, so that k can be cut further (8 x 8192 -> 2048 in
  // eight parts, the weight in L2: 8.7 -> 7.5 us)
  static constexpr int CTAS = BN == 32 ? 2 : 1;
  static constexpr int FIT = (226 * 1024 / CTAS - RED - 2048) / STAGE, STAGES = FIT < 8 ? FIT : 8;
  static constexpr int SUMS = STAGES * STAGE, CTRL = SUMS + RED, SMEM = CTRL + 512;
  static_assert((SMEM + 1024) * CTAS <= 228 * 1024, "CTAs per SM");
};

// D^T: 128 features on the rows, BN tokens on the columns; the cluster's CTAs take p.splits
// parts of k.  W_MN: the weight's rows are k (dx).
template <int BN, bool W_MN>
__global__ void __launch_bounds__(kThreads, FewCfg<BN>::CTAS) linear_few_kernel(const __grid_constant__ GemmParams p) {
  using C = FewCfg<BN>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  Ctrl& ctrl = *reinterpret_cast<Ctrl*>(smem + C::CTRL);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int32_t rank = static_cast<int32_t>(cluster_rank());
  volatile int32_t* abort_flag = &ctrl.abort_flag;
  if (threadIdx.x == 0) {
    if (base & 1023u) atomicOr(&g_err, DEV_ERR_INTERNAL);
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&ctrl.full[i]), 1);
      mbar_init(smem_u32(&ctrl.empty[i]), 1);
    }
    mbar_init(smem_u32(&ctrl.acc_full[0]), 1);
    mbar_init(smem_u32(&ctrl.final_bar), 1);
    mbar_init(smem_u32(&ctrl.never), 1);
    ctrl.abort_flag = (base & 1023u) ? 1 : 0;
    ctrl.gave_up = 0u;
    fence_mbar_init();
  }
  if (warp == 0 && lane < 2) tma_prefetch_desc(lane ? &p.tb : &p.ta);
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctrl.tmem_base), BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();                        // this CTA's control block is set up (waited for at the end)
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, ctrl.tmem_base, 0);
  if (!p.late) grid_wait();
  if (p.pass_on) grid_pass_on();
  grid_launch_dependents();
  const int32_t tile = static_cast<int32_t>(blockIdx.x) / p.splits;
  const int32_t f_tile = tile % p.row_tiles, t_tile = tile / p.row_tiles;
  const int32_t b = p.by_batch(t_tile), n0 = (t_tile - b * static_cast<int32_t>(p.by_batch.d)) * BN;
  const int32_t k0 = static_cast<int32_t>(static_cast<int64_t>(p.k_steps) * rank / p.splits);
  const int32_t k1 = static_cast<int32_t>(static_cast<int64_t>(p.k_steps) * (rank + 1) / p.splits);
  if (warp == 0) {
    const uint32_t elect = elect_lane();
    Walk<W_MN, 2> ca(p.a_dim, f_tile * 128, k0, 0, 0);
    Walk<false, 1> cb(p.b_dim, n0, k0, 0, b);
    int st = 0;
    uint32_t parity = 1u;
    int32_t issued = 0;
    for (int32_t s = k0; s < k1; ++s) {
      if (!mbar_wait_warp(smem_u32(&ctrl.empty[st]), parity, abort_flag, &g_err, p.timeout_ns)) break;
      const uint32_t a = base + st * C::STAGE, bar = smem_u32(&ctrl.full[st]);
      mbar_arrive_expect_tx(elect, bar, C::STAGE);
      ca.template load<1>(elect, a, &p.ta, bar);
      cb.template load<1>(elect, a + C::A_BYTES, &p.tb, bar);
      ca.advance();
      cb.advance();
      ++issued;
      if (++st == C::STAGES) {
        st = 0;
        parity ^= 1u;
      }
    }
    // every copy has landed before the CTA ends; normally they all have been waited for
    volatile int32_t no = 0;
    for (int32_t k = max(0, issued - C::STAGES); k < issued; ++k)
      mbar_wait_warp(smem_u32(&ctrl.full[k % C::STAGES]), static_cast<uint32_t>(k / C::STAGES) & 1u, &no, &g_err,
                     p.timeout_ns);
  } else if (warp == 1) {
    const uint32_t elect = elect_lane();
    int st = 0;
    uint32_t parity = 0u;
    bool ok = true;
    for (int32_t s = k0; s < k1; ++s) {
      if (!mbar_wait_warp(smem_u32(&ctrl.full[st]), parity, abort_flag, &g_err, p.timeout_ns)) { ok = false; break; }
      tc_fence_after();
      const uint32_t a = base + st * C::STAGE, t = a + C::A_BYTES;
#pragma unroll
      for (int k = 0; k < BK / 16; ++k) {
        const uint64_t da = W_MN ? sdesc_sw128(a + k * 2048, 64 * 128, 1024) : sdesc_sw128(a + k * 32, 16, 1024);
        mma_bf16_ss(elect, tmem, da, sdesc_sw128(t + k * 32, 16, 1024), p.idesc, s > k0 || k > 0);
      }
      mma_commit(elect, smem_u32(&ctrl.empty[st]));
      if (p.stall && !mbar_wait_warp(smem_u32(&ctrl.never), 0, abort_flag, &g_err, p.timeout_ns)) { ok = false; break; }
      if (++st == C::STAGES) {
        st = 0;
        parity ^= 1u;
      }
    }
    if (ok) mma_commit(elect, smem_u32(&ctrl.acc_full[0]));
    mma_commit(elect, smem_u32(&ctrl.final_bar));
    // the products in flight end before TMEM is freed
    volatile int32_t no = 0;
    mbar_wait_warp(smem_u32(&ctrl.final_bar), 0, &no, &g_err, p.timeout_ns);
  } else {
    const int ew = warp - 2, quarter = warp & 3, half = ew >> 2;
    if (mbar_wait_warp(smem_u32(&ctrl.acc_full[0]), 0, abort_flag, &g_err, p.timeout_ns)) {
      tc_fence_after();
      float* sums = reinterpret_cast<float*>(smem + C::SUMS) + quarter * 32 + lane;
#pragma unroll 1
      for (int c = half * 16; c < BN; c += 32) {
        if (n0 + c >= p.n_rows) break;
        uint32_t v[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c, v);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[(c + i) * 128] = __uint_as_float(v[i]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_wait();
  // a CTA that gave up tells the others, and nobody stores (their flags read by all: 5.2 -> 5.7
  // us for 32 x 1024 -> 1024)
  if (*abort_flag && threadIdx.x < p.splits) st_cluster(cluster_addr(smem_u32(&ctrl.gave_up), threadIdx.x), 1u);
  cluster_sync();                          // all CTAs' sums lie in their shared memory
  // token rank, rank + splits, ... of the tile, 8 features a thread
  const int32_t tokens = ctrl.gave_up ? 0 : min(BN, p.n_rows - n0);
  for (int32_t i = threadIdx.x; i < (tokens - rank + p.splits - 1) / p.splits * 16; i += kThreads) {
    const int32_t t = rank + i / 16 * p.splits, f = f_tile * 128 + i % 16 * 8;
    if (f >= p.cols) continue;
    const uint32_t src = base + C::SUMS + (t * 128 + i % 16 * 8) * 4;
    F2 v[4] = {};
    for (int32_t s = 0; s < p.splits; ++s) {
      const uint32_t at = cluster_addr(src, static_cast<uint32_t>(s));
      const float4 x = ld_cluster(at), y = ld_cluster(at + 16);
      v[0] = add2(v[0], pack2(x.x, x.y));
      v[1] = add2(v[1], pack2(x.z, x.w));
      v[2] = add2(v[2], pack2(y.x, y.y));
      v[3] = add2(v[3], pack2(y.z, y.w));
    }
    by_kind(p.epi.f16, p.epi.act, [&](auto f16, auto act) { finish8<f16.value, act.value>(p.epi, v, b, n0 + t, f); });
  }
  cluster_sync();                          // nobody leaves while its sums are read
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, BN);
  }
  if (p.late) grid_wait();
}

}  // namespace linear

}  // namespace tsr
