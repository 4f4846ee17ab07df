// rope.cu -- rotary positions with several axes (time, height, width), forward
// and backward, between any two strided layouts.
//
// Channels [c_x, c_x + D_x) of a head belong to axis x and hold D_x / 2 pairs;
// pair j of a token at position p_x turns by the angle p_x * theta^(-2 j / D_x):
//     (a, b) -> (a cos - b sin, a sin + b cos).
// The rotation is orthogonal, so its gradient is the same kernel with -angle.
//
// Angles.  A frequency is held in turns as a 64-bit fixed-point fraction
// F = round(2^64 * theta^(-2 j / D_x) / 2 pi); p * F mod 2^64 is then the angle's
// place on the circle, exact in integer arithmetic but for F itself, which comes from
// doubles: off by a few 2^-54 of the frequency (at most 1 / 2 pi of a turn for theta
// >= 1), so about p * 2^-55 of a turn: 4e-7 rad at position 2^31, 2e-11 at 100,000.  Its top
// bits go to sincospi as a float in [-1, 1).  (p * freq in fp32 would be off by 2^-24
// of the whole angle, 0.006 rad at position 100,000.)
//
// Bound: HBM, one read and one write of every element.  A thread owns one unit of
// pairs of one token (16 bytes, or two 16-byte pieces for half-split pairs),
// computes its few cosines and sines once, and applies them to every head of
// every tensor of the call, 128 bytes of loads in flight; the angles so cost
// 1 / (heads * tensors) of a sincos per pair.  Strides are free, so the
// projections' [B, N, H, d] is read in place and the attention's [B, H, N, d]
// written without a transposing copy.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "internal.h"

namespace tsr {

namespace {

constexpr int kMaxPairs = 128;     // d <= 256
constexpr int kMaxTensors = 4;
constexpr int kThreads = 256;
constexpr int kRows = 4;           // heads a CTA takes at least, where there are enough

struct RopeParams {
  const void* x[kMaxTensors];
  void* out[kMaxTensors];
  int64_t xs[kMaxTensors][3], os[kMaxTensors][3];   // element strides of b, h, n
  int32_t row0[kMaxTensors + 1];                    // rows (t, h) numbered tensor after tensor
  const int32_t* positions;
  int64_t pos_batch;              // elements between batches' positions (0: shared)
  int32_t n_tensors, N, n_axes, n_pairs, units, tokens, rows_per_cta, inverse;
  int32_t extent[4];
  uint64_t freq[kMaxPairs];       // turns per position, 2^64 = one turn
  uint8_t axis[kMaxPairs];
  uint16_t c0[kMaxPairs], c1[kMaxPairs];   // a unit's first channels (halves: both pieces)
};

// Two values of type T as floats, and back (16-bit types: one 32-bit word).
template <typename T>
struct Two;
template <>
struct Two<float> {
  using Word = float2;
  static __device__ __forceinline__ float2 load(Word w) { return w; }
  static __device__ __forceinline__ Word store(float2 v) { return v; }
};
template <>
struct Two<__half> {
  using Word = uint32_t;
  static __device__ __forceinline__ float2 load(Word w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ Word store(float2 v) {
    const __half2 h = __float22half2_rn(v);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Two<__nv_bfloat16> {
  using Word = uint32_t;
  static __device__ __forceinline__ float2 load(Word w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ Word store(float2 v) {
    const __nv_bfloat162 h = __float22bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

template <typename T>
__device__ __forceinline__ float to_f(T v) { return static_cast<float>(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v) { return static_cast<T>(v); }   // to nearest even

// A row's unit in registers.  ADJ: P pairs of neighbouring channels, one piece.
// Otherwise two pieces of P channels.  P = 1: two single elements either way.
template <typename T, int P, bool ADJ>
struct Unit {
  static constexpr int WORDS = P == 1 ? 1 : ADJ ? P : P / 2;     // per piece
  using Word = typename Two<T>::Word;
  struct alignas(sizeof(Word) * WORDS) Piece {
    Word w[WORDS];
  };
  Piece a, b;
  T e0, e1;
  __device__ __forceinline__ void load(const T* p0, const T* p1) {
    if constexpr (P == 1) {
      e0 = *p0;
      e1 = *p1;
    } else {
      a = *reinterpret_cast<const Piece*>(p0);
      if constexpr (!ADJ) b = *reinterpret_cast<const Piece*>(p1);
    }
  }
  __device__ __forceinline__ void store(T* p0, T* p1) const {
    if constexpr (P == 1) {
      *p0 = e0;
      *p1 = e1;
    } else {
      *reinterpret_cast<Piece*>(p0) = a;
      if constexpr (!ADJ) *reinterpret_cast<Piece*>(p1) = b;
    }
  }
  // channels past the rotated ones (pairs from `n` on) stay bit for bit
  __device__ __forceinline__ void turn(const float (&cs)[P], const float (&sn)[P], int n) {
    if constexpr (P == 1) {
      if (n > 0) {
        const float u = to_f(e0), v = to_f(e1);
        e0 = from_f<T>(u * cs[0] - v * sn[0]);
        e1 = from_f<T>(u * sn[0] + v * cs[0]);
      }
    } else if constexpr (ADJ) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float2 x = Two<T>::load(a.w[i]);
        const Word y = Two<T>::store(make_float2(x.x * cs[i] - x.y * sn[i], x.x * sn[i] + x.y * cs[i]));
        if (i < n) a.w[i] = y;
      }
    } else {
      // n is 0 or P: a unit of half-split pairs lies in one axis or past them all
      if (n == 0) return;
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        const float2 u = Two<T>::load(a.w[i]), v = Two<T>::load(b.w[i]);
        const float c0 = cs[2 * i], c1 = cs[2 * i + 1], s0 = sn[2 * i], s1 = sn[2 * i + 1];
        a.w[i] = Two<T>::store(make_float2(u.x * c0 - v.x * s0, u.y * c1 - v.y * s1));
        b.w[i] = Two<T>::store(make_float2(u.x * s0 + v.x * c0, u.y * s1 + v.y * c1));
      }
    }
  }
};

template <typename T, int P, bool ADJ>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  // heads whose loads are in flight together: 128 bytes a thread
  constexpr int R = P == 1 ? 8 : (ADJ ? 8 : 4);
  const int tok = threadIdx.x / p.units, unit = threadIdx.x - tok * p.units;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * p.tokens + tok;
  if (tok >= p.tokens || n >= p.N) return;
  const int64_t b = blockIdx.z;
  float cs[P], sn[P];
  const int turning = min(max(p.n_pairs - unit * P, 0), P);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
    if (i < turning) {
      const int pair = unit * P + i, ax = p.axis[pair];
      int64_t pos;
      if (p.positions) {
        pos = __ldg(p.positions + b * p.pos_batch + n * p.n_axes + ax);
      } else {
        int32_t rest = static_cast<int32_t>(n);
        for (int a = p.n_axes - 1; a > ax; --a) rest /= p.extent[a];
        pos = ax ? rest % p.extent[ax] : rest;
      }
      const uint64_t turn = static_cast<uint64_t>(pos) * p.freq[pair];
      // half turns in [-1, 1): sincospi takes the angle over pi
      const float half_turns = static_cast<float>(static_cast<int64_t>(turn)) * 0x1p-63f;
      sincospif(half_turns, &sn[i], &cs[i]);
      if (p.inverse) sn[i] = -sn[i];
    }
  }
  const int ch0 = p.c0[unit], ch1 = p.c1[unit];
  const int lo = blockIdx.y * p.rows_per_cta, hi = min(lo + p.rows_per_cta, p.row0[p.n_tensors]);
  for (int t = 0; t < p.n_tensors; ++t) {
    const int h0 = max(lo - p.row0[t], 0), h1 = min(hi, p.row0[t + 1]) - p.row0[t];
    const int64_t xs = p.xs[t][1], os = p.os[t][1];
    const T* src = static_cast<const T*>(p.x[t]) + b * p.xs[t][0] + n * p.xs[t][2] + h0 * xs;
    T* dst = static_cast<T*>(p.out[t]) + b * p.os[t][0] + n * p.os[t][2] + h0 * os;
    int h = h0;
    for (; h + R <= h1; h += R, src += R * xs, dst += R * os) {
      Unit<T, P, ADJ> u[R];
#pragma unroll
      for (int k = 0; k < R; ++k) u[k].load(src + k * xs + ch0, src + k * xs + ch1);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        u[k].turn(cs, sn, turning);
        u[k].store(dst + k * os + ch0, dst + k * os + ch1);
      }
    }
    for (; h < h1; ++h, src += xs, dst += os) {
      Unit<T, P, ADJ> u;
      u.load(src + ch0, src + ch1);
      u.turn(cs, sn, turning);
      u.store(dst + ch0, dst + ch1);
    }
  }
}

template <typename T, int P, bool ADJ>
tsr_status launch(RopeParams& p, int32_t B, cudaStream_t st) {
  const int threads = kThreads;
  p.tokens = threads / p.units;
  const int rows = p.row0[p.n_tensors];
  int dev = 0;
  TSR_CUDA(cudaGetDevice(&dev));
  // heads are spread over CTAs only until there are four CTAs per SM: each CTA
  // computes its tokens' angles once
  const int64_t tiles = (static_cast<int64_t>(p.N) + p.tokens - 1) / p.tokens;
  const int64_t want = static_cast<int64_t>(num_sms(dev)) * 4;
  int64_t groups = std::min<int64_t>((rows + kRows - 1) / kRows, (want + tiles * B - 1) / (tiles * B));
  if (tiles * B * ((rows + kRows - 1) / kRows) < want) groups = rows;
  p.rows_per_cta = static_cast<int32_t>((rows + groups - 1) / groups);
  groups = (rows + p.rows_per_cta - 1) / p.rows_per_cta;
  if (groups > 65535) return fail(TSR_ERR_UNSUPPORTED, "too many heads");
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(groups), static_cast<unsigned>(B));
  rope_kernel<T, P, ADJ><<<grid, threads, 0, st>>>(p);
  TSR_CUDA(cudaGetLastError());
  return TSR_OK;
}

}  // namespace

// The arguments have been checked (api_ops.cu).
tsr_status launch_rope(const tsr_rope_desc& d, const tsr_rope_tensor* t, int32_t n, cudaStream_t st) {
  RopeParams p;
  memset(&p, 0, sizeof p);
  const size_t es = d.dtype == TSR_DTYPE_F32 ? 4 : 2;
  p.n_tensors = n;
  p.N = d.N;
  p.n_axes = d.n_axes;
  p.positions = d.positions;
  p.pos_batch = d.positions_per_batch ? static_cast<int64_t>(d.N) * d.n_axes : 0;
  p.inverse = d.inverse != 0;
  int32_t at = 0;
  for (int a = 0; a < d.n_axes; ++a) {
    p.extent[a] = d.positions ? 1 : d.grid[a];
    for (int j = 0; j < d.axis_dim[a] / 2; ++j) {
      const double turns = std::pow(d.theta, -2.0 * j / d.axis_dim[a]) / 6.283185307179586476925286766559;
      // the fraction of a turn, as 2^64 fixed point (whole turns drop out)
      const double frac = turns - std::floor(turns);
      const double scaled = frac * 18446744073709551616.0;
      p.freq[at / 2 + j] = scaled >= 18446744073709551615.0 ? 0u : static_cast<uint64_t>(scaled + 0.5);
      p.axis[at / 2 + j] = static_cast<uint8_t>(a);
    }
    at += d.axis_dim[a];
  }
  p.n_pairs = at / 2;
  // The largest piece (in bytes) that every pointer, stride and, for half-split
  // pairs, half width allows.
  uint64_t bits = 0;
  for (int i = 0; i < n; ++i) {
    p.x[i] = t[i].x;
    p.out[i] = t[i].out;
    for (int k = 0; k < 3; ++k) {
      p.xs[i][k] = t[i].x_stride[k];
      p.os[i][k] = t[i].out_stride[k];
      bits |= static_cast<uint64_t>(t[i].x_stride[k]) * es | static_cast<uint64_t>(t[i].out_stride[k]) * es;
    }
    bits |= reinterpret_cast<uint64_t>(t[i].x) | reinterpret_cast<uint64_t>(t[i].out);
    p.row0[i + 1] = p.row0[i] + t[i].H;
  }
  bits |= static_cast<uint64_t>(d.d) * es;
  if (d.halves)
    for (int a = 0; a < d.n_axes; ++a) bits |= static_cast<uint64_t>(d.axis_dim[a] / 2) * es;
  const int bytes = (bits & 15) == 0 ? 16 : (bits & 7) == 0 ? 8 : static_cast<int>(es);
  // pairs per unit
  int P = d.halves ? bytes / static_cast<int>(es) : bytes / (2 * static_cast<int>(es));
  if (!d.halves && bytes < 16) P = 1;
  if (d.halves && bytes == 8 && es == 4) P = 1;
  // half-split pairs: the channels that are not rotated are paired off too, P and P
  if (d.halves && (d.d - at) % (2 * P)) P = 1;
  p.units = (d.d / 2) / P;
  for (int u = 0; u < p.units; ++u) {
    const int pair = u * P;
    if (!d.halves) {
      p.c0[u] = static_cast<uint16_t>(2 * pair);
      p.c1[u] = static_cast<uint16_t>(2 * pair + 1);
    } else if (pair < p.n_pairs) {
      int c = 0, a = 0;
      while (pair >= (c + d.axis_dim[a]) / 2) c += d.axis_dim[a++];
      p.c0[u] = static_cast<uint16_t>(c + (pair - c / 2));
      p.c1[u] = static_cast<uint16_t>(p.c0[u] + d.axis_dim[a] / 2);
    } else {
      p.c0[u] = static_cast<uint16_t>(2 * pair);
      p.c1[u] = static_cast<uint16_t>(2 * pair + P);
    }
  }
#define TSR_ROPE(T, P_, ADJ_) return launch<T, P_, ADJ_>(p, d.B, st)
#define TSR_ROPE_16(T)                  \
  if (!d.halves) {                      \
    if (P == 4) TSR_ROPE(T, 4, true);   \
    TSR_ROPE(T, 1, true);               \
  }                                     \
  if (P == 8) TSR_ROPE(T, 8, false);    \
  if (P == 4) TSR_ROPE(T, 4, false);    \
  TSR_ROPE(T, 1, false)
  switch (d.dtype) {
    case TSR_DTYPE_BF16:
      TSR_ROPE_16(__nv_bfloat16);
    case TSR_DTYPE_F16:
      TSR_ROPE_16(__half);
    default:
      if (!d.halves) {
        if (P == 2) TSR_ROPE(float, 2, true);
        TSR_ROPE(float, 1, true);
      }
      if (P == 4) TSR_ROPE(float, 4, false);
      TSR_ROPE(float, 1, false);
  }
#undef TSR_ROPE_16
#undef TSR_ROPE
}

}  // namespace tsr
