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
#include <algorithm>
#include <cstring>

#include "internal.h"
#include "rope_units.cuh"

namespace tsr {

namespace {

using rope::kMaxTensors;
using rope::Unit;

constexpr int kThreads = 256;
constexpr int kRows = 4;           // heads a CTA takes at least, where there are enough

struct RopeParams {
  const void* x[kMaxTensors];
  void* out[kMaxTensors];
  int64_t xs[kMaxTensors][3], os[kMaxTensors][3];   // element strides of b, h, n
  int32_t row0[kMaxTensors + 1];                    // rows (t, h) numbered tensor after tensor
  rope::Angles ang;
  int32_t n_tensors, N, tokens, rows_per_cta;
};

template <typename T, int P, bool ADJ>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  // heads whose loads are in flight together: 128 bytes a thread
  constexpr int R = P == 1 ? 8 : (ADJ ? 8 : 4);
  const int tok = threadIdx.x / p.ang.units, unit = threadIdx.x - tok * p.ang.units;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * p.tokens + tok;
  if (tok >= p.tokens || n >= p.N) return;
  const int64_t b = blockIdx.z;
  float cs[P], sn[P];
  const int turning = rope::angles_of<P>(p.ang, b, n, unit, cs, sn);
  const int ch0 = p.ang.c0[unit], ch1 = p.ang.c1[unit];
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
  p.tokens = threads / p.ang.units;
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
  const int P = rope::fill_angles(d, bits, p.ang);
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
