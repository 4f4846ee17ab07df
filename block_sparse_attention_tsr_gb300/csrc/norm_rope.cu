// norm_rope.cu -- RMS norm of every head's row with the position rotation: the host side of
// both directions, the forward's kernels and the sum of the weights' gradients
// (norm_rope_kernel.cuh).
#include <algorithm>
#include <cstring>

#include "norm_rope_kernel.cuh"

namespace tsr {

namespace norm {

template tsr_status launch<false>(const NormParams&, int, const Shape&, cudaStream_t);

namespace {

struct SumParams {
  const float* part;
  void* dw[kMaxTensors];
  int32_t cta0[kMaxTensors + 1];
  int32_t d, dtype;
};

// dw of one tensor and 32 channels: the CTAs' rows, 32 at a time.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const __grid_constant__ SumParams p) {
  __shared__ float red[32][33];
  const int blocks = (p.d + 31) / 32, t = blockIdx.x / blocks, lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = (blockIdx.x % blocks) * 32 + lane;
  grid_wait();
  float s = 0.f;
  if (c < p.d)
    for (int i = p.cta0[t] + slice; i < p.cta0[t + 1]; i += 32) s += p.part[static_cast<int64_t>(i) * p.d + c];
  red[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < p.d && p.dw[t]) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][lane];
    if (p.dtype == TSR_DTYPE_F32) static_cast<float*>(p.dw[t])[c] = s;
    else if (p.dtype == TSR_DTYPE_BF16) static_cast<__nv_bfloat16*>(p.dw[t])[c] = __float2bfloat16_rn(s);
    else static_cast<__half*>(p.dw[t])[c] = __float2half_rn(s);
  }
}

// CTAs of each tensor: as many as run together, in proportion to the tensors' heads and four
// more (an item's angles take about as long as four rows), or one for each item where there
// are fewer.  An item takes all heads of its tokens (their angles
// are computed once) unless there are too few items for the card.
void spread(NormParams& p, int ctas) {
  const int tokens = kThreads >> p.lanes_log2;
  const int64_t tiles = (static_cast<int64_t>(p.N) + tokens - 1) / tokens * p.B;
  const int64_t want = ctas;
  int64_t rows = 0;
  for (int i = 0; i < p.n_tensors; ++i) rows += p.H[i] + 4;
  p.cta0[0] = 0;
  for (int i = 0; i < p.n_tensors; ++i) {
    int64_t chunks = std::min<int64_t>(p.H[i], std::max<int64_t>(1, want / (tiles * p.n_tensors)));
    p.chunk[i] = static_cast<int32_t>((p.H[i] + chunks - 1) / chunks);
    chunks = (p.H[i] + p.chunk[i] - 1) / p.chunk[i];
    const int64_t share = std::max<int64_t>(1, (want * (p.H[i] + 4) + rows / 2) / rows);
    p.cta0[i + 1] = p.cta0[i] + static_cast<int32_t>(std::min<int64_t>(tiles * chunks, share));
  }
}

// Parameters of a call, the lanes that share a row among them.
Shape fill(const tsr_rope_desc& d, double eps, const tsr_norm_rope_tensor* t, int32_t n, bool grad, NormParams& p) {
  memset(&p, 0, sizeof p);
  const size_t es = d.dtype == TSR_DTYPE_F32 ? 4 : 2;
  p.n_tensors = n;
  p.N = d.N;
  p.B = d.B;
  p.d = d.d;
  p.eps = static_cast<float>(eps);
  uint64_t bits = 0;
  for (int i = 0; i < n; ++i) {
    p.x[i] = t[i].x;
    p.w[i] = t[i].weight;
    p.out[i] = t[i].out;
    p.H[i] = t[i].H;
    p.w_f32 = t[i].weight_dtype == TSR_DTYPE_F32;
    bits |= reinterpret_cast<uint64_t>(t[i].x) | reinterpret_cast<uint64_t>(t[i].out);
    if (grad) {
      p.g[i] = t[i].dout;
      bits |= reinterpret_cast<uint64_t>(t[i].dout);
    }
    const int64_t size[3] = {d.B, t[i].H, d.N};
    for (int k = 0; k < 3; ++k) {
      if (size[k] == 1) continue;
      p.xs[i][k] = t[i].x_stride[k];
      p.os[i][k] = t[i].out_stride[k];
      if (grad) p.gs[i][k] = t[i].dout_stride[k];
      bits |= static_cast<uint64_t>(p.xs[i][k] | p.os[i][k] | p.gs[i][k]) * es;
    }
  }
  bits |= static_cast<uint64_t>(d.d) * es;
  for (int a = 0; a < d.n_axes; ++a) p.inv_extent[a] = d.positions ? 0.f : 1.f / d.grid[a];
  // A unit is 16 bytes of neighbouring pairs, or two pieces of 8 (fp32: 16) bytes of half-split
  // ones, where rows start on 16 bytes and the half widths are whole pieces; else its pairs
  // are gathered one by one, from the ring or, of rows that start elsewhere, from memory.
  Shape s{static_cast<int>(16 / (2 * es)), NEAR, 1};
  const bool rows = (bits & 15) == 0;
  if (d.halves && rows) {
    int32_t width = 0;
    uint64_t halves = 0;
    for (int a = 0; a < d.n_axes; ++a) {
      halves |= static_cast<uint64_t>(d.axis_dim[a] / 2) * es;
      width += d.axis_dim[a];
    }
    halves |= static_cast<uint64_t>(d.d - width) / 2 * es;
    s.L = halves % (4 * es) ? ANY : HALVES;
    s.P = s.L == HALVES ? 4 : s.P;
    bits |= s.L == ANY ? es : 4 * es;
  } else if (!rows) {
    s.P = 1;
    s.L = HALVES;
    bits |= es;
  }
  rope::fill_angles(d, bits, p.ang);
  p.ang.units = d.d / 2 / s.P;
  s.K = s.P == 1 ? 4 : p.ang.units > 32 ? 2 : 1;
  while ((1 << p.lanes_log2) < p.ang.units && p.lanes_log2 < 5) ++p.lanes_log2;
  return s;
}

}  // namespace

}  // namespace norm

using namespace norm;

// The arguments of the three have been checked (api_layer.cu).
tsr_status launch_norm_rope(const tsr_rope_desc& d, double eps, const tsr_norm_rope_tensor* t, int32_t n,
                            cudaStream_t st) {
  NormParams p;
  const Shape s = fill(d, eps, t, n, false, p);
  int dev = 0;
  TSR_CUDA(cudaGetDevice(&dev));
  spread(p, num_sms(dev) * ctas_per_sm(false, s.P, s.L));
  return launch<false>(p, d.dtype, s, st);
}

// One partial row of weight gradients per CTA that any call of this shape may use.
size_t norm_rope_workspace(const tsr_rope_desc& d, int32_t n) {
  constexpr int64_t kMostSms = 256;
  return static_cast<size_t>((kMostSms * 2 + 2 * n) * d.d) * sizeof(float);
}

tsr_status launch_norm_rope_backward(const tsr_rope_desc& d, double eps, const tsr_norm_rope_tensor* t, int32_t n,
                                     void* ws, cudaStream_t st) {
  NormParams p;
  const Shape s = fill(d, eps, t, n, true, p);
  int dev = 0;
  TSR_CUDA(cudaGetDevice(&dev));
  spread(p, std::min(num_sms(dev), 256) * ctas_per_sm(true, s.P, s.L));
  SumParams q;
  memset(&q, 0, sizeof q);
  bool any = false;
  for (int i = 0; i < n; ++i) {
    q.dw[i] = t[i].dweight;
    any = any || t[i].dweight;
  }
  p.part = any ? static_cast<float*>(ws) : nullptr;
  if (tsr_status e = launch<true>(p, d.dtype, s, st)) return e;
  if (!any) return TSR_OK;
  q.part = p.part;
  memcpy(q.cta0, p.cta0, sizeof q.cta0);
  q.d = d.d;
  q.dtype = p.w_f32 ? TSR_DTYPE_F32 : d.dtype;
  TSR_CUDA(launch_dependent(norm_weight_kernel, static_cast<unsigned>(n * ((d.d + 31) / 32)), 1024u, 0, st, q));
  return TSR_OK;
}

}  // namespace tsr
