// norm_rope.cu -- RMS norm of every head's row and the position rotation in one pass,
// forward and backward, between any two strided layouts.
//
// With r = 1 / sqrt(mean_c x_c^2 + eps), xhat = x r and R the rotation of the row's
// token (rope.cu):
//     y = R (w o xhat)
// and for a gradient dy of y, g = R^T dy, S = sum_c g_c w_c x_c:
//     dx = r (g o w - x r^2 S / d),        dw = sum over rows of g o xhat.
// The backward takes x, not y: r is computed again, nothing is kept by the forward.
//
// Bound: HBM, one read of x (and dy) and one write.  A row lies in registers across a
// group of lanes, 16 bytes each, and its sums are butterflies in the group: a pass of its
// own for the norm would read and write everything once more.  As in rope.cu a thread
// keeps its unit of pairs of one token and goes over the heads of every tensor, so the
// angles cost 1 / heads of a sincos per pair.
//
// The row's sums stand between its loads and its stores, so loads held in registers leave
// the memory idle in between (480p forward 199 us, 720p backward 876).  Every thread
// therefore has a ring of four stages of 64 bytes in shared memory, which cp.async fills
// three stages ahead, across heads and tokens, at no cost in registers and without a
// barrier: a thread reads what it copied itself.
//
// dw: a thread sums its channels over all rows it meets in fp32, the CTA adds its groups
// in shared memory and stores one partial row, and a dependent kernel adds the CTAs' rows
// in their order: no atomics, the same bits every run.
#include <algorithm>
#include <cstring>

#include "internal.h"
#include "ptx.cuh"
#include "rope_units.cuh"

namespace tsr {

namespace {

using rope::kMaxTensors;
using rope::Unit;

constexpr int kThreads = 256;
constexpr int kStages = 4;
constexpr int kCtasPerSm = 2;

struct NormParams {
  const void* x[kMaxTensors];
  const void* w[kMaxTensors];        // null: 1
  const void* g[kMaxTensors];        // backward: dy
  void* out[kMaxTensors];            // y or dx
  int64_t xs[kMaxTensors][3], gs[kMaxTensors][3], os[kMaxTensors][3];   // element strides of b, h, n
  int32_t H[kMaxTensors];
  int32_t cta0[kMaxTensors + 1];     // CTAs of each tensor, one after another
  int32_t chunk[kMaxTensors];        // heads an item takes
  rope::Angles ang;
  int32_t n_tensors, N, B, d, lanes_log2, w_f32;
  float eps;
  float* part;                       // backward: [CTA][d], null: no weight gradient
};

// The pairs of a unit as floats, first and second elements, and back.
template <typename T, int P, bool ADJ>
__device__ __forceinline__ void get(const Unit<T, P, ADJ>& u, float (&a)[P], float (&b)[P]) {
  using rope::Two;
  if constexpr (P == 1) {
    a[0] = rope::to_f(u.e0);
    b[0] = rope::to_f(u.e1);
  } else if constexpr (ADJ) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 v = Two<T>::load(u.a.w[i]);
      a[i] = v.x;
      b[i] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const float2 v = Two<T>::load(u.a.w[i]), z = Two<T>::load(u.b.w[i]);
      a[2 * i] = v.x;
      a[2 * i + 1] = v.y;
      b[2 * i] = z.x;
      b[2 * i + 1] = z.y;
    }
  }
}
template <typename T, int P, bool ADJ>
__device__ __forceinline__ void put(Unit<T, P, ADJ>& u, const float (&a)[P], const float (&b)[P]) {
  using rope::Two;
  if constexpr (P == 1) {
    u.e0 = rope::from_f<T>(a[0]);
    u.e1 = rope::from_f<T>(b[0]);
  } else if constexpr (ADJ) {
#pragma unroll
    for (int i = 0; i < P; ++i) u.a.w[i] = Two<T>::store(make_float2(a[i], b[i]));
  } else {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      u.a.w[i] = Two<T>::store(make_float2(a[2 * i], a[2 * i + 1]));
      u.b.w[i] = Two<T>::store(make_float2(b[2 * i], b[2 * i + 1]));
    }
  }
}

// Channels of a unit's pair i.
template <int P, bool ADJ>
__device__ __forceinline__ int first_of(int ch0, int i) { return P == 1 ? ch0 : ADJ ? ch0 + 2 * i : ch0 + i; }
template <int P, bool ADJ>
__device__ __forceinline__ int second_of(int ch0, int ch1, int i) {
  return P == 1 ? ch1 : ADJ ? ch0 + 2 * i + 1 : ch1 + i;
}

template <typename T>
__device__ __forceinline__ float weight_at(const NormParams& p, int t, int c) {
  if (!p.w[t]) return 1.f;
  if (p.w_f32) return __ldg(static_cast<const float*>(p.w[t]) + c);
  return rope::to_f(static_cast<const T*>(p.w[t])[c]);
}

// What a thread holds of a row, and how many rows at a time.
template <typename T, int P, bool ADJ, int K, bool GRAD>
struct Batch {
  static constexpr int PIECES = P == 1 || !ADJ ? 2 : 1;                      // of a unit
  static constexpr int BYTES = P == 1 ? sizeof(T) : (ADJ ? 2 : 1) * P * static_cast<int>(sizeof(T));   // of a piece
  static constexpr bool RING = BYTES >= 8;                                   // what cp.async copies
  static constexpr int N = K * PIECES * (GRAD ? 2 : 1);                      // pieces of a row
  static constexpr int R = !RING ? (GRAD ? 1 : 2) : 64 / (N * BYTES) < 1 ? 1 : 64 / (N * BYTES);
  static constexpr int SLOT = R * N * BYTES * kThreads;                      // a stage of the CTA
  static constexpr int RED = GRAD ? 512 * P * K * 4 : 0;                     // weight gradients of its groups
  static constexpr int SMEM = (RING ? kStages * SLOT : 0) > RED ? kStages * SLOT : RED;
  static_assert(!RING || BYTES == 8 || BYTES == 16, "a cp.async");
};

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16) cp_async_16(dst, src);
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// Where a thread is: an item (`tokens` tokens, `chunk` heads) and its next head.
struct Place {
  int64_t tile, rest, n, b;        // item = rest * tiles + tile; rest = b * chunks + chunk
  int h, h1;
};

// One CTA works on one tensor, on items of `tokens` tokens and `chunk` heads.  A row is
// K units in each of 2^lanes_log2 lanes.
template <typename T, int P, bool ADJ, int K, bool GRAD>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) norm_rope_kernel(const __grid_constant__ NormParams p) {
  using B = Batch<T, P, ADJ, K, GRAD>;
  constexpr int R = B::R;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lanes = 1 << p.lanes_log2;
  const int group = threadIdx.x >> p.lanes_log2, lane = threadIdx.x & (lanes - 1);
  const int tokens = kThreads >> p.lanes_log2;
  const uint32_t mask = (lanes == 32 ? 0xFFFFFFFFu : (1u << lanes) - 1u) << ((threadIdx.x & 31) - lane);
  int t = 0;
  while (t + 1 < p.n_tensors && static_cast<int>(blockIdx.x) >= p.cta0[t + 1]) ++t;
  const int64_t tiles = (static_cast<int64_t>(p.N) + tokens - 1) / tokens;
  const int H = p.H[t], chunk = p.chunk[t], chunks = (H + chunk - 1) / chunk;
  const int64_t rests = static_cast<int64_t>(p.B) * chunks, stride = p.cta0[t + 1] - p.cta0[t];
  const float inv_d = 1.f / p.d;

  int ch0[K], ch1[K];
  bool on[K];
  float wa[K][P], wb[K][P];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int unit = lane + k * lanes;
    on[k] = unit < p.ang.units;
    ch0[k] = on[k] ? p.ang.c0[unit] : 0;
    ch1[k] = on[k] ? p.ang.c1[unit] : 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      wa[k][i] = on[k] ? weight_at<T>(p, t, first_of<P, ADJ>(ch0[k], i)) : 0.f;
      wb[k][i] = on[k] ? weight_at<T>(p, t, second_of<P, ADJ>(ch0[k], ch1[k], i)) : 0.f;
    }
  }
  float da[K][P], db[K][P];                // weight gradients of this thread's channels
  if constexpr (GRAD) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < P; ++i) da[k][i] = db[k][i] = 0.f;
  }

  // The place's first item, or the one `tiles` and `rests` on; false behind the last.
  // Items whose token this group does not have are passed over.
  const int64_t step_tile = stride % tiles, step_rest = stride / tiles;
  auto settle = [&](Place& q) -> bool {
    while (q.rest < rests) {
      q.n = q.tile * tokens + group;
      if (q.n < p.N) {
        q.b = chunks == 1 ? q.rest : q.rest / chunks;
        q.h = chunks == 1 ? 0 : static_cast<int>(q.rest - q.b * chunks) * chunk;
        q.h1 = min(q.h + chunk, H);
        return true;
      }
      q.tile += step_tile;
      q.rest += step_rest;
      if (q.tile >= tiles) {
        q.tile -= tiles;
        ++q.rest;
      }
    }
    return false;
  };
  auto next = [&](Place& q) -> bool {
    q.tile += step_tile;
    q.rest += step_rest;
    if (q.tile >= tiles) {
      q.tile -= tiles;
      ++q.rest;
    }
    return settle(q);
  };
  const int64_t first = blockIdx.x - p.cta0[t];
  Place cur;
  cur.rest = first / tiles;
  cur.tile = first - cur.rest * tiles;
  bool live = settle(cur);

  const int64_t xs = p.xs[t][1], os = p.os[t][1], gs = GRAD ? p.gs[t][1] : 0;
  auto row_of = [&](const void* base, const int64_t (&s)[3], const Place& q) {
    return static_cast<const T*>(base) + q.b * s[0] + q.n * s[2] + q.h * s[1];
  };
  // A stage's piece of this thread.
  auto slot = [&](int stage, int j, int piece) {
    return (stage * R * B::N + j * B::N + piece) * (B::BYTES * kThreads) + threadIdx.x * B::BYTES;
  };
  Place far = cur;                         // the next rows to copy
  bool more = live;
  const T *far_x = nullptr, *far_g = nullptr;
  auto point = [&]() {
    far_x = row_of(p.x[t], p.xs[t], far);
    if constexpr (GRAD) far_g = row_of(p.g[t], p.gs[t], far);
  };
  auto fetch = [&](int stage) {
    if (more) {
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (far.h + j < far.h1) {
#pragma unroll
          for (int k = 0; k < K; ++k)
            if (on[k]) {
#pragma unroll
              for (int i = 0; i < B::PIECES; ++i) {
                const int c = i ? ch1[k] : ch0[k];
                cp_async<B::BYTES>(smem_u32(smem + slot(stage, j, k * B::PIECES + i)), far_x + j * xs + c);
                if constexpr (GRAD)
                  cp_async<B::BYTES>(smem_u32(smem + slot(stage, j, (K + k) * B::PIECES + i)), far_g + j * gs + c);
              }
            }
        }
      far.h += R;
      far_x += R * xs;
      far_g += R * gs;
      if (far.h >= far.h1) {
        more = next(far);
        if (more) point();
      }
    }
    cp_async_commit();
  };
  if constexpr (B::RING) {
    if (more) point();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
  }

  float cs[K][P], sn[K][P];
  int turning[K];
  bool whole = true;
  T* dst = nullptr;
  auto begin = [&]() {                     // an item's angles and rows
    whole = true;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      turning[k] = rope::angles_of<P>(p.ang, cur.b, cur.n, on[k] ? lane + k * lanes : p.ang.units, cs[k], sn[k]);
      whole = whole && turning[k] == P;
    }
    dst = const_cast<T*>(row_of(p.out[t], p.os[t], cur));
  };
  if (live) begin();
  int stage = 0;
  while (live) {
    Unit<T, P, ADJ> u[R][K], v[GRAD ? R : 1][K];
    if constexpr (B::RING) {
      fetch(stage ? stage - 1 : kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int k = 0; k < K; ++k) {
          auto piece = [&](int i) { return reinterpret_cast<const T*>(smem + slot(stage, j, i)); };
          const int i = k * B::PIECES, g = (K + k) * B::PIECES;
          u[j][k].load(piece(i), piece(i + B::PIECES - 1));
          if constexpr (GRAD) v[j][k].load(piece(g), piece(g + B::PIECES - 1));
        }
      stage = stage + 1 == kStages ? 0 : stage + 1;
    } else {
      const T* src = row_of(p.x[t], p.xs[t], cur);
      const T* grd = GRAD ? row_of(p.g[t], p.gs[t], cur) : nullptr;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (cur.h + j < cur.h1) {
#pragma unroll
          for (int k = 0; k < K; ++k)
            if (on[k]) {
              u[j][k].load(src + j * xs + ch0[k], src + j * xs + ch1[k]);
              if constexpr (GRAD) v[j][k].load(grd + j * gs + ch0[k], grd + j * gs + ch1[k]);
            }
        }
    }
    float ss[R], sp[R];
    float ga[GRAD ? R : 1][K][P], gb[GRAD ? R : 1][K][P];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float s0 = 0.f, s1 = 0.f, p0 = 0.f, p1 = 0.f;
      if (cur.h + j < cur.h1) {
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (on[k]) {
            float a[P], c[P];
            get(u[j][k], a, c);
#pragma unroll
            for (int i = 0; i < P; ++i) {
              s0 = fmaf(a[i], a[i], s0);
              s1 = fmaf(c[i], c[i], s1);
            }
            if constexpr (GRAD) {
              float e[P], f[P];
              get(v[j][k], e, f);
#pragma unroll
              for (int i = 0; i < P; ++i) {
                const bool turn = whole || i < turning[k];
                ga[j][k][i] = turn ? fmaf(f[i], sn[k][i], e[i] * cs[k][i]) : e[i];
                gb[j][k][i] = turn ? fmaf(f[i], cs[k][i], -(e[i] * sn[k][i])) : f[i];
                p0 = fmaf(ga[j][k][i] * wa[k][i], a[i], p0);
                p1 = fmaf(gb[j][k][i] * wb[k][i], c[i], p1);
              }
            }
          }
      }
      ss[j] = s0 + s1;
      sp[j] = p0 + p1;
    }
    for (int m = lanes >> 1; m; m >>= 1) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        ss[j] += __shfl_xor_sync(mask, ss[j], m);
        if constexpr (GRAD) sp[j] += __shfl_xor_sync(mask, sp[j], m);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (cur.h + j < cur.h1) {
        const float r = rsqrtf(fmaf(ss[j], inv_d, p.eps));
        const float along = GRAD ? r * r * sp[j] * inv_d : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (on[k]) {
            float a[P], c[P], y[P], z[P];
            get(u[j][k], a, c);
#pragma unroll
            for (int i = 0; i < P; ++i) {
              if constexpr (GRAD) {
                y[i] = r * fmaf(-a[i], along, ga[j][k][i] * wa[k][i]);
                z[i] = r * fmaf(-c[i], along, gb[j][k][i] * wb[k][i]);
                da[k][i] = fmaf(ga[j][k][i], a[i] * r, da[k][i]);
                db[k][i] = fmaf(gb[j][k][i], c[i] * r, db[k][i]);
              } else {
                const float xa = a[i] * r * wa[k][i], xc = c[i] * r * wb[k][i];
                const bool turn = whole || i < turning[k];
                y[i] = turn ? fmaf(xa, cs[k][i], -(xc * sn[k][i])) : xa;
                z[i] = turn ? fmaf(xa, sn[k][i], xc * cs[k][i]) : xc;
              }
            }
            put(u[j][k], y, z);
            u[j][k].store(dst + j * os + ch0[k], dst + j * os + ch1[k]);
          }
      }
    }
    cur.h += R;
    dst += R * os;
    if (cur.h >= cur.h1) {
      live = next(cur);
      if (live) begin();
    }
  }
  if constexpr (GRAD) {
    if (!p.part) return;
    // the ring's memory, once every thread is through with it
    if constexpr (B::RING) cp_async_wait_all();
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (on[k]) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          red[group * p.d + first_of<P, ADJ>(ch0[k], i)] = da[k][i];
          red[group * p.d + second_of<P, ADJ>(ch0[k], ch1[k], i)] = db[k][i];
        }
      }
    __syncthreads();
    grid_launch_dependents();
    for (int c = threadIdx.x; c < p.d; c += kThreads) {
      float s = 0.f;
      for (int q = 0; q < tokens; ++q) s += red[q * p.d + c];
      p.part[static_cast<int64_t>(blockIdx.x) * p.d + c] = s;
    }
  }
}

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

// Lanes that share a row, and units each of them holds.
struct Shape {
  int lanes_log2, K;
};
Shape shape_of(int units, int P) {
  Shape s{0, P == 1 ? 4 : units > 32 ? 2 : 1};
  while ((1 << s.lanes_log2) < units && s.lanes_log2 < 5) ++s.lanes_log2;
  return s;
}

// CTAs of each tensor: as many as run together, in proportion to the tensors' heads, or one
// for each item where there are fewer.  An item takes all heads of its tokens (their angles
// are computed once) unless there are too few items for the card.
void spread(NormParams& p, int sms) {
  const int tokens = kThreads >> p.lanes_log2;
  const int64_t tiles = (static_cast<int64_t>(p.N) + tokens - 1) / tokens * p.B;
  const int64_t want = static_cast<int64_t>(sms) * kCtasPerSm;
  int64_t rows = 0;
  for (int i = 0; i < p.n_tensors; ++i) rows += p.H[i];
  p.cta0[0] = 0;
  for (int i = 0; i < p.n_tensors; ++i) {
    int64_t chunks = std::min<int64_t>(p.H[i], std::max<int64_t>(1, want / (tiles * p.n_tensors)));
    p.chunk[i] = static_cast<int32_t>((p.H[i] + chunks - 1) / chunks);
    chunks = (p.H[i] + p.chunk[i] - 1) / p.chunk[i];
    const int64_t share = std::max<int64_t>(1, (want * p.H[i] + rows / 2) / rows);
    p.cta0[i + 1] = p.cta0[i] + static_cast<int32_t>(std::min<int64_t>(tiles * chunks, share));
  }
}

tsr_status launch_one(void (*kern)(NormParams), int smem, unsigned ctas, const NormParams& p, cudaStream_t st) {
  if (smem > 48 * 1024) TSR_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  kern<<<ctas, kThreads, smem, st>>>(p);
  TSR_CUDA(cudaGetLastError());
  return TSR_OK;
}

template <bool GRAD>
tsr_status launch(const NormParams& p, int dtype, bool halves, int P, int K, cudaStream_t st) {
  const unsigned ctas = static_cast<unsigned>(p.cta0[p.n_tensors]);
#define TSR_NORM(T, P_, ADJ_, K_)                                              \
  if (P == P_ && halves != ADJ_ && K == K_) {                                  \
    return launch_one(norm_rope_kernel<T, P_, ADJ_, K_, GRAD>, Batch<T, P_, ADJ_, K_, GRAD>::SMEM, ctas, p, st); \
  }
#define TSR_NORM_16(T)      \
  TSR_NORM(T, 4, true, 1)   \
  TSR_NORM(T, 1, true, 4)   \
  TSR_NORM(T, 8, false, 1)  \
  TSR_NORM(T, 4, false, 1)  \
  TSR_NORM(T, 1, false, 4)
  if (dtype == TSR_DTYPE_BF16) {
    TSR_NORM_16(__nv_bfloat16)
  } else if (dtype == TSR_DTYPE_F16) {
    TSR_NORM_16(__half)
  } else {
    TSR_NORM(float, 2, true, 1)
    TSR_NORM(float, 2, true, 2)
    TSR_NORM(float, 1, true, 4)
    TSR_NORM(float, 4, false, 1)
    TSR_NORM(float, 1, false, 4)
  }
#undef TSR_NORM_16
#undef TSR_NORM
  return fail(TSR_ERR_INTERNAL, "no norm kernel for this layout");
}

// Parameters of a call; returns the pairs per unit.
int fill(const tsr_rope_desc& d, double eps, const tsr_norm_rope_tensor* t, int32_t n, bool grad, NormParams& p) {
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
  return rope::fill_angles(d, bits, p.ang);
}

}  // namespace

// The arguments of the three have been checked (api_layer.cu).
tsr_status launch_norm_rope(const tsr_rope_desc& d, double eps, const tsr_norm_rope_tensor* t, int32_t n,
                            cudaStream_t st) {
  NormParams p;
  const int P = fill(d, eps, t, n, false, p);
  const Shape s = shape_of(p.ang.units, P);
  p.lanes_log2 = s.lanes_log2;
  int dev = 0;
  TSR_CUDA(cudaGetDevice(&dev));
  spread(p, num_sms(dev));
  return launch<false>(p, d.dtype, d.halves != 0, P, s.K, st);
}

// One partial row of weight gradients per CTA that any call of this shape may use.
size_t norm_rope_workspace(const tsr_rope_desc& d, int32_t n) {
  constexpr int64_t kMostSms = 256;
  return static_cast<size_t>((kMostSms * kCtasPerSm + 2 * n) * d.d) * sizeof(float);
}

tsr_status launch_norm_rope_backward(const tsr_rope_desc& d, double eps, const tsr_norm_rope_tensor* t, int32_t n,
                                     void* ws, cudaStream_t st) {
  NormParams p;
  const int P = fill(d, eps, t, n, true, p);
  const Shape s = shape_of(p.ang.units, P);
  p.lanes_log2 = s.lanes_log2;
  int dev = 0;
  TSR_CUDA(cudaGetDevice(&dev));
  spread(p, std::min(num_sms(dev), 256));
  SumParams q;
  memset(&q, 0, sizeof q);
  bool any = false;
  for (int i = 0; i < n; ++i) {
    q.dw[i] = t[i].dweight;
    any = any || t[i].dweight;
  }
  p.part = any ? static_cast<float*>(ws) : nullptr;
  if (tsr_status e = launch<true>(p, d.dtype, d.halves != 0, P, s.K, st)) return e;
  if (!any) return TSR_OK;
  q.part = p.part;
  memcpy(q.cta0, p.cta0, sizeof q.cta0);
  q.d = d.d;
  q.dtype = p.w_f32 ? TSR_DTYPE_F32 : d.dtype;
  TSR_CUDA(launch_dependent(norm_weight_kernel, static_cast<unsigned>(n * ((d.d + 31) / 32)), 1024u, 0, st, q));
  return TSR_OK;
}

}  // namespace tsr
