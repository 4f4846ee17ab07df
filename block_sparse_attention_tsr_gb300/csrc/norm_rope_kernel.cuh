// norm_rope_kernel.cuh -- RMS norm of every head's row and the position rotation in one pass,
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
// therefore has 32 bytes (backward: of both rows, 64) in each of the two stages of a ring in
// shared memory, which cp.async fills one stage ahead, across heads and tokens, at no cost in
// registers; the lanes that share a row need the warp's barrier only.  A third stage only
// adds instructions and rows in flight (forward 126 -> 127 us, backward 426 -> 465).
// 32,760 tokens of 24 + 24 heads of 128, forward: 126 to 128 us, 6.3 TB/s, 93% of a copy's rate
// (fp32 264 us, 90%); 75,600 tokens backward: 426 to 428 us, 6.5 TB/s, 96%.
//
// dw: a thread sums its channels over all rows it meets in fp32, the CTA adds its groups
// in shared memory and stores one partial row, and a dependent kernel adds the CTAs' rows
// in their order: no atomics, the same bits every run.
#pragma once
#include "internal.h"
#include "ptx.cuh"
#include "rope_units.cuh"

namespace tsr {

namespace norm {

using rope::kMaxTensors;
using rope::Unit;

constexpr int kThreads = 256;
constexpr int kStages = 2;
// How a unit's pairs lie in a row: NEAR, neighbouring channels; HALVES, two pieces of P
// channels; ANY, pair by pair (half-split pairs whose half widths are no whole pieces), which
// are gathered from the ring's row and put back there before it is stored.
enum Layout { NEAR, HALVES, ANY };

// CTAs that an SM holds, by registers: a third one where 80 a thread are enough (forward
// 141 -> 126 us; ANY's gathers need more, 80 -> 87)
constexpr int ctas_per_sm(bool grad, int P, int L) { return grad || P == 1 || L == ANY ? 2 : 3; }

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
  float inv_extent[4];
  int32_t n_tensors, N, B, d, lanes_log2, w_f32;
  float eps;
  float* part;                       // backward: [CTA][d], null: no weight gradient
};

// The pairs of a unit as floats, first elements and second elements, two pairs a register
// (P = 1: the other half is 0), and back.
template <typename T, int P, bool ADJ>
__device__ __forceinline__ void get(const Unit<T, P, ADJ>& u, F2 (&a)[(P + 1) / 2], F2 (&b)[(P + 1) / 2]) {
  using rope::Two;
  if constexpr (P == 1) {
    a[0] = pack2(rope::to_f(u.e0), 0.f);
    b[0] = pack2(rope::to_f(u.e1), 0.f);
  } else if constexpr (ADJ) {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const float2 v = Two<T>::load(u.a.w[2 * i]), z = Two<T>::load(u.a.w[2 * i + 1]);
      a[i] = pack2(v.x, z.x);
      b[i] = pack2(v.y, z.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const float2 v = Two<T>::load(u.a.w[i]), z = Two<T>::load(u.b.w[i]);
      a[i] = pack2(v.x, v.y);
      b[i] = pack2(z.x, z.y);
    }
  }
}
template <typename T, int P, bool ADJ>
__device__ __forceinline__ void put(Unit<T, P, ADJ>& u, const F2 (&a)[(P + 1) / 2], const F2 (&b)[(P + 1) / 2]) {
  using rope::Two;
  if constexpr (P == 1) {
    u.e0 = rope::from_f<T>(unpack2(a[0]).x);
    u.e1 = rope::from_f<T>(unpack2(b[0]).x);
  } else {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const float2 v = unpack2(a[i]), z = unpack2(b[i]);
      if constexpr (ADJ) {
        u.a.w[2 * i] = Two<T>::store(make_float2(v.x, z.x));
        u.a.w[2 * i + 1] = Two<T>::store(make_float2(v.y, z.y));
      } else {
        u.a.w[i] = Two<T>::store(v);
        u.b.w[i] = Two<T>::store(z);
      }
    }
  }
}

// Channels of a unit's pair i.  at: a unit's first channels, first and second piece; of ANY
// each pair's, 16 bits each.
template <int P, int L>
struct Channels {
  uint32_t at[L == ANY ? P : 1];
  __device__ __forceinline__ int first(int i) const {
    return L == ANY ? at[L == ANY ? i : 0] & 0xFFFF : (at[0] & 0xFFFF) + (P == 1 ? 0 : L == NEAR ? 2 * i : i);
  }
  __device__ __forceinline__ int second(int i) const {
    return L == ANY ? at[L == ANY ? i : 0] >> 16
                    : L == NEAR && P > 1 ? (at[0] & 0xFFFF) + 2 * i + 1 : (at[0] >> 16) + (P == 1 ? 0 : i);
  }
  __device__ __forceinline__ void set(const rope::Angles& a, int unit) {
    if constexpr (L == ANY) {
#pragma unroll
      for (int i = 0; i < P; ++i) at[i] = a.c0[unit * P + i] | static_cast<uint32_t>(a.c1[unit * P + i]) << 16;
    } else {
      at[0] = a.c0[unit] | static_cast<uint32_t>(a.c1[unit]) << 16;
    }
  }
};
// A unit in registers: ANY's pairs lie there as neighbours.
template <typename T, int P, int L>
using UnitOf = Unit<T, P, L != HALVES>;

template <typename T, int P, int L>
__device__ __forceinline__ void gather(UnitOf<T, P, L>& u, const T* row, const Channels<P, L>& c) {
  if constexpr (L == ANY) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      struct alignas(2 * sizeof(T)) Both {
        T a, b;
      } v{row[c.first(i)], row[c.second(i)]};
      u.a.w[i] = *reinterpret_cast<const typename rope::Two<T>::Word*>(&v);
    }
  } else {
    u.load(row + c.first(0), row + c.second(0));
  }
}
template <typename T, int P, int L>
__device__ __forceinline__ void scatter(const UnitOf<T, P, L>& u, T* row, const Channels<P, L>& c) {
  if constexpr (L == ANY) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      struct alignas(2 * sizeof(T)) Both {
        T a, b;
      };
      const Both v = *reinterpret_cast<const Both*>(&u.a.w[i]);
      row[c.first(i)] = v.a;
      row[c.second(i)] = v.b;
    }
  } else {
    u.store(row + c.first(0), row + c.second(0));
  }
}

template <typename T>
__device__ __forceinline__ float weight_at(const NormParams& p, int t, int c) {
  if (!p.w[t]) return 1.f;
  if (p.w_f32) return __ldg(static_cast<const float*>(p.w[t]) + c);
  return rope::to_f(static_cast<const T*>(p.w[t])[c]);
}

// What a thread copies and holds of a row, and how many rows at a time.
template <typename T, int P, int L, int K, bool GRAD>
struct Batch {
  static constexpr bool RING = P > 1;
  static constexpr int Q = GRAD ? 2 : 1;                                     // rows of x, and of dy
  static constexpr int COPIES = RING ? K * 2 * P * static_cast<int>(sizeof(T)) / 16 : 0;   // of 16 bytes of a row
  // Two rows at a time in 16 bits: forward four leave registers for two CTAs only (126 -> 141
  // us), backward one is too few (426 -> 515 us), but enough where pairs are gathered (of two
  // 119 -> 195).
  static constexpr int BYTES = GRAD && L != ANY ? 64 : 32;
  static constexpr int R = !RING ? (GRAD ? 1 : 2) : BYTES < Q * COPIES * 16 ? 1 : BYTES / (Q * COPIES * 16);
  static constexpr int SLOT = R * Q * COPIES * 16 * kThreads;                // a stage of the CTA
  static constexpr int RED = GRAD ? 512 * P * K * 4 : 0;                     // weight gradients of its groups
  static constexpr int TABLE = kStages * SLOT > RED ? kStages * SLOT : RED;  // frequencies, axes behind it
  static constexpr int SMEM = TABLE + rope::kMaxPairs * 9;
};

// Where a CTA is: an item (`tokens` tokens, `chunk` heads) and its next head.  All threads
// are at the same place, so that its registers and branches are the warp's; a group whose
// token is past the last one goes along without loads and stores.
struct Place {
  // item = rest * tiles + tile, rest = b * chunks + chunk: below 2^24 and 2^16 (one chunk) or
  // as few as the CTAs
  int tile, rest, b, h, h1;
};

// One CTA works on one tensor, on items of `tokens` tokens and `chunk` heads.  A row is
// K units in each of 2^lanes_log2 lanes.  FULL: every lane has its K units and all their
// pairs turn.
template <typename T, int P, int L, int K, bool GRAD, bool FULL>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(GRAD, P, L)) norm_rope_kernel(const __grid_constant__ NormParams p) {
  using B = Batch<T, P, L, K, GRAD>;
  constexpr int R = B::R, NP = (P + 1) / 2;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lanes = 1 << p.lanes_log2;
  const int group = threadIdx.x >> p.lanes_log2, lane = threadIdx.x & (lanes - 1);
  const int tokens = kThreads >> p.lanes_log2;
  int t = 0;
  while (t + 1 < p.n_tensors && static_cast<int>(blockIdx.x) >= p.cta0[t + 1]) ++t;
  const int tiles = (p.N + tokens - 1) / tokens;
  const int H = p.H[t], chunk = p.chunk[t], chunks = (H + chunk - 1) / chunk;
  const int rests = p.B * chunks, stride = p.cta0[t + 1] - p.cta0[t];
  const float inv_d = 1.f / p.d;

  // the pairs' frequencies and axes: lanes differ in them, which constant memory serves one
  // by one
  uint64_t* const freq = reinterpret_cast<uint64_t*>(smem + B::TABLE);
  uint8_t* const axis = smem + B::TABLE + rope::kMaxPairs * 8;
  for (int i = threadIdx.x; i < p.ang.n_pairs; i += kThreads) {
    freq[i] = p.ang.freq[i];
    axis[i] = p.ang.axis[i];
  }
  __syncthreads();

  Channels<P, L> ch[K];
  bool has[K];
  auto on = [&](int k) { return FULL || has[k]; };
  F2 wa[K][NP], wb[K][NP];                 // weights of the first and of the second elements
  F2 da[K][NP], db[K][NP];                 // and their gradients, over the rows of this thread
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int unit = lane + k * lanes;
    has[k] = unit < p.ang.units;
    ch[k].set(p.ang, on(k) ? unit : 0);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      auto w0 = [&](int j) { return on(k) && j < P ? weight_at<T>(p, t, ch[k].first(j)) : 0.f; };
      auto w1 = [&](int j) { return on(k) && j < P ? weight_at<T>(p, t, ch[k].second(j)) : 0.f; };
      wa[k][i] = pack2(w0(2 * i), w0(2 * i + 1));
      wb[k][i] = pack2(w1(2 * i), w1(2 * i + 1));
      da[k][i] = db[k][i] = 0;
    }
  }

  const int step_tile = stride % tiles, step_rest = stride / tiles;
  const int first = static_cast<int>(blockIdx.x) - p.cta0[t];
  auto settle = [&](Place& q) -> bool {    // false behind the last item
    q.b = chunks == 1 ? q.rest : q.rest / chunks;
    q.h = chunks == 1 ? 0 : (q.rest - q.b * chunks) * chunk;
    q.h1 = min(q.h + chunk, H);
    return q.rest < rests;
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
  Place cur;
  cur.rest = first / tiles;
  cur.tile = first - cur.rest * tiles;
  bool live = settle(cur);

  const int64_t xs = p.xs[t][1], os = p.os[t][1], gs = GRAD ? p.gs[t][1] : 0;
  auto row_of = [&](const void* base, const int64_t (&s)[3], const Place& q) {
    const int n = q.tile * tokens + group;
    return static_cast<const T*>(base) + q.b * s[0] + (n < p.N ? n : 0) * s[2] + q.h * s[1];
  };
  // A row of the ring, a group's own: its lanes copy 16 bytes each, row after row in whole
  // lines (half-split pieces would be parts of sectors), and read their units back.
  const int row_bytes = p.d * static_cast<int>(sizeof(T)), pitch = tokens * row_bytes;
  const int stage_bytes = R * B::Q * pitch;
  uint8_t* const mine = smem + group * row_bytes;
  int filled = 0, read = 0;                // the ring's next stages to copy to and to read
  auto advance = [&](int& at) {
    at += stage_bytes;
    if (at == kStages * stage_bytes) at = 0;
  };
  Place far = cur;                         // the next rows to copy
  bool more = live;
  const T *far_x = nullptr, *far_g = nullptr;
  bool far_ok = false;
  auto point = [&]() {
    far_ok = far.tile * tokens + group < p.N;
    far_x = row_of(p.x[t], p.xs[t], far);
    if constexpr (GRAD) far_g = row_of(p.g[t], p.gs[t], far);
  };
  auto fetch = [&]() {
    if (more) {
      const uint32_t to = smem_u32(mine + filled) + lane * 16;
      const uint8_t* from_x = reinterpret_cast<const uint8_t*>(far_x) + lane * 16;
      const uint8_t* from_g = reinterpret_cast<const uint8_t*>(far_g) + lane * 16;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (far.h + j < far.h1) {
#pragma unroll
          for (int m = 0; m < B::COPIES; ++m) {
            const int at = m * lanes * 16;
            if (far_ok && (FULL || lane * 16 + at < row_bytes)) {
              cp_async_16(to + j * B::Q * pitch + at, from_x + j * xs * static_cast<int64_t>(sizeof(T)) + at);
              if constexpr (GRAD)
                cp_async_16(to + (j * B::Q + 1) * pitch + at, from_g + j * gs * static_cast<int64_t>(sizeof(T)) + at);
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
    advance(filled);
  };
  if constexpr (B::RING) {
    if (more) point();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();
  }

  // Pair (u, v) -> (u c0 - v s0, u s1 + v c1): of the weighted row forward (the weights are
  // in the factors), of the gradient back (c0 = c1 = cos, s0 = s1 = -sin).  Of pairs that do
  // not turn (cos 1, sin 0) the partner is masked out: 0 times one that is not finite would
  // not be 0.
  F2 c0[K][NP], s0[K][NP], s1[K][NP], c1[K][NP];
  F2 turns[FULL ? 1 : K][NP];              // all ones for pairs that turn
  T* dst = nullptr;
  bool ok = false;
  auto begin = [&]() {                     // an item's angles and rows
    const int n = cur.tile * tokens + group;
    ok = n < p.N;
    // the token's coordinates, once for all its pairs
    int at[4] = {0, 0, 0, 0};
    if (p.ang.positions) {
      const int32_t* src = p.ang.positions + cur.b * p.ang.pos_batch + static_cast<int64_t>(ok ? n : 0) * p.ang.n_axes;
#pragma unroll
      for (int a = 0; a < 4; ++a)
        if (a < p.ang.n_axes) at[a] = __ldg(src + a);
    } else {
      int rest = ok ? n : 0;
#pragma unroll
      for (int a = 3; a > 0; --a)
        if (a < p.ang.n_axes) {
          // rest < 2^24: the quotient by the reciprocal is off by one at most
          const int e = p.ang.extent[a];
          int q = static_cast<int>(static_cast<float>(rest) * p.inv_extent[a]);
          q -= q * e > rest;
          q += rest - q * e >= e;
          at[a] = rest - q * e;
          rest = q;
        }
      at[0] = rest;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float cs[P], sn[P];
      const int pair0 = (lane + k * lanes) * P;
      const int turning = on(k) ? min(max(p.ang.n_pairs - pair0, 0), P) : 0;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
        if (FULL || i < turning) {
          const int a = axis[pair0 + i];
          const int64_t pos = a == 0 ? at[0] : a == 1 ? at[1] : a == 2 ? at[2] : at[3];
          // the angle's place on the circle in 2^-32 of a turn (rope.cu), half turns in [-1, 1)
          const uint64_t turn = static_cast<uint64_t>(pos) * freq[pair0 + i];
          sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn[i], &cs[i]);
          if (p.ang.inverse) sn[i] = -sn[i];
        }
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float hi = P == 1 ? 0.f : cs[(2 * i + 1) % P], ti = P == 1 ? 0.f : sn[(2 * i + 1) % P];
        const F2 c = pack2(cs[2 * i % P], hi), s = pack2(sn[2 * i % P], ti), minus = pack2(-1.f, -1.f);
        if constexpr (!FULL)
          turns[k][i] = (2 * i < turning ? 0xFFFFFFFFull : 0ull) | (2 * i + 1 < turning ? 0xFFFFFFFFull << 32 : 0ull);
        if constexpr (GRAD) {
          c0[k][i] = c;
          s0[k][i] = s;                    // u cos + v sin
          s1[k][i] = mul2(s, minus);       // v cos - u sin
        } else {
          c0[k][i] = mul2(c, wa[k][i]);
          s0[k][i] = mul2(mul2(s, minus), wb[k][i]);
          s1[k][i] = mul2(s, wa[k][i]);
          c1[k][i] = mul2(c, wb[k][i]);
        }
      }
    }
    dst = const_cast<T*>(row_of(p.out[t], p.os[t], cur));
  };
  // the first and second elements of two pairs, turned
  auto turn = [&](int k, int i, F2 u, F2 v, F2& y, F2& z) {
    const F2 u1 = FULL ? u : u & turns[k][i], v1 = FULL ? v : v & turns[k][i];
    y = fma2(v1, s0[k][i], mul2(u, c0[k][i]));
    z = fma2(u1, s1[k][i], mul2(v, GRAD ? c0[k][i] : c1[k][i]));
  };
  if (live) begin();
  while (live) {
    UnitOf<T, P, L> u[R][K], v[GRAD ? R : 1][K];
    const int used = read;                 // the stage of these rows
    if constexpr (B::RING) {
      fetch();
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();                        // the copies of the lanes that share a row
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const T* x = reinterpret_cast<const T*>(mine + read + j * B::Q * pitch);
        const T* g = GRAD ? reinterpret_cast<const T*>(mine + read + (j * B::Q + 1) * pitch) : nullptr;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          gather<T, P, L>(u[j][k], x, ch[k]);
          if constexpr (GRAD) gather<T, P, L>(v[j][k], g, ch[k]);
        }
      }
      advance(read);
    } else {
      const T* src = row_of(p.x[t], p.xs[t], cur);
      const T* grd = GRAD ? row_of(p.g[t], p.gs[t], cur) : nullptr;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (cur.h + j < cur.h1 && ok) {
#pragma unroll
          for (int k = 0; k < K; ++k)
            if (on(k)) {
              gather<T, P, L>(u[j][k], src + j * xs, ch[k]);
              if constexpr (GRAD) gather<T, P, L>(v[j][k], grd + j * gs, ch[k]);
            }
        }
    }
    float ss[R], sp[R];
    F2 ga[GRAD ? R : 1][K][NP], gb[GRAD ? R : 1][K][NP];     // R^T dy
#pragma unroll
    for (int j = 0; j < R; ++j) {
      F2 q0 = 0, q1 = 0, t0 = 0, t1 = 0;
      if (cur.h + j < cur.h1) {
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (on(k)) {
            F2 a[NP], c[NP];
            get(u[j][k], a, c);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              q0 = fma2(a[i], a[i], q0);
              q1 = fma2(c[i], c[i], q1);
            }
            if constexpr (GRAD) {
              F2 e[NP], f[NP];
              get(v[j][k], e, f);
#pragma unroll
              for (int i = 0; i < NP; ++i) {
                turn(k, i, e[i], f[i], ga[j][k][i], gb[j][k][i]);
                t0 = fma2(mul2(ga[j][k][i], wa[k][i]), a[i], t0);
                t1 = fma2(mul2(gb[j][k][i], wb[k][i]), c[i], t1);
              }
            }
          }
      }
      const float2 x0 = unpack2(q0), x1 = unpack2(q1), y0 = unpack2(t0), y1 = unpack2(t1);
      ss[j] = (x0.x + x0.y) + (x1.x + x1.y);
      sp[j] = (y0.x + y0.y) + (y1.x + y1.y);
    }
    for (int m = lanes >> 1; m; m >>= 1) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        ss[j] += __shfl_xor_sync(0xFFFFFFFFu, ss[j], m);
        if constexpr (GRAD) sp[j] += __shfl_xor_sync(0xFFFFFFFFu, sp[j], m);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (cur.h + j < cur.h1 && ok) {
        const float r = rsqrtf(fmaf(ss[j], inv_d, p.eps));
        // r one factor at a time: r^2 alone is beyond fp32 where a row's mean square and eps are
        // small, r S / d is of the size of g o w
        const float off = GRAD ? -(r * sp[j] * inv_d * r) : 0.f;
        const F2 r2 = pack2(r, r), off2 = pack2(off, off);
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (on(k)) {
            F2 a[NP], c[NP], y[NP], z[NP];
            get(u[j][k], a, c);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              if constexpr (GRAD) {
                y[i] = mul2(r2, fma2(a[i], off2, mul2(ga[j][k][i], wa[k][i])));
                z[i] = mul2(r2, fma2(c[i], off2, mul2(gb[j][k][i], wb[k][i])));
                da[k][i] = fma2(ga[j][k][i], mul2(a[i], r2), da[k][i]);
                db[k][i] = fma2(gb[j][k][i], mul2(c[i], r2), db[k][i]);
              } else {
                // normed first: a large row's products with the weights stay finite
                turn(k, i, mul2(a[i], r2), mul2(c[i], r2), y[i], z[i]);
              }
            }
            put(u[j][k], y, z);
            scatter<T, P, L>(u[j][k], L == ANY ? reinterpret_cast<T*>(mine + used + j * B::Q * pitch) : dst + j * os, ch[k]);
          }
      }
    }
    if constexpr (L == ANY) {
      // the rows lie whole in the ring again: out as they came in (a lane's next copy goes to
      // where it has read itself)
      __syncwarp();
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (cur.h + j < cur.h1 && ok) {
#pragma unroll
          for (int m = 0; m < B::COPIES; ++m) {
            const int at = (lane + m * lanes) * 16;
            if (FULL || at < row_bytes)
              *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(dst + j * os) + at) =
                  *reinterpret_cast<const uint4*>(mine + used + j * B::Q * pitch + at);
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
      if (on(k)) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 x = unpack2(da[k][i / 2]), y = unpack2(db[k][i / 2]);
          red[group * p.d + ch[k].first(i)] = i % 2 ? x.y : x.x;
          red[group * p.d + ch[k].second(i)] = i % 2 ? y.y : y.x;
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

template <typename T, int P, int L, int K, bool GRAD, bool FULL>
tsr_status launch_one(unsigned ctas, const NormParams& p, cudaStream_t st) {
  constexpr int smem = Batch<T, P, L, K, GRAD>::SMEM;
  auto kern = norm_rope_kernel<T, P, L, K, GRAD, FULL>;
  if constexpr (smem > 48 * 1024) {
    static OncePerDevice once;
    int dev = 0;
    TSR_CUDA(cudaGetDevice(&dev));
    if (tsr_status e = allow_smem(kern, smem, dev, once)) return e;
  }
  kern<<<ctas, kThreads, smem, st>>>(p);
  TSR_CUDA(cudaGetLastError());
  return TSR_OK;
}

// Pairs per unit, how they lie, and units of a row in each of its lanes.
struct Shape {
  int P, L, K;
};

template <bool GRAD>
tsr_status launch(const NormParams& p, int dtype, const Shape& s, cudaStream_t st) {
  const unsigned ctas = static_cast<unsigned>(p.cta0[p.n_tensors]);
  const bool full = s.P > 1 && p.ang.units == s.K << p.lanes_log2 && p.ang.n_pairs == p.ang.units * s.P;
#define TSR_NORM(T, P_, L_, K_)                                                                    \
  if (s.P == P_ && s.L == L_ && s.K == K_) {                                                       \
    if constexpr (P_ > 1) {                                                                        \
      if (full) return launch_one<T, P_, L_, K_, GRAD, true>(ctas, p, st);                         \
    }                                                                                              \
    return launch_one<T, P_, L_, K_, GRAD, false>(ctas, p, st);                                    \
  }
#define TSR_NORM_16(T)      \
  TSR_NORM(T, 4, NEAR, 1)   \
  TSR_NORM(T, 4, HALVES, 1) \
  TSR_NORM(T, 4, ANY, 1)    \
  TSR_NORM(T, 1, HALVES, 4)
  if (dtype == TSR_DTYPE_BF16) {
    TSR_NORM_16(__nv_bfloat16)
  } else if (dtype == TSR_DTYPE_F16) {
    TSR_NORM_16(__half)
  } else {
    TSR_NORM(float, 2, NEAR, 1)
    TSR_NORM(float, 2, NEAR, 2)
    TSR_NORM(float, 4, HALVES, 1)
    TSR_NORM(float, 2, ANY, 1)
    TSR_NORM(float, 2, ANY, 2)
    TSR_NORM(float, 1, HALVES, 4)
  }
#undef TSR_NORM_16
#undef TSR_NORM
  return fail(TSR_ERR_INTERNAL, "no norm kernel for this layout");
}

// The forward's kernels (norm_rope.cu) and the backward's (norm_rope_bwd.cu) are compiled apart.
extern template tsr_status launch<false>(const NormParams&, int, const Shape&, cudaStream_t);
extern template tsr_status launch<true>(const NormParams&, int, const Shape&, cudaStream_t);

}  // namespace norm

}  // namespace tsr
