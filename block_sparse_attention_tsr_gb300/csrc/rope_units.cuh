// rope_units.cuh -- what the kernels that rotate heads share (rope.cu, norm_rope.cu):
// pieces of a head's row in registers, the angles of a token, and the host's choice of
// pieces.  The mathematics of the angles is described in rope.cu.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "internal.h"

namespace tsr {

namespace rope {

constexpr int kMaxPairs = 128;     // d <= 256
constexpr int kMaxTensors = 4;

// Angles of every token and pair, and where a unit's channels lie.
struct Angles {
  const int32_t* positions;
  int64_t pos_batch;              // elements between batches' positions (0: shared)
  int32_t n_axes, n_pairs, units, inverse;
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

// Cosines and sines of the pairs [P * unit, P * unit + P) of token n of batch b; pairs from
// `turning` on (their number is returned) do not turn.
template <int P>
__device__ __forceinline__ int angles_of(const Angles& p, int64_t b, int64_t n, int unit, float (&cs)[P],
                                         float (&sn)[P]) {
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
  return turning;
}

// Host: fills `p` for rows whose pointers and strides (in bytes) are or-ed into `bits`;
// returns the pairs per unit, from the largest piece that every pointer, stride and, for
// half-split pairs, half width allows.
inline int fill_angles(const tsr_rope_desc& d, uint64_t bits, Angles& p) {
  const size_t es = d.dtype == TSR_DTYPE_F32 ? 4 : 2;
  p.n_axes = d.n_axes;
  p.positions = d.positions;
  p.pos_batch = d.positions_per_batch ? static_cast<int64_t>(d.N) * d.n_axes : 0;
  p.inverse = d.inverse != 0;
  // The frequencies of the thread's last call are kept: 64 powers take 3 us.
  struct Table {
    double theta = 0.0;
    int32_t n_axes = 0, axis_dim[4];
    uint64_t freq[kMaxPairs];
    uint8_t axis[kMaxPairs];
  };
  static thread_local Table last;
  bool same = last.theta == d.theta && last.n_axes == d.n_axes;
  for (int a = 0; a < d.n_axes; ++a) same = same && last.axis_dim[a] == d.axis_dim[a];
  int32_t at = 0;
  for (int a = 0; a < d.n_axes; ++a) {
    p.extent[a] = d.positions ? 1 : d.grid[a];
    for (int j = 0; !same && j < d.axis_dim[a] / 2; ++j) {
      const double turns = std::pow(d.theta, -2.0 * j / d.axis_dim[a]) / 6.283185307179586476925286766559;
      // the fraction of a turn, as 2^64 fixed point (whole turns drop out)
      const double frac = turns - std::floor(turns);
      const double scaled = frac * 18446744073709551616.0;
      last.freq[at / 2 + j] = scaled >= 18446744073709551615.0 ? 0u : static_cast<uint64_t>(scaled + 0.5);
      last.axis[at / 2 + j] = static_cast<uint8_t>(a);
    }
    last.axis_dim[a] = d.axis_dim[a];
    at += d.axis_dim[a];
  }
  last.theta = d.theta;
  last.n_axes = d.n_axes;
  memcpy(p.freq, last.freq, sizeof(uint64_t) * (at / 2));
  memcpy(p.axis, last.axis, at / 2);
  p.n_pairs = at / 2;
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
  return P;
}

}  // namespace rope

}  // namespace tsr
