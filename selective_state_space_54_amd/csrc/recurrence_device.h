// Device-side pieces of the operators around a gated recurrence (gfx950): a lane's adjacent
// channels in memory, the sigmoid, and the decay of the gated recurrence.
#pragma once

#include "scan_device.h"
#include "sequences.h"

// Fused multiply-adds are written out: every kernel forms the same numbers, bit for bit.
#pragma clang fp contract(off)

namespace mssm {

// V adjacent values as they lie in memory (any element-aligned address).
template <typename T, int V>
struct Raw {
  static constexpr int kWords = (sizeof(T) * V + 3) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (sizeof(T) * V < 4) w[0] = *p;
    else __builtin_memcpy(w, p, sizeof(w));
  }
  // At `voff` bytes of the lane's plus `soff` of the wavefront's own in a buffer.
  __device__ __forceinline__ void load(buf_t r, int voff, int soff) {
    if constexpr (sizeof(T) * V == 2) {
      w[0] = __builtin_amdgcn_raw_buffer_load_b16(r, voff, soff, 0);
    } else if constexpr (sizeof(T) * V == 4) {
      w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
    } else {
      static_assert(sizeof(T) * V == 8, "two, four or eight bytes");
      const u32x2 u = __builtin_amdgcn_raw_buffer_load_b64(r, voff, soff, 0);
      w[0] = u.x, w[1] = u.y;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = 0u;
  }
  // Here the values are in registers as they were loaded.
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) asm volatile("" : "+v"(w[k]));
  }
  __device__ __forceinline__ float get(int v) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[v]);
    else return __uint_as_float(v & 1 ? w[v / 2] & 0xffff0000u : w[v / 2] << 16);
  }
  // The values rounded to T once, to nearest even.
  static __device__ __forceinline__ void store(T* p, const float (&f)[V]) {
    if constexpr (sizeof(T) == 4) {
      __builtin_memcpy(p, f, sizeof(f));
    } else {
      __bf16 e[V];
#pragma unroll
      for (int v = 0; v < V; ++v) e[v] = static_cast<__bf16>(f[v]);
      __builtin_memcpy(p, e, sizeof(e));
    }
  }
  static __device__ __forceinline__ void store(buf_t r, int voff, int soff, const float (&f)[V]) {
    T e[V];
    store(e, f);
    if constexpr (sizeof(e) == 2) {
      unsigned short u;
      __builtin_memcpy(&u, e, 2);
      __builtin_amdgcn_raw_buffer_store_b16(u, r, voff, soff, 0);
    } else if constexpr (sizeof(e) == 4) {
      uint32_t u;
      __builtin_memcpy(&u, e, 4);
      __builtin_amdgcn_raw_buffer_store_b32(u, r, voff, soff, 0);
    } else {
      // (no more: nothing keeps the instruction after a store of more than eight bytes with a
      // wave-uniform offset from writing the registers it has not read yet)
      static_assert(sizeof(e) == 8, "two, four or eight bytes");
      u32x2 u;
      __builtin_memcpy(&u, e, 8);
      __builtin_amdgcn_raw_buffer_store_b64(u, r, voff, soff, 0);
    }
  }
};

// S rows of a tensor from token t0 on as a buffer: addresses are a lane's own part and a wave-uniform
// one for the row.  step: bytes from row to row; bytes: of a row.
template <int S>
__device__ __forceinline__ buf_t rows_from(const void* base, int64_t t0, int64_t step,
                                           int64_t bytes) {
  return make_buf(static_cast<const char*>(base) + t0 * step,
                  static_cast<uint32_t>((S - 1) * step + bytes));
}

// S rows from token t0 on, each lane its V channels; rows past the last token repeat it.
template <typename T, int V, int S>
__device__ __forceinline__ void load_rows(const void* base, int64_t row, int64_t D, int64_t t0,
                                          int64_t tokens, int c, Raw<T, V> (&v)[S]) {
  const int64_t step = row * static_cast<int64_t>(sizeof(T));
  const int64_t left = tokens - t0;
  const buf_t r = rows_from<S>(base, left > 0 ? t0 : tokens - 1, step, D * sizeof(T));
  const int last = left > S ? S - 1 : left > 0 ? static_cast<int>(left) - 1 : 0;
#pragma unroll
  for (int s = 0; s < S; ++s)
    v[s].load(r, c * static_cast<int>(sizeof(T)), (s < last ? s : last) * static_cast<int>(step));
}

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-v * kLog2e));
}

// s = sigmoid(v) with 1 - s, for a slope s (1 - s), as one number.  Past v = 0, where 1 - s cancels
// (at 10 only ten of its bits are left), the number is -(1 - s) from the same exponential, e s with
// e = exp(-v) < 1; elsewhere it is s.  The sign bit says which, of a zero too.  (The gradient of
// 4 x 8192 x 2048 bf16: 280 us, 270 with slopes from s alone.)
struct Gate {
  float q;
  __device__ __forceinline__ float make(float v) {     // returns s
    const float e = fast_exp2(-v * kLog2e), s = __builtin_amdgcn_rcpf(1.0f + e);
    q = e < 1.0f ? -(e * s) : s;
    asm volatile("" : "+v"(q));       // (as one number from here on: s and 1 - s both kept would spill)
    return s;
  }
  __device__ __forceinline__ bool open() const { return __float_as_int(q) < 0; }
  __device__ __forceinline__ float value() const { return open() ? 1.0f - fabsf(q) : fabsf(q); }
  __device__ __forceinline__ float rest() const { return open() ? fabsf(q) : 1.0f - fabsf(q); }
};

__device__ __forceinline__ float sqrt_(float v) { return __builtin_amdgcn_sqrtf(v); }

// The decay a = exp(u), u = A s <= 0, as one number q that keeps both a and 1 - a^2.
//
// A state that remembers thousands of tokens has a within 1e-3 of 1, where 1 - a^2 cancels and
// where a bias of a's last place (the exponential's own rounding) adds up over those tokens.
// So down to u = -1/4 q is e = exp(u) - 1 <= 0 from u (1 + u p(u)), p of degree 3 the closest there
// (7.2e-9 of e with its rounded coefficients, 1e-7 as float32 evaluates it; the series needs two terms
// more): a = 1 + e
// is rounded once, 1 - a^2 = -e (2 + e).  Below, q is a itself, positive; decays forget within a
// few tokens and the exponential's last place is enough.  (dA of 4 x 8192 x 2048 bf16, whose
// terms cancel to 1 in 100: off by 1e-5 of its norm with the exponential alone.)
// kNear: u > -1/4 everywhere.  With rates from -exp(-4) to -exp(1.5), 131072 x 2560 bf16 takes 628 us where
// they are in order (half of the wavefronts have one below -1/4) and 650 mixed (all have), 630 without;
// the training pass 4 x 8192 x 2048 449, 456 and 439.
constexpr float kSeries = -0.25f;

template <bool kNear>
__device__ __forceinline__ float decay_of(float u) {
  float e = __builtin_fmaf(u, 0.0075347293f, 0.041502327f);
  e = __builtin_fmaf(e, u, 0.16665322f);
  e = __builtin_fmaf(e, u, 0.49999964f);
  e = __builtin_fmaf(e, u, 1.0f) * u;
  if constexpr (!kNear) {
    // (a decay below the normal numbers stays positive; NaN goes on as it is)
    const float a = fast_exp2(u * kLog2e);
    e = u <= kSeries ? (a > 1.2e-38f ? a : 1.2e-38f) : e;
  }
  return e;
}
template <bool kNear>
__device__ __forceinline__ float decay(float q) {
  return kNear || !(q > 0.0f) ? 1.0f + q : q;
}
template <bool kNear>
__device__ __forceinline__ float one_minus_square(float q) {
  return kNear || !(q > 0.0f) ? -q * (2.0f + q) : __builtin_fmaf(-q, q, 1.0f);
}

}  // namespace mssm
