// Device-side pieces of the operators around a gated recurrence (gfx950): a lane's adjacent
// channels in memory, the sigmoid, and the decay of the gated recurrence.
#pragma once

#include "scan_device.h"
#include "sequences.h"

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
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = 0u;
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
};

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-v * kLog2e));
}
__device__ __forceinline__ float sqrt_(float v) { return __builtin_amdgcn_sqrtf(v); }
__device__ __forceinline__ float rsqrt_(float v) { return __builtin_amdgcn_rsqf(v); }

// a = exp(A s) and m2 = 1 - a^2 with s = sigmoid(r), A <= 0.
//
// A state that remembers thousands of tokens has a within 1e-3 of 1, where 1 - a^2 cancels and
// where a bias of a's last place (the exponential's own rounding) adds up over those tokens.
// So e = exp(A s) - 1 comes from its series down to A s = -1/4 (the next term is 2e-9 of it) and
// a = 1 + e is rounded once; below, decays forget within a few tokens and the
// exponential's last place is enough.  (dA of 4 x 8192 x 2048 bf16, whose terms
// cancel to 1 in 100: off by 1e-5 of its norm with the exponential alone.)
struct Decay {
  float s, a, m2;
};
constexpr float kSeries = -0.25f;

__device__ __forceinline__ Decay decay_of(float A, float r) {
  Decay d;
  d.s = sigmoid(r);
  const float u = A * d.s;
  float e = __builtin_fmaf(u, 1.0f / 5040.0f, 1.0f / 720.0f);
  e = __builtin_fmaf(e, u, 1.0f / 120.0f);
  e = __builtin_fmaf(e, u, 1.0f / 24.0f);
  e = __builtin_fmaf(e, u, 1.0f / 6.0f);
  e = __builtin_fmaf(e, u, 0.5f);
  e = __builtin_fmaf(e, u, 1.0f) * u;
  const float b = fast_exp2(u * kLog2e);
  d.a = u > kSeries ? 1.0f + e : b;
  d.m2 = u > kSeries ? -e * (2.0f + e) : __builtin_fmaf(-b, b, 1.0f);
  return d;
}

}  // namespace mssm
