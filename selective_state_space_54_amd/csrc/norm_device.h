// A row's values in 16-byte pieces, widened and rounded: what the norms' kernels share (gfx950).
#pragma once

#include "scan_device.h"

namespace mssm {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T>
constexpr int kPer = 16 / sizeof(T);   // values in a piece

template <int N>
__device__ __forceinline__ void load_param(const float* p, int64_t c, int64_t D, float (&v)[N]) {
  if (c + N <= D) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      f32x4 u;
      __builtin_memcpy(&u, p + c + j, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j + i] = u[i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = c + j < D ? p[c + j] : 0.0f;
  }
}

__device__ __forceinline__ float narrow(float v, float) { return v; }
__device__ __forceinline__ uint16_t narrow(float v, uint16_t) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

__device__ __forceinline__ void widen(const uint4& u, float (&v)[4]) {
  v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y);
  v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void widen(const uint4& u, float (&v)[8]) {
  v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
  v[4] = __uint_as_float(u.z << 16), v[5] = __uint_as_float(u.z & 0xffff0000u);
  v[6] = __uint_as_float(u.w << 16), v[7] = __uint_as_float(u.w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 v;
  v[0] = static_cast<__bf16>(a);
  v[1] = static_cast<__bf16>(b);
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint4 packed(const float (&v)[4]) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                    __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 packed(const float (&v)[8]) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

}  // namespace mssm
