// Layer norm over rows of D values, forward and backward (gfx950).
//
//   t = x + residual (rounded to the type; t = x without a residual)
//   y = (t - mean) rstd w + b,    mean, var over the row, rstd = 1 / sqrt(var + eps)
// With xhat = (t - mean) rstd and the means taken over the row,
//   dt = rstd (w dy - mean(w dy) - xhat mean(w dy xhat))  (+ the gradient that
//        reaches t itself, when t is also passed on)
//   dw = sum over rows of dy xhat,   db = sum over rows of dy.
//
// Both are bound by memory: every tensor is read or written once.  A row is
// held in registers by TPR threads (8 to 64 lanes of a wavefront, or a whole
// block of 256 or 1024), VPT 16-byte pieces each, so the variance is the mean
// square of the centred values (nothing cancels) at no second read.  Sums are
// float32 butterflies.  Pieces are read at any alignment (global memory allows
// it), so odd D and unaligned tensors take the same path; only a row's last,
// partial piece goes element by element.
//
// The gradients of w and b: a block runs over many rows and keeps its columns'
// sums in registers; at the end it writes one row of partial sums, and a second
// kernel adds the blocks' rows, all in a fixed order.
#include "mssm_internal.h"
#include "scan_device.h"

namespace mssm {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T>
constexpr int kPer = 16 / sizeof(T);   // values in a piece

// Piece at column c of a row: values past D are zero.
template <typename T>
__device__ __forceinline__ void load_piece(const T* row, int64_t c, int64_t D,
                                           float (&v)[kPer<T>]) {
  if (c + kPer<T> <= D) {
    T e[kPer<T>];
    __builtin_memcpy(e, row + c, 16);
#pragma unroll
    for (int j = 0; j < kPer<T>; ++j) v[j] = to_float(e[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kPer<T>; ++j) v[j] = c + j < D ? to_float(row[c + j]) : 0.0f;
  }
}
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

template <typename T>
__device__ __forceinline__ void store_piece(T* row, int64_t c, int64_t D,
                                            const float (&v)[kPer<T>]) {
  T e[kPer<T>];
#pragma unroll
  for (int j = 0; j < kPer<T>; ++j) e[j] = narrow(v[j], T());
  if (c + kPer<T> <= D) {
    __builtin_memcpy(row + c, e, 16);
  } else {
#pragma unroll
    for (int j = 0; j < kPer<T>; ++j)
      if (c + j < D) row[c + j] = e[j];
  }
}

// Sum over the TPR threads of a row; every one of them gets it.  `red` has two
// floats per wavefront; `flip` alternates so that one barrier per sum is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red, int& flip) {
#pragma unroll
  for (int o = (TPR < 64 ? TPR : 64) / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* m = red + flip * W;
    flip ^= 1;
    if ((threadIdx.x & 63) == 0) m[threadIdx.x >> 6] = v;
    block_sync();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += m[w];
  }
  return v;
}

template <typename T, int TPR, int VPT>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void layer_norm_kernel(NormArgs a) {
  constexpr int N = kPer<T>;
  constexpr int kBlock = TPR > 256 ? TPR : 256;
  __shared__ float red[TPR > 64 ? 2 * TPR / 64 : 1];
  int flip = 0;
  const int64_t r = int64_t(blockIdx.x) * (kBlock / TPR) + threadIdx.x / TPR;
  if (r >= a.rows) return;         // whole rows of threads; with TPR > 64 whole blocks
  const int lane = threadIdx.x % TPR;
  const int64_t D = a.D;
  const T* x = static_cast<const T*>(a.x) + r * D;
  float v[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i) load_piece<T>(x, int64_t(lane + TPR * i) * N, D, v[i]);
  if (a.residual) {
    const T* q = static_cast<const T*>(a.residual) + r * D;
    float u[VPT][N];
#pragma unroll
    for (int i = 0; i < VPT; ++i) load_piece<T>(q, int64_t(lane + TPR * i) * N, D, u[i]);
    T* t = static_cast<T*>(a.sum) + r * D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[i][j] = to_float(narrow(v[i][j] + u[i][j], T()));
      store_piece<T>(t, int64_t(lane + TPR * i) * N, D, v[i]);
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) s += v[i][j];
  const float mean = row_sum<TPR>(s, red, flip) / static_cast<float>(D);
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int64_t c = int64_t(lane + TPR * i) * N;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      v[i][j] = c + j < D ? v[i][j] - mean : 0.0f;
      s = __builtin_fmaf(v[i][j], v[i][j], s);
    }
  }
  const float var = row_sum<TPR>(s, red, flip) / static_cast<float>(D);
  const float rstd = 1.0f / sqrtf(var + a.eps);
  if (lane == 0 && a.mean) {
    a.mean[r] = mean;
    a.rstd[r] = rstd;
  }
  T* y = static_cast<T*>(a.y) + r * D;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int64_t c = int64_t(lane + TPR * i) * N;
    float w[N], b[N];
    load_param<N>(a.weight, c, D, w);
    if (a.bias) {
      load_param<N>(a.bias, c, D, b);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) b[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) v[i][j] = __builtin_fmaf(v[i][j] * rstd, w[j], b[j]);
    if (c < D) store_piece<T>(y, c, D, v[i]);
  }
}

// part: [gridDim.x, 2, D]: the block's sums of dy xhat and of dy.
template <typename T, int TPR, int VPT>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void layer_norm_bwd_kernel(NormBwdArgs a,
                                                                               float* part) {
  constexpr int N = kPer<T>;
  constexpr int kBlock = TPR > 256 ? TPR : 256;
  constexpr int kRows = kBlock / TPR;                  // rows at a time
  __shared__ float red[TPR > 64 ? 2 * TPR / 64 : 1];
  __shared__ float cols[TPR < 256 ? kBlock * N : 1];
  int flip = 0;
  const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int64_t D = a.D;
  const float inv = 1.0f / static_cast<float>(D);
  float dw[VPT][N], db[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) dw[i][j] = db[i][j] = 0.0f;
  for (int64_t r = int64_t(blockIdx.x) * kRows + group; r < a.rows;
       r += int64_t(gridDim.x) * kRows) {
    const float mean = a.mean[r], rstd = a.rstd[r];
    float g[VPT][N], v[VPT][N];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t c = int64_t(lane + TPR * i) * N;
      load_piece<T>(static_cast<const T*>(a.dy) + r * D, c, D, g[i]);
      load_piece<T>(static_cast<const T*>(a.x) + r * D, c, D, v[i]);
    }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t c = int64_t(lane + TPR * i) * N;
      float w[N];
      load_param<N>(a.weight, c, D, w);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float xh = (v[i][j] - mean) * rstd;      // past D: dy and w are zero
        dw[i][j] = __builtin_fmaf(g[i][j], xh, dw[i][j]);
        db[i][j] += g[i][j];
        v[i][j] = xh;
        g[i][j] *= w[j];
        s1 += g[i][j];
        s2 = __builtin_fmaf(g[i][j], xh, s2);
      }
    }
    const float m1 = row_sum<TPR>(s1, red, flip) * inv;
    const float m2 = row_sum<TPR>(s2, red, flip) * inv;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t c = int64_t(lane + TPR * i) * N;
      float out[N];
#pragma unroll
      for (int j = 0; j < N; ++j) out[j] = rstd * (g[i][j] - __builtin_fmaf(v[i][j], m2, m1));
      if (a.dsum) {
        float e[N];
        load_piece<T>(static_cast<const T*>(a.dsum) + r * D, c, D, e);
#pragma unroll
        for (int j = 0; j < N; ++j) out[j] += e[j];
      }
      if (c < D) store_piece<T>(static_cast<T*>(a.dx) + r * D, c, D, out);
    }
  }
  float* dst = part + int64_t(blockIdx.x) * 2 * D;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float(&acc)[N] = k ? db[i] : dw[i];
      if constexpr (TPR >= 256) {
        const int64_t c = int64_t(lane + TPR * i) * N;
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (c + j < D) dst[k * D + c + j] = acc[j];
      } else {
        // the block's rows of threads hold the same columns: add them in order
        block_sync();
#pragma unroll
        for (int j = 0; j < N; ++j) cols[(group * TPR + lane) * N + j] = acc[j];
        block_sync();
        for (int q = threadIdx.x; q < TPR * N; q += kBlock) {
          float t = 0.0f;
          for (int w = 0; w < kRows; ++w) t += cols[w * TPR * N + q];
          const int64_t c = int64_t(TPR) * i * N + q;
          if (c < D) dst[k * D + c] = t;
        }
      }
    }
  }
}

// out[c] = the sum of `blocks` rows of part, for the 2 D columns of [dw | db].
// A block takes 64 columns, 16 threads of four columns by 16 rows at a time.
__global__ __launch_bounds__(256) void layer_norm_sum_kernel(const float* __restrict__ part,
                                                             int blocks, int64_t D, float* dw,
                                                             float* db) {
  __shared__ float m[16][64];
  const int64_t c0 = int64_t(blockIdx.x) * 64;
  const int64_t width = 2 * D;
  const int q = threadIdx.x % 16, row = threadIdx.x / 16;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t c = c0 + 4 * q;
#pragma unroll 4
  for (int b = row; b < blocks; b += 16) {
    float u[4];
    load_param<4>(part + int64_t(b) * width, c, width, u);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += u[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) m[row][4 * q + j] = s[j];
  block_sync();
  if (threadIdx.x < 64) {
    const int64_t col = c0 + threadIdx.x;
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) t += m[r][threadIdx.x];
    if (col < D) dw[col] = t;
    else if (col < width && db) db[col - D] = t;
  }
}

__global__ __launch_bounds__(256) void fill_zero_kernel(float* p, int64_t n) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// Calls f.template operator()<TPR, VPT>() for the threads per row and pieces
// per thread that hold D values: a part of a wavefront for the shortest rows,
// one wavefront up to eight pieces a lane, then a block of 256, then of 1024
// with at most 32 values a thread.
template <typename T, typename F>
hipError_t dispatch_row(int64_t D, F f) {
  const int64_t pieces = (D + kPer<T> - 1) / kPer<T>;
  if (pieces <= 8) return f.template operator()<8, 1>();
  if (pieces <= 16) return f.template operator()<16, 1>();
  if (pieces <= 32) return f.template operator()<32, 1>();
  switch ((pieces + 63) / 64) {
    case 1: return f.template operator()<64, 1>();
    case 2: return f.template operator()<64, 2>();
    case 3: return f.template operator()<64, 3>();
    case 4: return f.template operator()<64, 4>();
    case 5: return f.template operator()<64, 5>();
    case 6: return f.template operator()<64, 6>();
    case 7: return f.template operator()<64, 7>();
    case 8: return f.template operator()<64, 8>();
    default: break;
  }
  switch ((pieces + 255) / 256) {
    case 3: return f.template operator()<256, 3>();
    case 4: return f.template operator()<256, 4>();
    case 5: return f.template operator()<256, 5>();
    case 6: return f.template operator()<256, 6>();
    case 7: return f.template operator()<256, 7>();
    case 8: return f.template operator()<256, 8>();
    default: break;
  }
  switch ((pieces + 1023) / 1024) {
    case 3: return f.template operator()<1024, 3>();
    case 4: return f.template operator()<1024, 4>();
    default: break;
  }
  if constexpr (sizeof(T) == 4) {
    switch ((pieces + 1023) / 1024) {
      case 5: return f.template operator()<1024, 5>();
      case 6: return f.template operator()<1024, 6>();
      case 7: return f.template operator()<1024, 7>();
      case 8: return f.template operator()<1024, 8>();
      default: break;
    }
  }
  return hipErrorInvalidValue;
}

template <typename T>
struct RunNorm {
  const NormArgs& a;
  hipStream_t stream;
  template <int TPR, int VPT>
  hipError_t operator()() const {
    constexpr int kBlock = TPR > 256 ? TPR : 256;
    const int64_t per = kBlock / TPR;
    hipLaunchKernelGGL((layer_norm_kernel<T, TPR, VPT>),
                       dim3(static_cast<uint32_t>((a.rows + per - 1) / per)), dim3(kBlock), 0,
                       stream, a);
    return hipGetLastError();
  }
};

// Blocks of the backward pass: enough to fill the compute units, and at most
// one for each set of rows.
template <typename T>
struct NormBlocks {
  int64_t rows;
  int64_t* blocks;
  template <int TPR, int VPT>
  hipError_t operator()() const {
    const int64_t per = TPR >= 256 ? 1 : 256 / TPR;
    const int64_t most = TPR > 256 ? 256 : 512;
    const int64_t need = (rows + per - 1) / per;
    *blocks = need < most ? need : most;
    return hipSuccess;
  }
};

template <typename T>
struct RunNormBwd {
  const NormBwdArgs& a;
  float* part;
  int64_t blocks;
  hipStream_t stream;
  template <int TPR, int VPT>
  hipError_t operator()() const {
    constexpr int kBlock = TPR > 256 ? TPR : 256;
    hipLaunchKernelGGL((layer_norm_bwd_kernel<T, TPR, VPT>), dim3(static_cast<uint32_t>(blocks)),
                       dim3(kBlock), 0, stream, a, part);
    return hipGetLastError();
  }
};

int64_t norm_blocks(int64_t rows, int64_t D, mssm_dtype dtype) {
  int64_t blocks = 0;
  if (dtype == MSSM_BFLOAT16) dispatch_row<uint16_t>(D, NormBlocks<uint16_t>{rows, &blocks});
  else dispatch_row<float>(D, NormBlocks<float>{rows, &blocks});
  return blocks;
}

}  // namespace

bool norm_size_supported(int64_t D) { return D >= 0 && D <= 32768; }

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  if (a.dtype == MSSM_BFLOAT16) return dispatch_row<uint16_t>(a.D, RunNorm<uint16_t>{a, stream});
  return dispatch_row<float>(a.D, RunNorm<float>{a, stream});
}

size_t norm_bwd_workspace(int64_t rows, int64_t D, mssm_dtype dtype) {
  return static_cast<size_t>(norm_blocks(rows, D, dtype)) * 2 * D * sizeof(float);
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, void* ws, hipStream_t stream) {
  if (a.rows == 0) {
    const dim3 g(static_cast<uint32_t>((a.D + 255) / 256));
    hipLaunchKernelGGL(fill_zero_kernel, g, dim3(256), 0, stream, a.dweight, a.D);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.dbias) return e;
    hipLaunchKernelGGL(fill_zero_kernel, g, dim3(256), 0, stream, a.dbias, a.D);
    return hipGetLastError();
  }
  float* part = static_cast<float*>(ws);
  const int64_t blocks = norm_blocks(a.rows, a.D, a.dtype);
  hipError_t e;
  if (a.dtype == MSSM_BFLOAT16)
    e = dispatch_row<uint16_t>(a.D, RunNormBwd<uint16_t>{a, part, blocks, stream});
  else
    e = dispatch_row<float>(a.D, RunNormBwd<float>{a, part, blocks, stream});
  if (e != hipSuccess) return e;
  const uint32_t n = static_cast<uint32_t>((2 * a.D + 63) / 64);
  hipLaunchKernelGGL(layer_norm_sum_kernel, dim3(n), dim3(256), 0, stream, part,
                     static_cast<int>(blocks), a.D, a.dweight, a.dbias);
  return hipGetLastError();
}

}  // namespace mssm
