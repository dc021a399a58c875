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
// float32 butterflies.
//
// Where a wavefront (or a part of one) holds a row, it works through many rows
// and loads the next one before it needs it; w and b wait in LDS, whose reads
// are counted apart from those loads.  No branch stands around the loads: a
// piece past the row's end loads the row's last 16 bytes instead and shifts out
// what is not its own, which also serves rows of any length and alignment
// (global memory takes 16-byte loads at any address).
//
// The gradients of w and b: a block runs over many rows and keeps its columns'
// sums in registers; at the end it writes one row of partial sums, and a second
// kernel adds the blocks' rows, all in a fixed order.
//
// Measured: 32768 x 2560 bf16 with the residual 135 us (671 MB, 5.0 TB/s; a large
// copy runs at 5.1 to 5.4), its gradient 146 + 6 us (4.6 TB/s); 16384 x 1536 float32
// gradient 63 us with the sums (4.8 TB/s); 8 rows of 2560: 6 us, a launch and two
// trips to memory, less than the host takes for the call.  The forward pass is near the
// copy's rate up to 4096 values a row (8192 x 4096 bf16 with the residual: 51 us, 5.2
// TB/s; 60000 x 333 float32: 34 us, 4.7) and falls off where a block holds a row and loads
// nothing ahead (4096 x 8192 bf16: 39 us, 3.4; 2048 x 16384 float32: 68 us, 4.0).  The
// gradient is far from it away from the widths above: rows of 64 have too few blocks and
// 16 bytes a lane in flight (65536 x 64 bf16: 24 us, 1.0 TB/s); rows of a whole block
// load nothing ahead (8192 x 4096 bf16: 67 us, 3.0; 4096 x 8192: 79 us, 2.5); float32
// rows of 1793 to 2048 spill (16384 x 2048 with the stream's gradient: 219 us, 2.5).
#include "mssm_internal.h"
#include "norm_device.h"

namespace mssm {

namespace {

// The pieces of a row that thread `lane` of its TPR holds, as they lie in
// memory: piece i begins at column (lane + TPR i) kPer.  Only the last of a
// thread's pieces can reach past the row's end.  (Rows shorter than a piece:
// element by element.)
template <typename T, int TPR, int VPT>
struct Row {
  static constexpr int N = kPer<T>;
  static constexpr bool kLong = TPR > 8;      // rows of more than eight pieces
  uint4 v[VPT];

  __device__ __forceinline__ void load(const T* row, int lane, int D) {
    if (kLong || D >= N) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (lane + TPR * i) * N;
        __builtin_memcpy(&v[i], row + (i + 1 < VPT ? c : min(c, D - N)), 16);
      }
    } else {
      T e[N];
#pragma unroll
      for (int j = 0; j < N; ++j) e[j] = row[min(j, D - 1)];
      __builtin_memcpy(&v[0], e, 16);
    }
  }
  // Piece i widened; zero past the row's end.
  __device__ __forceinline__ void get(int i, int lane, int D, float (&out)[N]) const {
    uint4 u = v[i];
    if (i + 1 == VPT) {
      const int c = (lane + TPR * i) * N;
      if (kLong || D >= N) {          // values that came from before c go, zeros follow
        const uint32_t s = static_cast<uint32_t>(max(c - (D - N), 0)) * sizeof(T) * 8;
        if (s & 64) u = make_uint4(u.z, u.w, 0u, 0u);
        if (s & 32) u = make_uint4(u.y, u.z, u.w, 0u);
        if (s & 16)
          u = make_uint4(u.x >> 16 | u.y << 16, u.y >> 16 | u.z << 16, u.z >> 16 | u.w << 16,
                         u.w >> 16);
        if (s >= 128) u = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    widen(u, out);
    if (!kLong && D < N) {
#pragma unroll
      for (int j = 0; j < N; ++j) out[j] = lane == 0 && j < D ? out[j] : 0.0f;
    }
  }
  __device__ __forceinline__ void keep_packed() {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      asm volatile("" : "+v"(v[i].x), "+v"(v[i].y), "+v"(v[i].z), "+v"(v[i].w));
  }
  static __device__ __forceinline__ void store(T* row, int i, int lane, int D,
                                               const float (&out)[N]) {
    const int c = (lane + TPR * i) * N;
    if (i + 1 < VPT || c + N <= D) {
      const uint4 u = packed(out);
      __builtin_memcpy(row + c, &u, 16);
    } else {
      T* p = row + c;
#pragma unroll
      for (int j = 0; j + 1 < N; ++j)       // a whole piece went the other way
        if (c + j < D) p[j] = narrow(out[j], T());
    }
  }
};

// Sums over the TPR threads of a row; every one of them gets them.  `red` has
// room for the wavefronts' parts, twice; `flip` alternates so that one barrier
// for each call is enough.
template <int TPR, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float* red, int& flip) {
#pragma unroll
  for (int o = (TPR < 64 ? TPR : 64) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], o, 64);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* m = red + flip * (2 * W);
    flip ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) m[k * W + (threadIdx.x >> 6)] = v[k];
    block_sync();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) v[k] += m[k * W + w];
    }
  }
}

// The parameters a block keeps in LDS (rows of up to a wavefront): D values
// rounded up to whole pieces of all threads, zero past D.
template <int TPR, int VPT, int N>
constexpr int kWidth = TPR * VPT * N;

template <int W, int kBlock>
__device__ __forceinline__ void stage_params(float* lds, const float* p, int D) {
  for (int c = threadIdx.x; c < W; c += kBlock) lds[c] = p && c < D ? p[c] : 0.0f;
}

template <typename T, int TPR, int VPT, bool kResidual>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void layer_norm_kernel(NormArgs a) {
  constexpr int N = kPer<T>;
  constexpr int kBlock = TPR > 256 ? TPR : 256;
  constexpr int kRows = kBlock / TPR;
  constexpr bool kAhead = TPR <= 64;
  constexpr int W = kWidth<TPR, VPT, N>;
  using R = Row<T, TPR, VPT>;
  __shared__ float red[TPR > 64 ? 4 * TPR / 64 : 1];
  __shared__ __align__(16) float sw[kAhead ? W : 4], sb[kAhead ? W : 4];
  int flip = 0;
  const int lane = threadIdx.x % TPR;
  const int D = static_cast<int>(a.D);
  const float inv = 1.0f / static_cast<float>(D);
  const T* X = static_cast<const T*>(a.x);
  const T* Q = static_cast<const T*>(a.residual);
  if constexpr (kAhead) {
    stage_params<W, kBlock>(sw, a.weight, D);
    stage_params<W, kBlock>(sb, a.bias, D);
    block_sync();
  }
  int64_t r = int64_t(blockIdx.x) * kRows + threadIdx.x / TPR;
  const int64_t stride = int64_t(gridDim.x) * kRows;
  R x, q;
  if (r < a.rows) {
    x.load(X + r * a.D, lane, D);
    if constexpr (kResidual) q.load(Q + r * a.D, lane, D);
  }
  for (; r < a.rows; r += stride) {
    float v[VPT][N];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      x.get(i, lane, D, v[i]);
      if constexpr (kResidual) {
        float u[N];
        q.get(i, lane, D, u);
#pragma unroll
        for (int j = 0; j < N; ++j) v[i][j] = to_float(narrow(v[i][j] + u[j], T()));
      }
    }
    const int64_t next = min(r + stride, a.rows - 1);
    if constexpr (kAhead) x.load(X + next * a.D, lane, D);
    if constexpr (kResidual) {
      if constexpr (kAhead) q.load(Q + next * a.D, lane, D);
      T* t = static_cast<T*>(a.sum) + r * a.D;
#pragma unroll
      for (int i = 0; i < VPT; ++i) R::store(t, i, lane, D, v[i]);
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) s[0] += v[i][j];
    row_sums<TPR>(s, red, flip);
    const float mean = s[0] * inv;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (lane + TPR * i) * N;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        v[i][j] = i + 1 < VPT || c + j < D ? v[i][j] - mean : 0.0f;
        s[0] = __builtin_fmaf(v[i][j], v[i][j], s[0]);
      }
    }
    row_sums<TPR>(s, red, flip);
    const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
    if (lane == 0 && a.mean) {
      a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
    T* y = static_cast<T*>(a.y) + r * a.D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (lane + TPR * i) * N;
      float w[N], b[N];
      if constexpr (kAhead) {
        load_param<N>(sw, c, W, w);
        load_param<N>(sb, c, W, b);
      } else {
        load_param<N>(a.weight, c, D, w);
        if (a.bias) {
          load_param<N>(a.bias, c, D, b);
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j) b[j] = 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < N; ++j) v[i][j] = __builtin_fmaf(v[i][j] * rstd, w[j], b[j]);
      R::store(y, i, lane, D, v[i]);
    }
  }
}

// part: [gridDim.x, 2, D]: the block's sums of dy xhat and of dy.
template <typename T, int TPR, int VPT, bool kSum>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256, TPR > 256 ? 4 : 2) void layer_norm_bwd_kernel(NormBwdArgs a,
                                                                               float* part) {
  constexpr int N = kPer<T>;
  constexpr int kBlock = TPR > 256 ? TPR : 256;
  constexpr int kRows = kBlock / TPR;                  // rows at a time
  constexpr bool kAhead = TPR <= 64;
  constexpr int W = kWidth<TPR, VPT, N>;
  using R = Row<T, TPR, VPT>;
  __shared__ float red[TPR > 64 ? 4 * TPR / 64 : 1];
  __shared__ __align__(16) float sw[kAhead ? W : 4];
  __shared__ float cols[TPR < 256 ? kBlock * N : 1];
  int flip = 0;
  const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int D = static_cast<int>(a.D);
  const float inv = 1.0f / static_cast<float>(D);
  const T* DY = static_cast<const T*>(a.dy);
  const T* X = static_cast<const T*>(a.x);
  if constexpr (kAhead) {
    stage_params<W, kBlock>(sw, a.weight, D);
    block_sync();
  }
  float dw[VPT][N], db[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) dw[i][j] = db[i][j] = 0.0f;
  auto weights = [&](int i, float (&w)[N]) {
    const int c = (lane + TPR * i) * N;
    if constexpr (kAhead) load_param<N>(sw, c, W, w);
    else load_param<N>(a.weight, c, D, w);
  };

  int64_t r = int64_t(blockIdx.x) * kRows + group;
  const int64_t stride = int64_t(gridDim.x) * kRows;
  R gs[2], xs[2];
  float ms[2], rs[2];
  auto load = [&](int k, int64_t row) __attribute__((always_inline)) {
    gs[k].load(DY + row * a.D, lane, D);
    xs[k].load(X + row * a.D, lane, D);
    ms[k] = a.mean[row];
    rs[k] = a.rstd[row];
  };
  auto work = [&](int k, int64_t row) __attribute__((always_inline)) {
    const float mean = ms[k], rstd = rs[k];
    R e;
    if constexpr (kSum) e.load(static_cast<const T*>(a.dsum) + row * a.D, lane, D);
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float g[N], v[N], w[N];
      gs[k].get(i, lane, D, g);
      xs[k].get(i, lane, D, v);
      weights(i, w);
#pragma unroll
      for (int j = 0; j < N; ++j) {                    // past D: g and w are zero
        const float xh = (v[j] - mean) * rstd;
        dw[i][j] = __builtin_fmaf(g[j], xh, dw[i][j]);
        db[i][j] += g[j];
        const float wg = g[j] * w[j];
        s[0] += wg;
        s[1] = __builtin_fmaf(wg, xh, s[1]);
      }
    }
    // The sums over rows are up to date here, and the row is widened once more
    // below: kept as it was loaded it takes half the registers.
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) asm volatile("" : "+v"(dw[i][j]), "+v"(db[i][j]));
    gs[k].keep_packed();
    xs[k].keep_packed();
    row_sums<TPR>(s, red, flip);
    const float m1 = s[0] * inv, m2 = s[1] * inv;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float g[N], v[N], w[N], out[N];
      gs[k].get(i, lane, D, g);
      xs[k].get(i, lane, D, v);
      weights(i, w);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float xh = (v[j] - mean) * rstd;
        out[j] = rstd * (g[j] * w[j] - __builtin_fmaf(xh, m2, m1));
      }
      if constexpr (kSum) {
        float u[N];
        e.get(i, lane, D, u);
#pragma unroll
        for (int j = 0; j < N; ++j) out[j] += u[j];
      }
      R::store(static_cast<T*>(a.dx) + row * a.D, i, lane, D, out);
    }
  };
  if constexpr (kAhead) {
    // two rows' registers in turn: the next row is on its way while one is worked on
    if (r < a.rows) load(0, r);
    while (r < a.rows) {
      load(1, min(r + stride, a.rows - 1));
      work(0, r);
      r += stride;
      if (r >= a.rows) break;
      load(0, min(r + stride, a.rows - 1));
      work(1, r);
      r += stride;
    }
  } else {
    for (; r < a.rows; r += stride) {
      load(0, r);
      work(0, r);
    }
  }

  float* dst = part + int64_t(blockIdx.x) * 2 * a.D;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float(&acc)[N] = k ? db[i] : dw[i];
      if constexpr (TPR >= 256) {
        const int c = (lane + TPR * i) * N;
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (c + j < D) dst[k * a.D + c + j] = acc[j];
      } else {
        // the block's rows of threads hold the same columns: add them in order
        block_sync();
#pragma unroll
        for (int j = 0; j < N; ++j) cols[(group * TPR + lane) * N + j] = acc[j];
        block_sync();
        for (int q = threadIdx.x; q < TPR * N; q += kBlock) {
          float t = 0.0f;
          for (int w = 0; w < kRows; ++w) t += cols[w * TPR * N + q];
          const int c = TPR * i * N + q;
          if (c < D) dst[k * a.D + c] = t;
        }
      }
    }
  }
}

// out[c] = the sum of `blocks` rows of part, for the 2 D columns of [dw | db].
// A block takes 64 columns: 16 threads of four columns by 64 rows at a time.
__global__ __launch_bounds__(1024) void layer_norm_sum_kernel(const float* __restrict__ part,
                                                              int blocks, int64_t D, float* dw,
                                                              float* db) {
  __shared__ float m[64][65];
  const int64_t c0 = int64_t(blockIdx.x) * 64;
  const int64_t width = 2 * D;
  const int q = threadIdx.x % 16, row = threadIdx.x / 16;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t c = c0 + 4 * q;
#pragma unroll 8
  for (int b = row; b < blocks; b += 64) {
    float u[4];
    load_param<4>(part + int64_t(b) * width, c, width, u);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += u[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) m[row][4 * q + j] = s[j];
  block_sync();
  // 16 threads a column, four rows each, then a butterfly
  const int col = threadIdx.x / 16, r0 = 4 * (threadIdx.x % 16);
  float t = (m[r0][col] + m[r0 + 1][col]) + (m[r0 + 2][col] + m[r0 + 3][col]);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) t += __shfl_xor(t, o, 64);
  const int64_t to = c0 + col;
  if (threadIdx.x % 16 == 0) {
    if (to < D) dw[to] = t;
    else if (to < width && db) db[to - D] = t;
  }
}

__global__ __launch_bounds__(256) void fill_zero_kernel(float* p, int64_t n) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// Calls f.template operator()<TPR, VPT>() for the threads per row and pieces
// per thread that hold D values: a part of a wavefront for the shortest rows,
// one wavefront up to 40 values a lane (the backward pass keeps five numbers for
// each), then a block of 256 up to 32 values a thread, then of 1024.
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
    default: break;
  }
  if constexpr (sizeof(T) == 4) {
    switch ((pieces + 63) / 64) {
      case 6: return f.template operator()<64, 6>();
      case 7: return f.template operator()<64, 7>();
      case 8: return f.template operator()<64, 8>();
      default: break;
    }
    switch ((pieces + 255) / 256) {
      case 5: return f.template operator()<256, 5>();
      case 6: return f.template operator()<256, 6>();
      case 7: return f.template operator()<256, 7>();
      case 8: return f.template operator()<256, 8>();
      default: break;
    }
  } else {
    if (pieces <= 512) return f.template operator()<256, 2>();
  }
  switch ((pieces + 255) / 256) {
    case 3: return f.template operator()<256, 3>();
    case 4: return f.template operator()<256, 4>();
    default: break;
  }
  if constexpr (sizeof(T) == 4) {
    switch ((pieces + 1023) / 1024) {
      case 3: return f.template operator()<1024, 3>();
      case 4: return f.template operator()<1024, 4>();
      default: break;
    }
  } else {
    if (pieces <= 2048) return f.template operator()<1024, 2>();
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
    // A wavefront that holds whole rows works through several of them: 2048 blocks
    // (32768 x 2560 with a residual: 134 to 140 us from 256 to 4096 blocks; 60000 x
    // 333 float32: 65 us with 256, 34 from 768 on).
    int64_t blocks = (a.rows + per - 1) / per;
    if (TPR <= 64) return launch<TPR, VPT>(a, blocks > 2048 ? 2048 : blocks);
    // A block that holds one row takes one; the rows past what a grid can be get a
    // launch of their own.
    constexpr int64_t most = (int64_t(1) << 32) / kBlock - 1;
    for (int64_t r = 0; r < a.rows; r += most) {
      NormArgs p = a;
      p.rows = a.rows - r < most ? a.rows - r : most;
      const int64_t n = r * a.D;
      p.x = static_cast<const T*>(a.x) + n;
      p.y = static_cast<T*>(a.y) + n;
      if (a.residual) {
        p.residual = static_cast<const T*>(a.residual) + n;
        p.sum = static_cast<T*>(a.sum) + n;
      }
      if (a.mean) p.mean += r, p.rstd += r;
      const hipError_t e = launch<TPR, VPT>(p, p.rows);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  template <int TPR, int VPT>
  hipError_t launch(const NormArgs& p, int64_t blocks) const {
    constexpr int kBlock = TPR > 256 ? TPR : 256;
    const dim3 grid(static_cast<uint32_t>(blocks));
    if (p.residual)
      hipLaunchKernelGGL((layer_norm_kernel<T, TPR, VPT, true>), grid, dim3(kBlock), 0, stream, p);
    else
      hipLaunchKernelGGL((layer_norm_kernel<T, TPR, VPT, false>), grid, dim3(kBlock), 0, stream, p);
    return hipGetLastError();
  }
};

// Blocks of the backward pass: sixteen turns of the row loop each, which leaves
// few partial sums, but no fewer than 256 blocks and no more than 512 (32768 x
// 2560: 200 us with 256, 155 with 512, 191 with 768; 16384 x 1536 float32: 68 us
// with 256, 73 with 512).
template <typename T>
struct NormBlocks {
  int64_t rows;
  int64_t* blocks;
  template <int TPR, int VPT>
  hipError_t operator()() const {
    const int64_t per = TPR >= 256 ? 1 : 256 / TPR;
    const int64_t need = (rows + per - 1) / per;
    const int64_t want = need / 16 < 256 ? 256 : need / 16 > 512 ? 512 : need / 16;
    *blocks = need < want ? need : want;
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
    const dim3 grid(static_cast<uint32_t>(blocks));
    if (a.dsum)
      hipLaunchKernelGGL((layer_norm_bwd_kernel<T, TPR, VPT, true>), grid, dim3(kBlock), 0, stream,
                         a, part);
    else
      hipLaunchKernelGGL((layer_norm_bwd_kernel<T, TPR, VPT, false>), grid, dim3(kBlock), 0,
                         stream, a, part);
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

bool norm_size_supported(int64_t D) { return D >= 0 && D <= 16384; }

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
  hipLaunchKernelGGL(layer_norm_sum_kernel, dim3(n), dim3(1024), 0, stream, part,
                     static_cast<int>(blocks), a.D, a.dweight, a.dbias);
  return hipGetLastError();
}

}  // namespace mssm
