// The norms around a block with its gate, residual scale and residual add, forward and
// gradient (gfx950).  Per row of D values, with c = scale act(z):
//   post = 1 / sqrt(mean(y^2) + eps),  yhat = y post       (without post_weight: yhat = y, pw = 1)
//   t = residual + c yhat pw           rounded to the type
//   rstd = 1 / sqrt(mean(t^2) + eps),  that = t rstd,  out = that w
// Backwards, the means taken over the row and q = c pw yhat:
//   d   = dt + rstd (w dout - that mean(w dout that))          the gradient of t, and of residual
//   dy  = post (d c pw - yhat mean(d q))
//   dz  = d yhat pw scale act'(z),     dw = sum dout that,   dpw = sum d c yhat,
//   dscale = sum d yhat pw act(z)      (sums over rows; dz over the rows that share a gate)
// mean(d q) follows from sums that need no d: with S2 = sum (dt + rstd w dout) q and
// S3 = sum that q it is (S2 - rstd mean(w dout that) S3) / D, so a row meets one
// reduction.
//
// Bound by memory.  A thread holds 16-byte pieces of the same columns of every row it meets, and the
// parameters and the column sums of those columns in registers.  Short rows take a part of
// a wavefront, others as many wavefronts as they have pieces.
#include "mssm_internal.h"
#include "norm_device.h"

namespace mssm {

namespace {

constexpr int kMaxWaves = 16;

template <typename T>
__device__ __forceinline__ uint4 load_piece(const T* row, int c, int D) {
  constexpr int N = kPer<T>;
  uint4 u;
  if (D >= N) {
    __builtin_memcpy(&u, row + (c < D - N ? c : D - N), 16);
  } else {
    T e[N];
#pragma unroll
    for (int j = 0; j < N; ++j) e[j] = row[j < D ? j : D - 1];
    __builtin_memcpy(&u, e, 16);
  }
  return u;
}

// The piece that load_piece read for column c, widened; zero past the row's end.
template <typename T>
__device__ __forceinline__ void get_piece(uint4 u, int c, int D, float (&out)[kPer<T>]) {
  constexpr int N = kPer<T>;
  if (D >= N) {
    const uint32_t s = static_cast<uint32_t>(c > D - N ? c - (D - N) : 0) * sizeof(T) * 8;
    if (s & 64) u = make_uint4(u.z, u.w, 0u, 0u);
    if (s & 32) u = make_uint4(u.y, u.z, u.w, 0u);
    if (s & 16)
      u = make_uint4(u.x >> 16 | u.y << 16, u.y >> 16 | u.z << 16, u.z >> 16 | u.w << 16,
                     u.w >> 16);
    if (s >= 128) u = make_uint4(0u, 0u, 0u, 0u);
  }
  widen(u, out);
  if (D < N) {
#pragma unroll
    for (int j = 0; j < N; ++j) out[j] = c == 0 && j < D ? out[j] : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store_piece(T* row, int c, int D, const float (&v)[kPer<T>]) {
  constexpr int N = kPer<T>;
  if (c + N <= D) {
    const uint4 u = packed(v);
    __builtin_memcpy(row + c, &u, 16);
  } else {
#pragma unroll
    for (int j = 0; j + 1 < N; ++j)
      if (c + j < D) row[c + j] = narrow(v[j], T());
  }
}

// Sums over the threads of a row (TPR lanes of a wavefront, or with TPR = 0 the whole block), in a
// fixed order; all of them get them.  `flip` alternates, so one barrier is enough.
template <int TPR, int K>
__device__ __forceinline__ void sum_row(float (&v)[K], float (*red)[kMaxWaves][4], int& flip) {
#pragma unroll
  for (int o = (TPR ? TPR : 64) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], o, 64);
  if constexpr (TPR == 0) {
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) red[flip][threadIdx.x >> 6][k] = v[k];
    block_sync();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.0f;
    for (int w = 0; w < waves; ++w)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += red[flip][w][k];
    flip ^= 1;
  }
}

struct Slope {
  float value, slope;
};
__device__ __forceinline__ Slope gate_of(float z, bool silu_form) {
  if (!silu_form) return {z, 1.0f};
  const float s = __builtin_amdgcn_rcpf(1.0f + fast_exp2(-z * kLog2e));
  return {z * s, s * __builtin_fmaf(z, 1.0f - s, 1.0f)};
}

// Which rows a block meets: `per` rows at a time (one for each TPR threads), blocks side by side.
template <int TPR>
struct Rows {
  int tpr, per, lane, slot;
  __device__ __forceinline__ Rows() {
    tpr = TPR ? TPR : static_cast<int>(blockDim.x);
    per = TPR ? static_cast<int>(blockDim.x) / TPR : 1;
    lane = TPR ? static_cast<int>(threadIdx.x) % TPR : static_cast<int>(threadIdx.x);
    slot = TPR ? static_cast<int>(threadIdx.x) / TPR : 0;
  }
};

template <typename T, int N>
__device__ __forceinline__ void load_columns(const float* p, int c, int D, float other,
                                             float (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = c + j < D ? (p ? p[c + j] : other) : 0.0f;
}

template <typename T, int TPR, int VPT, bool kGate>
__global__ __launch_bounds__(TPR ? 256 : 1024) void residual_norm_kernel(ResidualNormArgs a) {
  constexpr int N = kPer<T>;
  __shared__ float red[2][kMaxWaves][4];
  int flip = 0;
  const Rows<TPR> at;
  const int D = static_cast<int>(a.D);
  const float inv = 1.0f / static_cast<float>(D);
  float w[VPT][N], pw[VPT][N];                     // pw: times the scale
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (at.lane + at.tpr * i) * N;
    float sc[N];
    load_columns<T>(a.weight, c, D, 1.0f, w[i]);
    load_columns<T>(a.post_weight, c, D, 1.0f, pw[i]);
    load_columns<T>(a.scale, c, D, 1.0f, sc);
#pragma unroll
    for (int j = 0; j < N; ++j) pw[i][j] *= sc[j];
  }
  const int64_t stride = int64_t(gridDim.x) * at.per;
  for (int64_t r0 = int64_t(blockIdx.x) * at.per; r0 < a.rows; r0 += stride) {
    const bool mine = r0 + at.slot < a.rows;
    const int64_t r = mine ? r0 + at.slot : a.rows - 1;
    uint4 y[VPT], q[VPT], z[VPT];
    const int64_t zr = a.gate_rows > 1 ? static_cast<uint32_t>(r) / static_cast<uint32_t>(a.gate_rows)
                                       : r;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (at.lane + at.tpr * i) * N;
      y[i] = load_piece(static_cast<const T*>(a.y) + r * D, c, D);
      if constexpr (kGate) z[i] = load_piece(static_cast<const T*>(a.gate) + zr * D, c, D);
      q[i] = load_piece(static_cast<const T*>(a.residual) + r * D, c, D);
    }
    float v[VPT][N], s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      get_piece<T>(y[i], (at.lane + at.tpr * i) * N, D, v[i]);
#pragma unroll
      for (int j = 0; j < N; ++j) s[0] = __builtin_fmaf(v[i][j], v[i][j], s[0]);
    }
    float post = 1.0f;
    if (a.post_weight) {
      sum_row<TPR>(s, red, flip);
      post = 1.0f / sqrtf(s[0] * inv + a.eps);
      if (mine && at.lane == 0 && a.post_rstd) a.post_rstd[r] = post;
    }
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (at.lane + at.tpr * i) * N;
      float u[N], g[N];
      get_piece<T>(q[i], c, D, u);
      if constexpr (kGate) get_piece<T>(z[i], c, D, g);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float t = v[i][j] * post * pw[i][j];
        if constexpr (kGate) t *= gate_of(g[j], a.silu).value;
        v[i][j] = to_float(narrow(u[j] + t, T()));
        s[0] = __builtin_fmaf(v[i][j], v[i][j], s[0]);
      }
      if (mine) store_piece(static_cast<T*>(a.total) + r * D, c, D, v[i]);
    }
    sum_row<TPR>(s, red, flip);
    const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
    if (mine && at.lane == 0 && a.rstd) a.rstd[r] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[i][j] = v[i][j] * rstd * w[i][j];
      if (mine) store_piece(static_cast<T*>(a.out) + r * D, (at.lane + at.tpr * i) * N, D, v[i]);
    }
  }
}

// The sums of the block's rows of threads for column piece i, into dst (those of slot 0 write).
template <int TPR, int N>
__device__ __forceinline__ bool sum_slots(const Rows<TPR>& at, float* cols, float (&v)[N]) {
  if constexpr (TPR == 0) return true;
  block_sync();
#pragma unroll
  for (int j = 0; j < N; ++j) cols[threadIdx.x * N + j] = v[j];
  block_sync();
  if (at.slot != 0) return false;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float t = 0.0f;
    for (int k = 0; k < at.per; ++k) t += cols[(k * at.tpr + at.lane) * N + j];
    v[j] = t;
  }
  return true;
}

template <int N>
__device__ __forceinline__ void store_columns(float* p, int c, int D, const float (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (c + j < D) p[c + j] = v[j];
}

// Rows in `sets` of `rows` each that share a gate (one set of all rows where each has its own, or
// none has one); `split` blocks work on a set.  part: [gridDim.x, 3, D] the blocks' sums
// for w, pw and the scale; gpart: [sets, split, D] those for the shared gates, where split > 1.
template <typename T, int TPR, int VPT, bool kGate>
__global__ __launch_bounds__(TPR ? 256 : 1024) void residual_norm_bwd_kernel(
    ResidualNormArgs a, ResidualNormGrads d, int64_t sets, int64_t rows, int64_t split, float* part,
    float* gpart) {
  constexpr int N = kPer<T>;
  __shared__ float red[2][kMaxWaves][4];
  __shared__ float cols[TPR ? 256 * N : 1];
  int flip = 0;
  const Rows<TPR> at;
  const int D = static_cast<int>(a.D);
  const float inv = 1.0f / static_cast<float>(D);
  const bool shared = kGate && a.gate_rows > 1;
  float w[VPT][N], pw[VPT][N], sc[VPT][N], dw[VPT][N], dpw[VPT][N], dsc[VPT][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (at.lane + at.tpr * i) * N;
    load_columns<T>(a.weight, c, D, 1.0f, w[i]);
    load_columns<T>(a.post_weight, c, D, 1.0f, pw[i]);
    load_columns<T>(a.scale, c, D, 1.0f, sc[i]);
#pragma unroll
    for (int j = 0; j < N; ++j) dw[i][j] = dpw[i][j] = dsc[i][j] = 0.0f;
  }
  const int64_t part_of = blockIdx.x % split, set_step = gridDim.x / split;
  for (int64_t set = blockIdx.x / split; set < sets; set += set_step) {
    float dz[VPT][N];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) dz[i][j] = 0.0f;
    for (int64_t r0 = part_of * at.per; r0 < rows; r0 += split * at.per) {
      const bool mine = r0 + at.slot < rows;
      const int64_t r = set * rows + (mine ? r0 + at.slot : rows - 1);
      uint4 g[VPT], e[VPT], t[VPT], y[VPT], z[VPT];
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (at.lane + at.tpr * i) * N;
        g[i] = load_piece(static_cast<const T*>(d.dout) + r * D, c, D);
        t[i] = load_piece(static_cast<const T*>(a.total) + r * D, c, D);
        y[i] = load_piece(static_cast<const T*>(a.y) + r * D, c, D);
        if constexpr (kGate)
          z[i] = load_piece(static_cast<const T*>(a.gate) + (shared ? set : r) * D, c, D);
        if (d.dtotal) e[i] = load_piece(static_cast<const T*>(d.dtotal) + r * D, c, D);
        else e[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      const float rstd = a.rstd[r];
      const float post = a.post_weight ? a.post_rstd[r] : 1.0f;
      float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (at.lane + at.tpr * i) * N;
        float gv[N], ev[N], tv[N], yv[N], zv[N];
        get_piece<T>(g[i], c, D, gv);
        get_piece<T>(e[i], c, D, ev);
        get_piece<T>(t[i], c, D, tv);
        get_piece<T>(y[i], c, D, yv);
        if constexpr (kGate) get_piece<T>(z[i], c, D, zv);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float that = tv[j] * rstd, wd = gv[j] * w[i][j];
          float q = sc[i][j] * pw[i][j] * (yv[j] * post);
          if constexpr (kGate) q *= gate_of(zv[j], a.silu).value;
          s[0] = __builtin_fmaf(wd, that, s[0]);
          s[1] = __builtin_fmaf(__builtin_fmaf(rstd, wd, ev[j]), q, s[1]);
          s[2] = __builtin_fmaf(that, q, s[2]);
        }
      }
      sum_row<TPR>(s, red, flip);
      const float m1 = s[0] * inv;
      const float m2 = a.post_weight ? (s[1] - rstd * m1 * s[2]) * inv : 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (at.lane + at.tpr * i) * N;
        float gv[N], ev[N], tv[N], yv[N], zv[N], dy[N], dr[N];
        get_piece<T>(g[i], c, D, gv);
        get_piece<T>(e[i], c, D, ev);
        get_piece<T>(t[i], c, D, tv);
        get_piece<T>(y[i], c, D, yv);
        if constexpr (kGate) get_piece<T>(z[i], c, D, zv);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float that = tv[j] * rstd, wd = gv[j] * w[i][j], yh = yv[j] * post;
          Slope k = {1.0f, 0.0f};
          if constexpr (kGate) k = gate_of(zv[j], a.silu);
          const float dt = __builtin_fmaf(rstd, wd - that * m1, ev[j]);
          const float dg = dt * k.value;                     // before the scale
          const float dc = dg * sc[i][j];
          dr[j] = dt;
          dy[j] = post * __builtin_fmaf(-yh, m2, dc * pw[i][j]);
          if (mine) {
            dw[i][j] = __builtin_fmaf(gv[j], that, dw[i][j]);
            dpw[i][j] = __builtin_fmaf(dc, yh, dpw[i][j]);
            dsc[i][j] = __builtin_fmaf(dg, yh * pw[i][j], dsc[i][j]);
          }
          if constexpr (kGate) {
            zv[j] = dt * yh * pw[i][j] * sc[i][j] * k.slope;
            if (mine) dz[i][j] += zv[j];
          }
        }
        if (mine) {
          store_piece(static_cast<T*>(d.dresidual) + r * D, c, D, dr);
          store_piece(static_cast<T*>(d.dy) + r * D, c, D, dy);
          if constexpr (kGate)
            if (!shared) store_piece(static_cast<T*>(d.dgate) + r * D, c, D, zv);
        }
      }
    }
    if (shared) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (at.lane + at.tpr * i) * N;
        if (sum_slots<TPR>(at, cols, dz[i])) {
          if (split == 1) store_piece(static_cast<T*>(d.dgate) + set * D, c, D, dz[i]);
          else store_columns(gpart + (set * split + part_of) * D, c, D, dz[i]);
        }
      }
    }
  }
  float* dst = part + int64_t(blockIdx.x) * 3 * D;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (at.lane + at.tpr * i) * N;
    if (sum_slots<TPR>(at, cols, dw[i])) store_columns(dst, c, D, dw[i]);
    if (sum_slots<TPR>(at, cols, dpw[i])) store_columns(dst + D, c, D, dpw[i]);
    if (sum_slots<TPR>(at, cols, dsc[i])) store_columns(dst + 2 * D, c, D, dsc[i]);
  }
}

// Sums of the rows of part for w, pw and the scale (blockIdx.y), in a fixed order.
__global__ __launch_bounds__(1024) void residual_norm_sum_kernel(const float* __restrict__ part,
                                                                 int64_t blocks, int64_t D,
                                                                 float* dw, float* dpw,
                                                                 float* dsc) {
  __shared__ double m[16][64];
  const int col = threadIdx.x & 63, w = threadIdx.x >> 6, k = blockIdx.y;
  float* to = k == 0 ? dw : k == 1 ? dpw : dsc;
  if (!to) return;
  const int64_t c = int64_t(blockIdx.x) * 64 + col;
  double s = 0.0;
  if (c < D)
    for (int64_t b = w; b < blocks; b += 16) s += part[(b * 3 + k) * D + c];
  m[w][col] = s;
  block_sync();
  if (w != 0 || c >= D) return;
  for (int j = 1; j < 16; ++j) s += m[j][col];
  to[c] = static_cast<float>(s);
}

// dgate [sets, D] = the sums of each set's `split` rows.
template <typename T>
__global__ __launch_bounds__(256) void residual_norm_gate_kernel(const float* __restrict__ part,
                                                                 int64_t split, int64_t D,
                                                                 int64_t n, T* dgate) {
  const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (e >= n) return;
  const int64_t set = e / D, c = e - set * D;
  float s = 0.0f;
  for (int64_t k = 0; k < split; ++k) s += part[(set * split + k) * D + c];
  dgate[e] = narrow(s, T());
}

__global__ __launch_bounds__(256) void residual_norm_zero_kernel(float* p, int64_t n) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// Calls f.template operator()<TPR, VPT>(threads of a block): a part of a wavefront for short
// rows, else the wavefronts that hold the row with VPT pieces a thread.
template <typename T, typename F>
hipError_t dispatch(int64_t D, F f) {
  const int64_t pieces = (D + kPer<T> - 1) / kPer<T>;
  if (pieces <= 8) return f.template operator()<8, 1>(256);
  if (pieces <= 16) return f.template operator()<16, 1>(256);
  if (pieces <= 32) return f.template operator()<32, 1>(256);
  if (pieces <= 64) return f.template operator()<64, 1>(256);
  auto threads = [&](int64_t vpt) {
    return static_cast<uint32_t>((pieces + 64 * vpt - 1) / (64 * vpt) * 64);
  };
  if (pieces <= 1024) return f.template operator()<0, 1>(threads(1));
  if (pieces <= 2048) return f.template operator()<0, 2>(threads(2));
  if constexpr (sizeof(T) == 4)
    if (pieces <= 4096) return f.template operator()<0, 4>(threads(4));
  return hipErrorInvalidValue;
}

template <typename T>
struct Fwd {
  const ResidualNormArgs& a;
  hipStream_t stream;
  template <int TPR, int VPT>
  hipError_t operator()(uint32_t threads) const {
    const int64_t per = TPR ? threads / TPR : 1;
    int64_t blocks = (a.rows + per - 1) / per;
    if (blocks > 4096) blocks = 4096;
    const dim3 grid(static_cast<uint32_t>(blocks)), block(threads);
    if (a.gate)
      hipLaunchKernelGGL((residual_norm_kernel<T, TPR, VPT, true>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((residual_norm_kernel<T, TPR, VPT, false>), grid, block, 0, stream, a);
    return hipGetLastError();
  }
};

// How the gradient's rows are dealt to blocks.
struct Deal {
  int64_t sets = 1, rows = 0, split = 1, blocks = 0;
};

template <typename T>
struct MakeDeal {
  int64_t rows, gate_rows;
  Deal* out;
  template <int TPR, int VPT>
  hipError_t operator()(uint32_t threads) const {
    const int64_t per = TPR ? threads / TPR : 1;
    const int64_t most = 1024;
    out->sets = gate_rows > 1 ? rows / gate_rows : 1;
    out->rows = rows / out->sets;
    const int64_t room = (out->rows + per - 1) / per;
    out->split = out->sets >= most ? 1 : (most + out->sets - 1) / out->sets;
    if (out->split > room) out->split = room;
    const int64_t wide = most / out->split > 0 ? most / out->split : 1;
    out->blocks = (out->sets < wide ? out->sets : wide) * out->split;
    return hipSuccess;
  }
};

Deal deal_of(int64_t rows, int64_t D, int64_t gate_rows, mssm_dtype dtype) {
  Deal d;
  if (dtype == MSSM_BFLOAT16) dispatch<uint16_t>(D, MakeDeal<uint16_t>{rows, gate_rows, &d});
  else dispatch<float>(D, MakeDeal<float>{rows, gate_rows, &d});
  return d;
}

template <typename T>
struct Bwd {
  const ResidualNormArgs& a;
  const ResidualNormGrads& d;
  const Deal& deal;
  float* part;
  float* gpart;
  hipStream_t stream;
  template <int TPR, int VPT>
  hipError_t operator()(uint32_t threads) const {
    const dim3 grid(static_cast<uint32_t>(deal.blocks)), block(threads);
    if (a.gate)
      hipLaunchKernelGGL((residual_norm_bwd_kernel<T, TPR, VPT, true>), grid, block, 0, stream, a,
                         d, deal.sets, deal.rows, deal.split, part, gpart);
    else
      hipLaunchKernelGGL((residual_norm_bwd_kernel<T, TPR, VPT, false>), grid, block, 0, stream, a,
                         d, deal.sets, deal.rows, deal.split, part, gpart);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_residual_norm(const ResidualNormArgs& a, hipStream_t stream) {
  if (a.dtype == MSSM_BFLOAT16) return dispatch<uint16_t>(a.D, Fwd<uint16_t>{a, stream});
  return dispatch<float>(a.D, Fwd<float>{a, stream});
}

size_t residual_norm_bwd_workspace(int64_t rows, int64_t D, int64_t gate_rows, mssm_dtype dtype) {
  if (rows == 0 || D == 0) return 0;
  const Deal d = deal_of(rows, D, gate_rows, dtype);
  const size_t gates = gate_rows > 1 && d.split > 1 ? static_cast<size_t>(d.sets) * d.split : 0;
  return (static_cast<size_t>(d.blocks) * 3 + gates) * D * sizeof(float);
}

hipError_t launch_residual_norm_bwd(const ResidualNormArgs& a, const ResidualNormGrads& d, void* ws,
                                    hipStream_t stream) {
  if (a.rows == 0) {
    for (float* p : {d.dweight, d.dpost_weight, d.dscale}) {
      if (!p) continue;
      hipLaunchKernelGGL(residual_norm_zero_kernel, dim3(static_cast<uint32_t>((a.D + 255) / 256)),
                         dim3(256), 0, stream, p, a.D);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const Deal deal = deal_of(a.rows, a.D, a.gate_rows, a.dtype);
  float* part = static_cast<float*>(ws);
  float* gpart = part + deal.blocks * 3 * a.D;
  hipError_t e;
  if (a.dtype == MSSM_BFLOAT16)
    e = dispatch<uint16_t>(a.D, Bwd<uint16_t>{a, d, deal, part, gpart, stream});
  else
    e = dispatch<float>(a.D, Bwd<float>{a, d, deal, part, gpart, stream});
  if (e != hipSuccess) return e;
  if (a.gate && a.gate_rows > 1 && deal.split > 1) {
    const int64_t n = deal.sets * a.D;
    const dim3 grid(static_cast<uint32_t>((n + 255) / 256));
    if (a.dtype == MSSM_BFLOAT16)
      hipLaunchKernelGGL(residual_norm_gate_kernel<uint16_t>, grid, dim3(256), 0, stream, gpart,
                         deal.split, a.D, n, static_cast<uint16_t*>(d.dgate));
    else
      hipLaunchKernelGGL(residual_norm_gate_kernel<float>, grid, dim3(256), 0, stream, gpart,
                         deal.split, a.D, n, static_cast<float*>(d.dgate));
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(residual_norm_sum_kernel, dim3(static_cast<uint32_t>((a.D + 63) / 64), 3),
                     dim3(1024), 0, stream, part, deal.blocks, a.D, d.dweight, d.dpost_weight,
                     d.dscale);
  return hipGetLastError();
}

}  // namespace mssm
