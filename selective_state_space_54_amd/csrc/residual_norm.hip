// The norms around a block with its gate, residual scale and residual add, forward and
// gradient (gfx950).  Per row of D values, with c = scale act(z):
//   post = 1 / sqrt(mean(y^2) + eps),  yhat = y post       (without post_weight: yhat = y, pw = 1)
//   t = residual + c yhat pw           rounded to the type
//   rstd = 1 / sqrt(mean(t^2) + eps),  that = t rstd,  out = that w
// Backwards, the means taken over the row and q = c pw yhat:
//   d   = dt + rstd (w dout - that mean(w dout that))          the gradient of t, and of residual
//   dy  = post (d c pw - yhat mean(d q))
//   dz  = d yhat pw scale act'(z),     dw = sum dout that
//   dpw = scale S,  dscale = pw S,     S = sum d act(z) yhat
// (sums over rows; dz over the rows that share a gate)
// mean(d q) follows from sums that need no d: with S2 = sum (dt + rstd w dout) q and
// S3 = sum that q it is (S2 - rstd mean(w dout that) S3) / D, so a row meets one
// reduction.
//
// Bound by memory.  A thread holds 16-byte pieces of the same columns of every row it meets, and
// the column sums of those columns in registers.  Short rows take a part of a wavefront, others as
// many wavefronts as they have pieces.
//
// There is no branch around a load or a store (one would have every wait for a load also wait
// for the stores before it): the last piece of a row whose end is not a piece's is the row's last
// N values, threads past the end repeat it, and rows past the last one repeat the last one.
// All of those compute the same values again and write them to the same place; only the sums leave
// them out.  So outputs must not be inputs.
//
// bfloat16, every part: 32768 x 2560 169 us (5.0 TB/s; 202 before the loads ahead), its gradient 286 us
// (4.7 TB/s; 614 with branches and the sums' own pass), 8 rows 7 us; float32 gradient 16384 x 1536 with
// gates that 2048 rows share 130 us (4.6 TB/s; 295).
#include <type_traits>

#include "mssm_internal.h"
#include "norm_device.h"

namespace mssm {

namespace {

constexpr int kMaxWaves = 16;
constexpr int kMinWaves = 4;              // wavefronts a SIMD: at most 128 registers

// Rows of up to 512 pieces: two fit a thread's registers.
template <int VPT, int kThreads>
constexpr bool kLoadsAhead = VPT == 1 && kThreads <= 512;

// A thread's N = 16 / sizeof(T) columns of a row: from c on, of which lo .. are its own (none past
// the row's end).  kShort: a row shorter than N, read and written value by value.
template <typename T, bool kShort>
struct Columns {
  static constexpr int N = kPer<T>;
  int c, lo, D;
  __device__ __forceinline__ Columns(int piece, int D_) : D(D_) {
    const int at = piece * N;
    c = kShort ? 0 : at < D - N ? at : D - N;
    lo = at - c < N ? at - c : N;
  }
  __device__ __forceinline__ bool own(int j) const { return j >= lo && (!kShort || j < D); }
  __device__ __forceinline__ uint4 load(const void* base, int64_t row) const {
    const T* p = static_cast<const T*>(base) + row * D;
    uint4 u;
    if constexpr (!kShort) {
      __builtin_memcpy(&u, p + c, 16);
    } else {
      T e[N];
#pragma unroll
      for (int j = 0; j < N; ++j) e[j] = p[j < D ? j : D - 1];
      __builtin_memcpy(&u, e, 16);
    }
    return u;
  }
  __device__ __forceinline__ void store(void* base, int64_t row, const float (&v)[N]) const {
    T* p = static_cast<T*>(base) + row * D;
    if constexpr (!kShort) {
      const uint4 u = packed(v);
      __builtin_memcpy(p + c, &u, 16);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (j < D) p[j] = narrow(v[j], T());
    }
  }
  __device__ __forceinline__ void store_sums(float* row, const float (&v)[N]) const {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (own(j)) row[c + j] = v[j];
  }
  __device__ __forceinline__ float param(const float* p, int j) const {
    return !p || (kShort && j >= D) ? 1.0f : p[c + j];
  }
};

// Value j of a piece.
template <typename T>
__device__ __forceinline__ float value(const uint4& u, int j) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
  else return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
}

template <int kCtrl>
__device__ __forceinline__ float plus_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xF, 0xF, true));
}

// The sum over each group of W neighbouring lanes, in every one of them.
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
  v = plus_dpp<0xB1>(v);                          // quad_perm [1, 0, 3, 2]
  v = plus_dpp<0x4E>(v);                          // quad_perm [2, 3, 0, 1]
  v = plus_dpp<0x141>(v);                         // row_half_mirror: the other quad of eight
  if constexpr (W > 8) v = plus_dpp<0x140>(v);    // row_mirror: the other eight of sixteen
  if constexpr (W > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (W > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Sums over the threads of a row (TPR lanes of a wavefront, or with TPR = 0 the whole block), in a
// fixed order; all of them get them.  `flip` alternates, so one barrier is enough.
template <int TPR, int K>
__device__ __forceinline__ void sum_row(float (&v)[K], float (*red)[kMaxWaves][4], int& flip) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lanes_sum<TPR ? TPR : 64>(v[k]);
  if constexpr (TPR == 0) {
    const int waves = blockDim.x >> 6;
#pragma unroll
    for (int k = 0; k < K; ++k) red[flip][threadIdx.x >> 6][k] = v[k];    // the same from every lane
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
  const float s = __builtin_amdgcn_rcpf(1.0f + fast_exp2(-z * kLog2e));
  Slope k = {z * s, s * __builtin_fmaf(z, 1.0f - s, 1.0f)};
  if (!silu_form) k = {z, 1.0f};
  return k;
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
  // Row r0 + slot of `rows`, or the last one.
  __device__ __forceinline__ int64_t at(int64_t r0, int64_t rows) const {
    const int64_t r = r0 + slot;
    return r < rows ? r : rows - 1;
  }
};

// Where a row's statistic goes; nowhere without p.
__device__ __forceinline__ void store_stat(float* p, int64_t r0, int slot, float v) {
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), make_buf(p + (p ? r0 : 0), p ? 4 * 64 : 0),
                                        slot * 4, 0, 0);
}

template <int VPT, bool kGate>
struct FwdRow {
  uint4 y[VPT], q[VPT], z[kGate ? VPT : 1];
};

template <typename T, int TPR, int VPT, int kThreads, bool kShort, bool kGate>
__global__ __launch_bounds__(kThreads, kMinWaves) void residual_norm_kernel(ResidualNormArgs a) {
  constexpr int N = kPer<T>;
  using Col = Columns<T, kShort>;
  __shared__ float red[2][kMaxWaves][4];
  int flip = 0;
  const Rows<TPR> at;
  const int D = static_cast<int>(a.D);
  const float inv = 1.0f / static_cast<float>(D);
  float w[VPT][N], cp[VPT][N];                     // cp: post_weight times the scale
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const Col col(at.lane + at.tpr * i, D);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      w[i][j] = col.param(a.weight, j);
      cp[i][j] = col.param(a.post_weight, j) * col.param(a.scale, j);
    }
  }
  using Row = FwdRow<VPT, kGate>;
  auto load = [&](Row& p, int64_t r0) __attribute__((always_inline)) {
    const int64_t r = at.at(r0, a.rows);
    const int64_t zr = a.gate_rows > 1 ? static_cast<uint32_t>(r) / static_cast<uint32_t>(a.gate_rows)
                                       : r;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const Col col(at.lane + at.tpr * i, D);
      p.y[i] = col.load(a.y, r);
      if constexpr (kGate) p.z[i] = col.load(a.gate, zr);
      p.q[i] = col.load(a.residual, r);
    }
  };
  auto work = [&](const Row& p, int64_t r0) __attribute__((always_inline)) {
    const int64_t r = at.at(r0, a.rows);
    const int slot = r0 + at.slot < a.rows ? at.slot : 64;
    float post = 1.0f, s[1];
    if (a.post_weight) {
      s[0] = 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const Col col(at.lane + at.tpr * i, D);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float v = col.own(j) ? value<T>(p.y[i], j) : 0.0f;
          s[0] = __builtin_fmaf(v, v, s[0]);
        }
      }
      sum_row<TPR>(s, red, flip);
      post = 1.0f / sqrtf(s[0] * inv + a.eps);
    }
    float t[VPT][N];
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const Col col(at.lane + at.tpr * i, D);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float v = value<T>(p.y[i], j) * post * cp[i][j];
        if constexpr (kGate) v *= gate_of(value<T>(p.z[i], j), a.silu).value;
        t[i][j] = to_float(narrow(value<T>(p.q[i], j) + v, T()));
        const float u = col.own(j) ? t[i][j] : 0.0f;
        s[0] = __builtin_fmaf(u, u, s[0]);
      }
      col.store(a.total, r, t[i]);
    }
    sum_row<TPR>(s, red, flip);
    const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
    store_stat(a.rstd, r0, slot, rstd);
    store_stat(a.post_rstd, r0, slot, post);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const Col col(at.lane + at.tpr * i, D);
#pragma unroll
      for (int j = 0; j < N; ++j) t[i][j] = t[i][j] * rstd * w[i][j];
      col.store(a.out, r, t[i]);
    }
  };
  const int64_t step = int64_t(gridDim.x) * at.per;
  int64_t r0 = int64_t(blockIdx.x) * at.per;
  if constexpr (kLoadsAhead<VPT, kThreads>) {
    // two rows' registers in turn: the next row is on its way while one is worked on
    Row p[2];
    load(p[0], r0);
    while (r0 < a.rows) {
      load(p[1], r0 + step);
      work(p[0], r0);
      r0 += step;
      if (r0 >= a.rows) break;
      load(p[0], r0 + step);
      work(p[1], r0);
      r0 += step;
    }
  } else {
    for (; r0 < a.rows; r0 += step) {
      Row p;
      load(p, r0);
      work(p, r0);
    }
  }
}

// The sums of the block's rows of threads for a column piece (those of slot 0 get them).
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

// How rows read gates.
enum Gate { kNoGate = 0, kOwnGate = 1, kSharedGate = 2 };

// w and cp = scale pw of a thread's columns, from LDS, whose reads are counted apart from the
// loads of the next row that are on their way.  The quarters of all pieces lie behind one another, so
// that a wavefront's 16-byte reads meet every bank once.
template <typename T, bool kShort>
struct Params {
  static constexpr int N = kPer<T>;
  const float* lds;
  int pieces;
  __device__ __forceinline__ void stage(const ResidualNormArgs& a, float* room, int n) {
    lds = room;
    pieces = n;
    for (int q = threadIdx.x; q < n; q += blockDim.x) {
      const Columns<T, kShort> col(q, static_cast<int>(a.D));
      for (int j = 0; j < N; ++j) {
        room[(j / 4 * n + q) * 4 + j % 4] = col.param(a.weight, j);
        room[((N / 4 + j / 4) * n + q) * 4 + j % 4] =
            col.param(a.post_weight, j) * col.param(a.scale, j);
      }
    }
    block_sync();
  }
  // Columns 4 h .. of a piece.
  __device__ __forceinline__ void get(int piece, int h, f32x4& w, f32x4& cp) const {
    __builtin_memcpy(&w, lds + (h * pieces + piece) * 4, 16);
    __builtin_memcpy(&cp, lds + ((N / 4 + h) * pieces + piece) * 4, 16);
  }
};

// A row's pieces as they lie in memory.
template <int VPT, int kGate, bool kSum>
struct BwdRow {
  uint4 g[VPT], t[VPT], y[VPT], z[kGate == kNoGate ? 1 : VPT], e[kSum ? VPT : 1];
  float rstd, post;
  static __device__ __forceinline__ void keep(uint4& u) {
    asm volatile("" : "+v"(u.x), "+v"(u.y), "+v"(u.z), "+v"(u.w));
  }
  // The row is widened twice; kept as it was loaded in between it takes half the registers.
  __device__ __forceinline__ void keep_packed() {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      keep(g[i]), keep(t[i]), keep(y[i]);
      if constexpr (kGate != kNoGate) keep(z[i]);
      if constexpr (kSum) keep(e[i]);
    }
  }
};

// Rows in `sets` of `rows` each that share a gate (one set of all rows where each has its own, or
// none has one); `split` blocks work on a set.  part: [gridDim.x, 2, D] the blocks' sums
// dw and S; gpart: [sets, split, D] those for the shared gates, where split > 1.
template <typename T, int TPR, int VPT, int kThreads, bool kShort, int kGate, bool kSum>
__global__ __launch_bounds__(kThreads, kMinWaves) void residual_norm_bwd_kernel(
    ResidualNormArgs a, ResidualNormGrads d, int64_t sets, int64_t rows, int64_t split, float* part,
    float* gpart) {
  constexpr int N = kPer<T>;
  using Col = Columns<T, kShort>;
  extern __shared__ __align__(16) float room[];
  __shared__ float red[2][kMaxWaves][4];
  __shared__ float cols[TPR ? 256 * N : 1];
  int flip = 0;
  const Rows<TPR> at;
  const int D = static_cast<int>(a.D);
  const float inv = 1.0f / static_cast<float>(D);
  const float* post_rstd = a.post_weight ? a.post_rstd : a.rstd;
  Params<T, kShort> params;
  params.stage(a, room, at.tpr * VPT);
  float dw[VPT][N], ds[VPT][N], dz[kGate == kSharedGate ? VPT : 1][N];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) dw[i][j] = ds[i][j] = 0.0f;
  using Row = BwdRow<VPT, kGate, kSum>;
  auto load = [&](Row& p, int64_t set, int64_t r0) __attribute__((always_inline)) {
    const int64_t r = set * rows + at.at(r0, rows);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const Col col(at.lane + at.tpr * i, D);
      p.t[i] = col.load(a.total, r);
      p.g[i] = col.load(d.dout, r);
      p.y[i] = col.load(a.y, r);
      if constexpr (kGate != kNoGate) p.z[i] = col.load(a.gate, kGate == kSharedGate ? set : r);
      if constexpr (kSum) p.e[i] = col.load(d.dtotal, r);
    }
    p.rstd = a.rstd[r];
    p.post = post_rstd[r];
  };
  auto work = [&](Row& p, int64_t set, int64_t r0) __attribute__((always_inline)) {
    const int64_t r = set * rows + at.at(r0, rows);
    const bool mine = TPR == 0 || r0 + at.slot < rows;
    const float rstd = p.rstd, post = a.post_weight ? p.post : 1.0f;
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int piece = at.lane + at.tpr * i;
      const Col col(piece, D);
#pragma unroll
      for (int h = 0; h < N / 4; ++h) {
        f32x4 w, cp;
        params.get(piece, h, w, cp);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = 4 * h + k;
          const float that = value<T>(p.t[i], j) * rstd;
          float wd = value<T>(p.g[i], j) * w[k];
          float q = cp[k] * (value<T>(p.y[i], j) * post);
          if constexpr (kGate != kNoGate) q *= gate_of(value<T>(p.z[i], j), a.silu).value;
          wd = col.own(j) ? wd : 0.0f;
          q = col.own(j) ? q : 0.0f;
          float e = rstd * wd;
          if constexpr (kSum) e += value<T>(p.e[i], j);
          s[0] = __builtin_fmaf(wd, that, s[0]);
          s[1] = __builtin_fmaf(e, q, s[1]);
          s[2] = __builtin_fmaf(that, q, s[2]);
        }
      }
    }
    p.keep_packed();
    sum_row<TPR>(s, red, flip);
    const float m1 = s[0] * inv;
    const float m2 = a.post_weight ? (s[1] - rstd * m1 * s[2]) * inv : 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int piece = at.lane + at.tpr * i;
      const Col col(piece, D);
      float dy[N], dr[N], dg[N];
#pragma unroll
      for (int h = 0; h < N / 4; ++h) {
        f32x4 w, cp;
        params.get(piece, h, w, cp);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = 4 * h + k;
          const float gv = value<T>(p.g[i], j), that = value<T>(p.t[i], j) * rstd;
          const float yh = value<T>(p.y[i], j) * post;
          Slope z = {1.0f, 0.0f};
          if constexpr (kGate != kNoGate) z = gate_of(value<T>(p.z[i], j), a.silu);
          float dt = rstd * (gv * w[k] - that * m1);
          if constexpr (kSum) dt += value<T>(p.e[i], j);
          const float dv = dt * z.value;
          dr[j] = dt;
          dy[j] = post * __builtin_fmaf(-yh, m2, dv * cp[k]);
          dg[j] = dt * (yh * cp[k]) * z.slope;
          dw[i][j] = mine ? __builtin_fmaf(gv, that, dw[i][j]) : dw[i][j];
          ds[i][j] = mine ? __builtin_fmaf(dv, yh, ds[i][j]) : ds[i][j];
          if constexpr (kGate == kSharedGate) dz[i][j] = mine ? dz[i][j] + dg[j] : dz[i][j];
        }
      }
      col.store(d.dresidual, r, dr);
      col.store(d.dy, r, dy);
      if constexpr (kGate == kOwnGate) col.store(d.dgate, r, dg);
    }
  };
  const int64_t part_of = blockIdx.x % split, set_step = gridDim.x / split;
  const int64_t first = part_of * at.per, step = split * at.per;
  for (int64_t set = blockIdx.x / split; set < sets; set += set_step) {
    if constexpr (kGate == kSharedGate) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) dz[i][j] = 0.0f;
    }
    int64_t r0 = first;
    if constexpr (kLoadsAhead<VPT, kThreads>) {
      // two rows' registers in turn: the next row is on its way while one is worked on
      Row p[2];
      load(p[0], set, r0);
      while (r0 < rows) {
        load(p[1], set, r0 + step);
        work(p[0], set, r0);
        r0 += step;
        if (r0 >= rows) break;
        load(p[0], set, r0 + step);
        work(p[1], set, r0);
        r0 += step;
      }
    } else {
      for (; r0 < rows; r0 += step) {
        Row p;
        load(p, set, r0);
        work(p, set, r0);
      }
    }
    if constexpr (kGate == kSharedGate) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const Col col(at.lane + at.tpr * i, D);
        if (sum_slots<TPR>(at, cols, dz[i])) {
          if (split == 1) col.store(d.dgate, set, dz[i]);
          else col.store_sums(gpart + (set * split + part_of) * D, dz[i]);
        }
      }
    }
  }
  float* dst = part + int64_t(blockIdx.x) * 2 * D;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const Col col(at.lane + at.tpr * i, D);
    if (sum_slots<TPR>(at, cols, dw[i])) col.store_sums(dst, dw[i]);
    if (sum_slots<TPR>(at, cols, ds[i])) col.store_sums(dst + D, ds[i]);
  }
}

// dw, and dpw and dscale from S: the sums of the rows of part (blockIdx.y: which), in a fixed order.
__global__ __launch_bounds__(1024) void residual_norm_sum_kernel(const float* __restrict__ part,
                                                                 int64_t blocks, int64_t D,
                                                                 const float* pw,
                                                                 const float* scale, float* dw,
                                                                 float* dpw, float* dscale) {
  __shared__ double m[16][64];
  const int col = threadIdx.x & 63, w = threadIdx.x >> 6, k = blockIdx.y;
  const int64_t c = int64_t(blockIdx.x) * 64 + col;
  double s = 0.0;
  if (c < D) {
#pragma unroll 8
    for (int64_t b = w; b < blocks; b += 16) s += part[(b * 2 + k) * D + c];
  }
  m[w][col] = s;
  block_sync();
  if (w != 0 || c >= D) return;
  for (int j = 1; j < 16; ++j) s += m[j][col];
  if (k == 0) {
    dw[c] = static_cast<float>(s);
  } else {
    if (dpw) dpw[c] = static_cast<float>(scale ? s * scale[c] : s);
    if (dscale) dscale[c] = static_cast<float>(pw ? s * pw[c] : s);
  }
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

// Calls f.template operator()<TPR, VPT, kThreads, kShort>(threads of a block, at most kThreads): a
// part of a wavefront for short rows, else the wavefronts that hold the row with VPT pieces a
// thread.
template <typename T, typename F>
hipError_t dispatch(int64_t D, F f) {
  const int64_t pieces = (D + kPer<T> - 1) / kPer<T>;
  if (D < kPer<T>) return f.template operator()<8, 1, 256, true>(256);
  if (pieces <= 8) return f.template operator()<8, 1, 256, false>(256);
  if (pieces <= 16) return f.template operator()<16, 1, 256, false>(256);
  if (pieces <= 32) return f.template operator()<32, 1, 256, false>(256);
  if (pieces <= 64) return f.template operator()<64, 1, 256, false>(256);
  auto threads = [&](int64_t vpt) {
    return static_cast<uint32_t>((pieces + 64 * vpt - 1) / (64 * vpt) * 64);
  };
  if (pieces <= 512) return f.template operator()<0, 1, 512, false>(threads(1));
  if (pieces <= 1024) return f.template operator()<0, 1, 1024, false>(threads(1));
  if (pieces <= 2048) return f.template operator()<0, 2, 1024, false>(threads(2));
  if constexpr (sizeof(T) == 4)
    if (pieces <= 4096) return f.template operator()<0, 4, 1024, false>(threads(4));
  return hipErrorInvalidValue;
}

// Blocks: what 256 compute units hold at about ten wavefronts each, since more of them only meet
// in the caches (32768 x 2560 bf16, 5 wavefronts a block: 210, 187, 170 us with 256, 384, 512 blocks and
// 176, 191 with 768, 1024; 8192 x 4096, 8 wavefronts: 65, 69 us with 256, 512), but not more than `most`.
// Rows of two and three wavefronts reach `most` before they reach ten, 3 blocks a unit forward and 2
// backward, which is not their best.  bf16 with 1 to 5 blocks a unit: 30000 x 640 (two wavefronts) 126, 88,
// 64, 53, 51 us and the gradient 163, 131, 95, 82, 84; 30000 x 1001 (two) 130, 93, 71, 65, 67 and 173, 139,
// 127, 131, 137; 30000 x 1536 (three; 3 blocks are ten wavefronts) 141, 101, 94 and 178, 156, 162.
int64_t blocks_for(uint32_t threads, int64_t most) {
  const int64_t fit = 10 / (threads / 64);
  return 256 * (fit < 1 ? 1 : fit > most ? most : fit);
}

template <typename T>
struct Fwd {
  const ResidualNormArgs& a;
  hipStream_t stream;
  template <int TPR, int VPT, int kThreads, bool kShort>
  hipError_t operator()(uint32_t threads) const {
    const int64_t per = TPR ? threads / TPR : 1;
    int64_t blocks = (a.rows + per - 1) / per;
    const int64_t most = blocks_for(threads, 3);
    if (blocks > most) blocks = most;
    const dim3 grid(static_cast<uint32_t>(blocks)), block(threads);
    if (a.gate)
      hipLaunchKernelGGL((residual_norm_kernel<T, TPR, VPT, kThreads, kShort, true>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((residual_norm_kernel<T, TPR, VPT, kThreads, kShort, false>), grid, block, 0, stream, a);
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
  template <int TPR, int VPT, int kThreads, bool kShort>
  hipError_t operator()(uint32_t threads) const {
    const int64_t per = TPR ? threads / TPR : 1;
    const int64_t most = blocks_for(threads, 2);
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
  if (dtype == MSSM_BFLOAT16) (void)dispatch<uint16_t>(D, MakeDeal<uint16_t>{rows, gate_rows, &d});
  else (void)dispatch<float>(D, MakeDeal<float>{rows, gate_rows, &d});
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
  template <int TPR, int VPT, int kThreads, bool kShort>
  hipError_t operator()(uint32_t threads) const {
    const dim3 grid(static_cast<uint32_t>(deal.blocks)), block(threads);
    const size_t lds = 2 * kPer<T> * sizeof(float) * VPT * (TPR ? TPR : threads);
    auto go = [&](auto gate, auto sum) {
      hipLaunchKernelGGL((residual_norm_bwd_kernel<T, TPR, VPT, kThreads, kShort, decltype(gate)::value,
                                                   decltype(sum)::value>),
                         grid, block, lds, stream, a, d, deal.sets, deal.rows, deal.split, part,
                         gpart);
    };
    auto with_sum = [&](auto gate) {
      if (d.dtotal) go(gate, std::true_type());
      else go(gate, std::false_type());
    };
    if (!a.gate) with_sum(std::integral_constant<int, kNoGate>());
    else if (a.gate_rows > 1) with_sum(std::integral_constant<int, kSharedGate>());
    else with_sum(std::integral_constant<int, kOwnGate>());
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
  return (static_cast<size_t>(d.blocks) * 2 + gates) * D * sizeof(float);
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
  float* gpart = part + deal.blocks * 2 * a.D;
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
  hipLaunchKernelGGL(residual_norm_sum_kernel, dim3(static_cast<uint32_t>((a.D + 63) / 64), 2),
                     dim3(1024), 0, stream, part, deal.blocks, a.D, a.post_weight, a.scale,
                     d.dweight, d.dpost_weight, d.dscale);
  return hipGetLastError();
}

}  // namespace mssm
