// Linear attention with a decay for each head on the matrix cores (gfx950):
// the pass that the forward and the backward kernels are instances of.
//
// Per sequence and head, with log decays g and a matrix state S [dk, dv],
//     S_t = exp(g_t) S_{t-1} + k_t v_t^T          o_t = scale S_t^T q_t.
// Cut into chunks of C tokens, with G_i = g_1 + .. + g_i inside the chunk and
// S the state before it:
//     o_i = scale exp(G_i) S^T q_i
//           + sum_{j <= i} scale exp(G_i - G_j) (q_i . k_j) v_j
//     S'  = exp(G_C) S + sum_j exp(G_C - G_j) k_j v_j^T
// which is five matrix products per chunk; only differences of G occur, so no
// factor exceeds 1 for decays at most 1.
//
// Backward.  With D_t = scale q_t do_t^T + exp(g_{t+1}) D_{t+1} (the adjoint
// of S_t), dq_t = scale S_t do_t, dv_t = D_t^T k_t, dk_t = D_t v_t.  So dq is
// the same operator on (do, v, k) with the state S^T, and dv, dk are the
// operator run backwards in time on (k, q, do) and (v, do, q):
//     o_j = exp(G_C - G_j) D^T x_j + sum_{i >= j} scale exp(G_i - G_j) (x_j . y_i) z_i
//     D'  = exp(G_C) D + sum_i scale exp(G_i) y_i z_i^T
// One kernel, la_pass, takes the three roles x (query), y (key), z (value) and
// the direction.
//
// dg_t = exp(g_t) <D_t, S_{t-1}> is what passes from tokens before t to tokens
// from t on.  Inside a chunk that is
//     sum_{i >= t} q_i . dqc_i + sum_{j < t <= i} W_ij + sum_{j < t} k_j . dkc_j
//     + exp(G_C) <D, S>
// where dqc, dkc are the parts of dq, dk that come through the states S and D
// and W_ij = scale exp(G_i - G_j)(q_i . k_j)(do_i . v_j).  The usual suffix sum
// of q.dq - k.dk over the whole sequence is the same number, but as a small
// difference of sums that grow with the length; here the sums stay inside a
// segment, whose end value <D, S> is computed from the two states themselves.
//
// Layout on the compute unit.  A block of four wavefronts owns one segment of
// one head.  Wavefront w owns 16 NT columns of the value dimension: its part
// of S [DA, 16 NT] stays in the accumulator registers for the whole segment,
// and is used as a matrix operand straight from them: a 16 x 16 result holds
// four consecutive rows per lane, and the rows of a matrix product's sum may
// be taken in any order if both operands take the same, so two result tiles
// are one 32-row operand without a trip through LDS.  The tiles of x, y and z
// are staged in LDS row by row; products that sum over tokens read them
// transposed (ds_read_b64_tr_b16).  The C x C products are shared out over the
// wavefronts by rows and exchanged through LDS.
//
// The float32 form is the same code: a fragment is then eight float32 values
// per lane and a product eight v_mfma_f32_16x16x4_f32, whose four sums per
// instruction take the fragments' values in the same order on both sides.
//
// Rounding.  Products of bfloat16 inputs accumulate in float32.  The decayed
// scores and the state are rounded to bfloat16 where they are operands of the
// output's products (the output is rounded to bfloat16 itself); where float32
// results depend on them (the state's own update, dg) the operand is split in
// a bfloat16 pair, hi + lo, about 16 bits (relative error about 7e-7 on
// average).  Decays, their sums (float64 inside a chunk, kept as a float32
// pair) and the state are 32 bits or more.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "la_args.h"
#include "scan_device.h"

namespace mssm {
namespace la {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// ---- fragments --------------------------------------------------------------------------------

// Eight values of one row (or column) per lane: lane l holds row l % 16 of a
// 16-row tile and eight of the 32 terms of the sum.
template <typename T>
struct Frag;
template <>
struct Frag<uint16_t> {
  bf16x8 v;
};
template <>
struct Frag<float> {
  float v[8];
};

__device__ __forceinline__ void mma(f32x4& acc, const Frag<uint16_t>& a, const Frag<uint16_t>& b) {
  acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4& acc, const Frag<float>& a, const Frag<float>& b) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], acc, 0, 0, 0);
}

// Eight consecutive values of an LDS row.
__device__ __forceinline__ Frag<uint16_t> frag_row(const uint16_t* p) {
  Frag<uint16_t> f;
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  __builtin_memcpy(&f.v, &u, 16);
  return f;
}
__device__ __forceinline__ Frag<float> frag_row(const float* p) {
  Frag<float> f;
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) f.v[e] = a[e], f.v[4 + e] = b[e];
  return f;
}

// Values 0..3 and 16..19 from p: the order in which two 16-row result tiles
// hold the rows of a 32-row operand.
__device__ __forceinline__ Frag<uint16_t> frag_split(const uint16_t* p) {
  Frag<uint16_t> f;
  uint2 u[2] = {*reinterpret_cast<const uint2*>(p), *reinterpret_cast<const uint2*>(p + 16)};
  __builtin_memcpy(&f.v, u, 16);
  return f;
}
__device__ __forceinline__ Frag<float> frag_split(const float* p) {
  Frag<float> f;
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 16);
#pragma unroll
  for (int e = 0; e < 4; ++e) f.v[e] = a[e], f.v[4 + e] = b[e];
  return f;
}

// Column of an LDS tile with row pitch P over eight consecutive rows r0 + 8
// (lane / 16) ..: lane l gets the column of its index l % 16, where indices
// 4 c .. 4 c + 3 are the columns c0 + cstep c ...  For bfloat16 the transposing
// LDS read gives 16 lanes four rows of sixteen columns: lane l % 16 addresses
// four columns of one row and receives one column of the four rows.
template <int P>
__device__ __forceinline__ Frag<uint16_t> frag_col(const uint16_t* t, int r0, int c0, int cstep,
                                                   int lane) {
  using lds_ptr = __attribute__((address_space(3))) s16x4*;
  const int r = r0 + 8 * (lane >> 4) + ((lane & 15) >> 2), c = c0 + cstep * (lane & 3);
  const s16x4 u[2] = {
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(t + r * P + c)),
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(t + (r + 4) * P + c))};
  Frag<uint16_t> f;
  __builtin_memcpy(&f.v, u, 16);
  return f;
}
template <int P>
__device__ __forceinline__ Frag<float> frag_col(const float* t, int r0, int c0, int cstep,
                                                int lane) {
  Frag<float> f;
  const int c = c0 + cstep * ((lane & 15) >> 2) + (lane & 3);
#pragma unroll
  for (int e = 0; e < 8; ++e) f.v[e] = t[(r0 + 8 * (lane >> 4) + e) * P + c];
  return f;
}

__device__ __forceinline__ void pack(Frag<uint16_t>& f, const float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f.v[e] = static_cast<__bf16>(v[e]);
}
__device__ __forceinline__ void pack(Frag<float>& f, const float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f.v[e] = v[e];
}
__device__ __forceinline__ void unpack(const Frag<uint16_t>& f, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(f.v[e]);
}
__device__ __forceinline__ void unpack(const Frag<float>& f, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = f.v[e];
}
// hi and lo with v = hi + lo to about 16 bits (float32: hi = v alone).
__device__ __forceinline__ void split(const float (&v)[8], Frag<uint16_t>& hi, Frag<uint16_t>& lo) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    hi.v[e] = static_cast<__bf16>(v[e]);
    lo.v[e] = static_cast<__bf16>(v[e] - static_cast<float>(hi.v[e]));
  }
}

__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
  bf16x2 a, b;
  a[0] = static_cast<__bf16>(v[0]), a[1] = static_cast<__bf16>(v[1]);
  b[0] = static_cast<__bf16>(v[2]), b[1] = static_cast<__bf16>(v[3]);
  uint2 u;
  __builtin_memcpy(&u.x, &a, 4);
  __builtin_memcpy(&u.y, &b, 4);
  __builtin_memcpy(p, &u, 8);
}
__device__ __forceinline__ void store4(float* p, f32x4 v) { __builtin_memcpy(p, &v, 16); }

__device__ __forceinline__ void lds_store4(uint16_t* p, f32x4 v) {
  uint2 u;
  store4(reinterpret_cast<uint16_t*>(&u), v);
  *reinterpret_cast<uint2*>(p) = u;
}
__device__ __forceinline__ void lds_store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }

// ---- a sequence's place -------------------------------------------------------------------------

struct Place {
  int64_t start = 0, len = 0;   // the segment's tokens
  int64_t seq = 0;
  int64_t local = 0, count = 0; // which of the sequence's segments
  bool ok = false;
};

// The segment of slot `slot`.  Packed sequences take slots start / seg_len + s
// on: at least as many as sequence s needs, whatever the lengths, and known
// without a pass over them.  Offsets are clamped to the token count, so no
// value of theirs leads outside the tensors.
__device__ __forceinline__ Place place_of(const Grid& p, int64_t slot) {
  Place r;
  if (!p.offsets) {
    r.seq = slot / p.segs;
    r.local = slot - r.seq * p.segs;
    r.count = p.segs;
    r.start = r.seq * p.L + r.local * p.seg_len;
    r.len = min(p.seg_len, p.L - r.local * p.seg_len);
    r.ok = true;
    return r;
  }
  auto at = [&](int64_t s) {
    const int64_t o = p.offsets[s];
    return o < 0 ? int64_t(0) : (o > p.tokens ? p.tokens : o);
  };
  int64_t lo = 0, hi = p.seqs - 1;          // the last sequence whose first slot is <= slot
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (at(mid) / p.seg_len + mid <= slot) lo = mid; else hi = mid - 1;
  }
  const int64_t a = at(lo), b = max(at(lo + 1), a);
  r.seq = lo;
  r.local = slot - (a / p.seg_len + lo);
  r.count = max((b - a + p.seg_len - 1) / p.seg_len, int64_t(1));
  r.start = a + r.local * p.seg_len;
  r.len = min(p.seg_len, b - r.start);
  r.ok = r.local >= 0 && r.local < r.count;
  return r;
}

// Blocks go to the eight dies in turn; each die takes a contiguous run of the
// (slot, head) pairs, heads fastest, so that heads that share queries and keys
// and the lines of g meet in one L2.
__device__ __forceinline__ uint32_t logical_block() {
  const uint32_t n = gridDim.x, b = blockIdx.x;
  const uint32_t q = n / 8, r = n % 8, die = b % 8;
  return die * q + min(die, r) + b / 8;
}

// ---- tiles ----------------------------------------------------------------------------------------

// C rows of D values, staged through registers: fetch issues the loads, stash
// writes them to LDS (row pitch P).  Rows past n and columns past d are zero.
template <typename T, int C, int D, int P>
struct Tile {
  static constexpr int kPer = 16 / sizeof(T);              // values in a 16-byte piece
  static constexpr int kRowPieces = D / kPer;
  static constexpr int kPieces = C * kRowPieces / kThreads;
  static_assert(C * kRowPieces % kThreads == 0, "whole pieces per thread");
  uint4 v[kPieces];

  __device__ __forceinline__ void fetch(const T* base, int64_t row, int n, int d, bool vec) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = threadIdx.x + kThreads * i;
      const int r = p / kRowPieces, c = (p % kRowPieces) * kPer;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < n && c < d) {
        const T* src = base + r * row + c;
        if (vec) {
          v[i] = *reinterpret_cast<const uint4*>(src);
        } else {
          T e[kPer];
#pragma unroll
          for (int j = 0; j < kPer; ++j) e[j] = src[j];
          __builtin_memcpy(&v[i], e, 16);
        }
      }
    }
  }
  __device__ __forceinline__ void stash(T* lds) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = threadIdx.x + kThreads * i;
      const int r = p / kRowPieces, c = (p % kRowPieces) * kPer;
      *reinterpret_cast<uint4*>(lds + r * P + c) = v[i];
    }
  }
};

// Decays of one chunk, in LDS.  Log decays are in powers of two.
template <int C>
struct Decay {
  float hi[C], lo[C];      // G, inclusive, as a float32 pair
  float ein[C];            // factor of the carried state at each token
  float w[C];              // factor of each token in the state's update
  float all;               // exp(G_C)
};

template <int C, bool kRev>
__device__ __forceinline__ void decays(Decay<C>& d, float g, float scale, int lane) {
  // far below what exp can represent, so that a decay to zero (minus infinity)
  // leaves the differences finite
  g = g < -1e4f ? -1e4f : g;
  double s = static_cast<double>(g) * 1.4426950408889634074;
#pragma unroll
  for (int o = 1; o < C; o <<= 1) {
    const double u = __shfl_up(s, o, 64);
    if (lane >= o) s += u;
  }
  const double total = __shfl(s, C - 1, 64);
  if (lane < C) {
    const float hi = static_cast<float>(s);
    d.hi[lane] = hi;
    d.lo[lane] = static_cast<float>(s - static_cast<double>(hi));
    const float in = fast_exp2(hi), out = fast_exp2(static_cast<float>(total - s));
    d.ein[lane] = kRev ? out : scale * in;
    d.w[lane] = kRev ? scale * in : out;
    if (lane == 0) d.all = fast_exp2(static_cast<float>(total));
  }
}

// ---- the pass ----------------------------------------------------------------------------------------

// kDot 0: nothing more.  1 (dq): also W and q . dqc, as one sum u for each
// token.  2 (dk): also k . dkc, and dg from it and u.
// kOut false: only the state over the segment (no x, no output).
// kExact: the state enters the output's product as a bfloat16 pair.
template <typename T, int C, int DA, int NT, bool kRev, bool kOut, int kDot>
struct Shape {
  static constexpr int TB = 64 * NT;                        // columns of z
  static constexpr int kPad = 32 / sizeof(T);               // 32 bytes
  static constexpr int PA = DA + kPad, PB = TB + kPad, PP = C + 16 / sizeof(T);
  struct Lds {
    T x[kOut ? C * PA : 8];
    T y[C * PA];
    T z[C * PB];
    T e[kDot == 1 ? C * PB : 8];
    T p[kOut ? C * PP : 8];
    Decay<C> d;
    float dot[kDot ? 4 : 1][C];
    float col[kDot == 1 ? 4 : 1][C];
    float sum[kDot ? C : 1];
  };
};

template <typename T, int C, int DA, int NT, bool kRev, bool kOut, int kDot>
__global__ __launch_bounds__(kThreads) void la_pass(PassArgs p) {
  using S = Shape<T, C, DA, NT, kRev, kOut, kDot>;
  constexpr bool kBf16 = sizeof(T) == 2;
  constexpr bool kExact = kBf16 && kDot != 0;
  constexpr int NR = C / 16, NK = C / 32, NM = DA / 16;
  constexpr int PA = S::PA, PB = S::PB, PP = S::PP;
  __shared__ __align__(16) typename S::Lds m;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;

  const uint32_t block = logical_block();
  const int64_t slot = block / p.heads;
  const int h = block % p.heads;
  const Place at = place_of(p.grid, slot);
  if (!at.ok) {
    if constexpr (kDot == 2) {
      if (p.head_part && tid == 0) p.head_part[block] = 0.0f;
    }
    return;
  }
  // a state-only pass has nothing to do for the segment that no other follows
  const bool last_seg = kRev ? at.local == 0 : at.local == at.count - 1;
  const bool first_seg = kRev ? at.local == at.count - 1 : at.local == 0;
  if (!kOut && last_seg && !p.every_segment) return;

  // columns of this wavefront: with two tiles, lane group g4's rows 4 g4 + r of
  // both are the eight consecutive columns 8 g4 + 4 t + r
  constexpr int kStep = NT == 2 ? 8 : 4;
  const int c_wave = 16 * NT * wave;
  auto col_of = [&](int t, int c) { return c_wave + kStep * (c >> 2) + 4 * t + (c & 3); };

  const T* X = kOut ? static_cast<const T*>(p.x.p) + at.start * p.x.row + (h / p.x.div) * int64_t(p.dA) : nullptr;
  const T* Y = static_cast<const T*>(p.y.p) + at.start * p.y.row + (h / p.y.div) * int64_t(p.dA);
  const T* Z = static_cast<const T*>(p.z.p) + at.start * p.z.row + (h / p.z.div) * int64_t(p.dB);
  const T* E = kDot ? static_cast<const T*>(p.e.p) + at.start * p.e.row + (h / p.e.div) * int64_t(p.dB) : nullptr;
  const float* G = p.g + (p.g_row ? at.start * p.g_row : 0) + h;
  const int64_t sh = (at.seq * p.heads + h) * (int64_t(p.dA) * p.dB);        // per sequence
  const int64_t wh = (slot * p.heads + h) * (int64_t(p.dA) * p.dB);          // per segment

  // the state: rows 16 mt + 4 g4 + r of dA, column col_of(t, l16)
  f32x4 s[NM][NT];
  {
    const float* init = !kOut ? nullptr
                        : p.seg_states ? p.seg_states + wh
                        : p.init ? p.init + sh : nullptr;
#pragma unroll
    for (int mt = 0; mt < NM; ++mt)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int c = col_of(t, l16);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int a = 16 * mt + 4 * g4 + r;
          s[mt][t][r] = init && a < p.dA && c < p.dB ? init[a * p.sA + c * p.sB] : 0.0f;
        }
      }
  }

  const int chunks = static_cast<int>((at.len + C - 1) / C);
  const float scale = p.scale;
  Tile<T, C, DA, PA> tx, ty;
  Tile<T, C, S::TB, PB> tz, te;
  float gv = 0.0f;
  auto fetch = [&](int c) {
    const int64_t t0 = int64_t(c) * C;
    const int n = static_cast<int>(min(at.len - t0, int64_t(C)));
    if constexpr (kOut) tx.fetch(X + t0 * p.x.row, p.x.row, n, p.dA, p.x.vec);
    ty.fetch(Y + t0 * p.y.row, p.y.row, n, p.dA, p.y.vec);
    tz.fetch(Z + t0 * p.z.row, p.z.row, n, p.dB, p.z.vec);
    if constexpr (kDot == 1) te.fetch(E + t0 * p.e.row, p.e.row, n, p.dB, p.e.vec);
    if (wave == 0) gv = lane < n ? G[p.g_row ? (t0 + lane) * p.g_row : 0] : 0.0f;
  };

  // dg: what crosses the segment's end, <D, S> of the states there
  float edge = 0.0f, head_sum = 0.0f;
  if constexpr (kDot == 2) {
    const float* ds = p.seg_states ? p.seg_states + wh : nullptr;
    const float* ss = p.fwd_states ? p.fwd_states + wh + int64_t(p.heads) * p.dA * p.dB : nullptr;
    if (first_seg) ds = p.init ? p.init + sh : nullptr, ss = p.fwd_last ? p.fwd_last + sh : nullptr;
    if (ds && ss) {
      float part = 0.0f;
      const int n = p.dA * p.dB;
      for (int i = tid; i < n; i += kThreads) part = __builtin_fmaf(ds[i], ss[i], part);
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) part += __shfl_xor(part, o, 64);
      if (lane == 0) m.dot[0][wave] = part;
      block_sync();
      edge = (m.dot[0][0] + m.dot[0][1]) + (m.dot[0][2] + m.dot[0][3]);
      block_sync();
    }
  }

  if (chunks > 0) fetch(kRev ? chunks - 1 : 0);
  for (int it = 0; it < chunks; ++it) {
    const int ck = kRev ? chunks - 1 - it : it;
    const int64_t t0 = int64_t(ck) * C;
    const int n = static_cast<int>(min(at.len - t0, int64_t(C)));
    if constexpr (kOut) tx.stash(m.x);
    ty.stash(m.y);
    tz.stash(m.z);
    if constexpr (kDot == 1) te.stash(m.e);
    if (wave == 0) decays<C, kRev>(m.d, gv, scale, lane);
    block_sync();
    if (it + 1 < chunks) fetch(kRev ? ck - 1 : ck + 1);

    f32x4 acc[NR][NT];
    if constexpr (kOut) {
      // the C x C products of this wavefront's part: tiles (rows of x, rows of
      // y), each result a lane's column i (row of x) and four rows j of y
      constexpr int kWaveTiles = NR == 4 ? 4 : 1;
      const int rt = NR == 4 ? wave : wave >> 1;
      const int i = 16 * rt + l16;
      const float gi = m.d.hi[i], gil = m.d.lo[i];
      float row_sum = 0.0f;
#pragma unroll
      for (int u = 0; u < kWaveTiles; ++u) {
        const int ct = NR == 4 ? u : wave & 1;
        const bool live = kRev ? ct >= rt : ct <= rt;
        f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f}, b = {0.0f, 0.0f, 0.0f, 0.0f};
        f32x4 wsum = {0.0f, 0.0f, 0.0f, 0.0f};
        if (live) {
#pragma unroll
          for (int k = 0; k < DA / 32; ++k)
            mma(a, frag_row(m.y + (16 * ct + l16) * PA + 32 * k + 8 * g4),
                frag_row(m.x + i * PA + 32 * k + 8 * g4));
          if constexpr (kDot == 1) {
#pragma unroll
            for (int k = 0; k < S::TB / 32; ++k)
              mma(b, frag_row(m.z + (16 * ct + l16) * PB + 32 * k + 8 * g4),
                  frag_row(m.e + i * PB + 32 * k + 8 * g4));
          }
          const int j0 = 16 * ct + 4 * g4;
          const f32x4 gj = *reinterpret_cast<const f32x4*>(&m.d.hi[j0]);
          const f32x4 gjl = *reinterpret_cast<const f32x4*>(&m.d.lo[j0]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool in = kRev ? j0 + r >= i : j0 + r <= i;
            const float diff = (gi - gj[r]) + (gil - gjl[r]);
            const float f = scale * fast_exp2(kRev ? -diff : diff);
            a[r] = in ? a[r] * f : 0.0f;
            if constexpr (kDot == 1) wsum[r] = in && j0 + r != i ? a[r] * b[r] : 0.0f;
          }
          if constexpr (kDot == 1) row_sum += (wsum[0] + wsum[1]) + (wsum[2] + wsum[3]);
        }
        lds_store4(m.p + i * PP + 16 * ct + 4 * g4, a);
        if constexpr (kDot == 1) {
          // sums over this wavefront's 16 rows i, for each of the four j
#pragma unroll
          for (int o = 1; o < 16; o <<= 1)
#pragma unroll
            for (int r = 0; r < 4; ++r) wsum[r] += __shfl_xor(wsum[r], o, 64);
          if (l16 == 0) *reinterpret_cast<f32x4*>(&m.col[NR == 4 ? wave : rt][16 * ct + 4 * g4]) = wsum;
        }
      }
      if constexpr (kDot == 1) {
        row_sum += __shfl_xor(row_sum, 16, 64);
        row_sum += __shfl_xor(row_sum, 32, 64);
        // with two row tiles, the two wavefronts of a row tile hold one column
        // tile each: their sums are kept apart
        if (g4 == 0) {
          if constexpr (NR == 4) m.sum[i] = row_sum;
          else m.col[2 + (wave & 1)][i] = row_sum;
        }
      }

      // the carried part: x S
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < DA / 32; ++k) {
        Frag<T> hi[NT], lo[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float v[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = s[2 * k][t][r], v[4 + r] = s[2 * k + 1][t][r];
          if constexpr (kExact) split(v, hi[t], lo[t]);
          else pack(hi[t], v);
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const Frag<T> xf = frag_split(m.x + (16 * r + l16) * PA + 32 * k + 4 * g4);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma(acc[r][t], hi[t], xf);
            if constexpr (kExact) mma(acc[r][t], lo[t], xf);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float f = m.d.ein[16 * r + l16];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] *= f;
      }
      if constexpr (kDot != 0) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int i = 16 * r + l16;
          float dot = 0.0f;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const int c = col_of(t, 4 * g4);
            float ev[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (kDot == 1) {
#pragma unroll
              for (int q = 0; q < 4; ++q) ev[q] = to_float(m.e[i * PB + c + q]);
            } else if (i < n && c < p.dB) {
              T raw[4];
              __builtin_memcpy(raw, E + (t0 + i) * p.e.row + c, sizeof(raw));
#pragma unroll
              for (int q = 0; q < 4; ++q) ev[q] = to_float(raw[q]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) dot = __builtin_fmaf(acc[r][t][q], ev[q], dot);
          }
          dot += __shfl_xor(dot, 16, 64);
          dot += __shfl_xor(dot, 32, 64);
          if (g4 == 0) m.dot[wave][i] = dot;
        }
      }
      block_sync();
    }

    // z by columns, for the scores' product and for the state
    Frag<T> zf[NK][NT];
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        zf[k][t] = frag_col<PB>(m.z, 32 * k, c_wave + 4 * t, kStep, lane);

    if constexpr (kOut) {
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          if (kRev ? k < r / 2 : k > r / 2) continue;
          const Frag<T> pf = frag_row(m.p + (16 * r + l16) * PP + 32 * k + 8 * g4);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma(acc[r][t], zf[k][t], pf);
        }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int i = 16 * r + l16;
        if (i >= n) continue;
        const int64_t row = ((at.start + t0 + i) * p.heads + h) * int64_t(p.dB);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int c = col_of(t, 4 * g4);
          if (c >= p.dB) continue;
          if (p.out_f32) store4(static_cast<float*>(p.out) + row + c, acc[r][t]);
          else store4(static_cast<T*>(p.out) + row + c, acc[r][t]);
        }
      }
      if constexpr (kDot == 1) {
        if (tid < C && tid < n) {
          float u = (m.dot[0][tid] + m.dot[1][tid]) + (m.dot[2][tid] + m.dot[3][tid]);
          float rows, cols = 0.0f;
          const int rt = tid >> 4;          // column sums exist for row tiles >= this one
          if constexpr (NR == 4) {
            rows = m.sum[tid];
            for (int q = rt; q < 4; ++q) cols += m.col[q][tid];
          } else {
            rows = m.col[2][tid] + (rt == 1 ? m.col[3][tid] : 0.0f);
            for (int q = rt; q < 2; ++q) cols += m.col[q][tid];
          }
          p.u[(at.start + t0 + tid) * p.heads + h] = u + (rows - cols);
        }
      }
      if constexpr (kDot == 2) {
        if (wave == 0) {
          const int64_t ti = (at.start + t0 + lane) * p.heads + h;
          const bool in = lane < n;
          const float kd = lane < C ? (m.dot[0][lane] + m.dot[1][lane]) + (m.dot[2][lane] + m.dot[3][lane]) : 0.0f;
          const float u = in ? p.u[ti] : 0.0f;
          float before = kd, after = u;     // inclusive sums up to, and from, this token
#pragma unroll
          for (int o = 1; o < 64; o <<= 1) {
            const float a = __shfl_up(before, o, 64), b = __shfl_down(after, o, 64);
            if (lane >= o) before += a;
            if (lane + o < 64) after += b;
          }
          const float through = edge - __shfl(before, 63, 64);
          const float prior = __shfl_up(before, 1, 64);
          const float dg = after + (lane > 0 ? prior : 0.0f) + through;
          edge = through + __shfl(after, 0, 64);
          if (in) {
            if (p.dg) p.dg[ti] = dg;
            head_sum += dg;
          }
        }
      }
    }

    // the state after the chunk
    const bool more = it + 1 < chunks || !kOut || (last_seg && p.last);
    if (more) {
      const float all = m.d.all;
#pragma unroll
      for (int mt = 0; mt < NM; ++mt)
#pragma unroll
        for (int t = 0; t < NT; ++t) s[mt][t] *= all;
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        Frag<T> hi[NT], lo[NT];
        float w[8];
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(&m.d.w[32 * k + 8 * g4]);
        const f32x4 w1 = *reinterpret_cast<const f32x4*>(&m.d.w[32 * k + 8 * g4 + 4]);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = w0[e], w[4 + e] = w1[e];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float v[8];
          unpack(zf[k][t], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= w[e];
          if constexpr (kBf16) split(v, hi[t], lo[t]);
          else pack(hi[t], v);
        }
#pragma unroll
        for (int mt = 0; mt < NM; ++mt) {
          const Frag<T> yf = frag_col<PA>(m.y, 32 * k, 16 * mt, 4, lane);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma(s[mt][t], yf, hi[t]);
            if constexpr (kBf16) mma(s[mt][t], yf, lo[t]);
          }
        }
      }
    }
    if constexpr (!kOut) {
      if (tid == 0) head_sum += m.d.hi[C - 1];     // the segment's log decay
    }
    block_sync();
  }

  if constexpr (kDot == 2) {
    if (p.head_part && wave == 0) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) head_sum += __shfl_xor(head_sum, o, 64);
      if (lane == 0) p.head_part[slot * p.heads + h] = head_sum;
    }
  }
  float* dst = nullptr;
  if constexpr (kOut) {
    if (last_seg && p.last) dst = p.last + sh;
  } else {
    dst = p.seg_out + wh;
    if (tid == 0) p.seg_decay[slot * p.heads + h] = fast_exp2(head_sum);
  }
  if (!dst) return;
#pragma unroll
  for (int mt = 0; mt < NM; ++mt)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = col_of(t, l16);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int a = 16 * mt + 4 * g4 + r;
        if (a < p.dA && c < p.dB) dst[a * p.sA + c * p.sB] = s[mt][t][r];
      }
    }
}

}  // namespace la
}  // namespace mssm
