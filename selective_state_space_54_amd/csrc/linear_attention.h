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
// chunk, and <D, S> is computed from the two states themselves, for every fourth
// chunk from the last (the forward states are kept for those); between them it
// follows from what q.dqc and k.dkc add and take away.
//
// Layout on the compute unit.  A block of four wavefronts owns one segment of
// one head.  Wavefront w owns 16 NT columns of the value dimension: its part
// of S [DA, 16 NT] stays in registers for the whole segment, and is used as a
// matrix operand straight from them: a 16 x 16 result holds four consecutive
// rows per lane, and the terms of a matrix product's sum may be taken in any
// order if both operands take the same, so two result tiles are one 32-row
// operand without a trip through LDS.  The tiles of x, y and z
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
// output's products (the output is rounded to bfloat16 itself), except the
// scores of the 16 x 16 tiles on the diagonal, which keep 16 bits: where decays
// are strong, or a sequence begins, a token's output is little more than its own
// term, and that rounding would not average out.  Where float32
// results depend on them (the state's own update, dg) the operand is split in
// three bfloat16 parts, 24 bits.  Decays, their sums (float64 inside a chunk,
// kept as a float32 pair) and the state are 32 bits or more.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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

// Where an LDS tile of D columns keeps value c of row r.  A row's 16-byte
// pieces are permuted by the row's number, so that the 8-byte reads of 32 lanes
// (16 rows of two neighbouring halves, or 8 rows of two neighbouring pieces)
// fall on all 64 banks once.  Reads of 16 bytes would take half the
// instructions, but their measured rate is a third of the 8-byte reads' (75
// against 256 bytes a cycle).
template <typename T, int D>
__device__ __forceinline__ int tile_at(int r, int c) {
  constexpr int kPer = 16 / sizeof(T);
  const int f = D / kPer > 8 ? (r & 7) << 1 | (r >> 3 & 1) : r >> 1 & 7;
  return r * D + ((c / kPer) ^ f) * kPer + c % kPer;
}

// A fragment's eight terms are numbers 0 .. 3 and 16 .. 19 from 4 (lane / 16) of
// a run of 32: the order in which two 16-row results hold the rows of an operand.
__device__ __forceinline__ Frag<uint16_t> frag_of(uint2 a, uint2 b) {
  Frag<uint16_t> f;
  const uint2 u[2] = {a, b};
  __builtin_memcpy(&f.v, u, 16);
  return f;
}
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ Frag<float> frag_of(const float* a, const float* b) {
  Frag<float> f;
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const f32x2 u = *reinterpret_cast<const f32x2*>(a + e);
    const f32x2 v = *reinterpret_cast<const f32x2*>(b + e);
    f.v[e] = u[0], f.v[e + 1] = u[1], f.v[4 + e] = v[0], f.v[5 + e] = v[1];
  }
  return f;
}

// An 8-byte LDS read of its own: the compiler would join the reads of two rows
// into one instruction, whose four registers are then no operand of either.
__device__ __forceinline__ uint2 lds_read8(const uint16_t* p) {
  using lds_ptr = const volatile __attribute__((address_space(3))) u32x2*;
  const u32x2 u = *(lds_ptr)(p);
  return make_uint2(u.x, u.y);
}

// Terms c .. c + 31 of row r of a tile; c = 32 k + 4 (lane / 16).
template <int D>
__device__ __forceinline__ Frag<uint16_t> frag_row(const uint16_t* t, int r, int c) {
  return frag_of(lds_read8(t + tile_at<uint16_t, D>(r, c)),
                 lds_read8(t + tile_at<uint16_t, D>(r, c + 16)));
}
template <int D>
__device__ __forceinline__ Frag<float> frag_row(const float* t, int r, int c) {
  return frag_of(t + tile_at<float, D>(r, c), t + tile_at<float, D>(r, c + 16));
}
// The same of a plain row.
__device__ __forceinline__ Frag<uint16_t> frag_at(const uint16_t* p) {
  return frag_of(lds_read8(p), lds_read8(p + 16));
}
__device__ __forceinline__ Frag<float> frag_at(const float* p) { return frag_of(p, p + 16); }

// Terms r0 .. r0 + 31 down a column of a tile: lane l gets the column of its
// index l % 16, where indices 4 c .. 4 c + 3 are the columns c0 + kStep c ...
// For bfloat16 the transposing LDS read gives 16 lanes four rows of sixteen
// columns: lane l % 16 addresses four columns of one row and receives one column
// of the four rows.
template <int D, int kStep>
__device__ __forceinline__ Frag<uint16_t> frag_col(const uint16_t* t, int r0, int c0, int lane) {
  using lds_ptr = __attribute__((address_space(3))) s16x4*;
  const int r = r0 + 4 * (lane >> 4) + ((lane & 15) >> 2), c = c0 + kStep * (lane & 3);
  const s16x4 u[2] = {
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(t + tile_at<uint16_t, D>(r, c))),
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(t + tile_at<uint16_t, D>(r + 16, c)))};
  Frag<uint16_t> f;
  __builtin_memcpy(&f.v, u, 16);
  return f;
}
template <int D, int kStep>
__device__ __forceinline__ Frag<float> frag_col(const float* t, int r0, int c0, int lane) {
  Frag<float> f;
  const int c = c0 + kStep * ((lane & 15) >> 2) + (lane & 3);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    f.v[e] = t[tile_at<float, D>(r0 + 4 * (lane >> 4) + 16 * (e >> 2) + (e & 3), c)];
  return f;
}

// Four consecutive values.
__device__ __forceinline__ f32x4 lds_load4(const uint16_t* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
               __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u)};
}
__device__ __forceinline__ f32x4 lds_load4(const float* p) {
  return *reinterpret_cast<const f32x4*>(p);
}

// Two values rounded to bfloat16, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  bf16x2 v;
  v[0] = static_cast<__bf16>(a);
  v[1] = static_cast<__bf16>(b);
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float low_half(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high_half(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

__device__ __forceinline__ void unpack(const Frag<uint16_t>& f, float (&v)[8]) {
  uint32_t u[4];
  __builtin_memcpy(u, &f.v, 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = low_half(u[i]), v[2 * i + 1] = high_half(u[i]);
}
__device__ __forceinline__ void unpack(const Frag<float>& f, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = f.v[e];
}

// v as a sum of N bfloat16 parts, each the rounding of what is left: to about
// 17 bits with two, exactly float32 with three.  (float32: v itself.)
template <int N>
__device__ __forceinline__ void split(const float (&v)[8], Frag<uint16_t> (&part)[N]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
    for (int q = 0; q < N; ++q) {
      uint32_t u = pack2(a, b);
      asm("" : "+v"(u));      // read the halves back, rather than round a and b once more
      __builtin_memcpy(reinterpret_cast<char*>(&part[q].v) + 4 * i, &u, 4);
      a -= low_half(u);
      b -= high_half(u);
    }
  }
}
template <int N>
__device__ __forceinline__ void split(const float (&v)[8], Frag<float> (&part)[N]) {
  static_assert(N == 1, "float32 needs one part");
#pragma unroll
  for (int e = 0; e < 8; ++e) part[0].v[e] = v[e];
}

__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
  const uint2 u = {pack2(v[0], v[1]), pack2(v[2], v[3])};
  __builtin_memcpy(p, &u, 8);
}
__device__ __forceinline__ void store4(float* p, f32x4 v) { __builtin_memcpy(p, &v, 16); }

__device__ __forceinline__ void lds_store4(uint16_t* p, f32x4 v) {
  *reinterpret_cast<uint2*>(p) = uint2{pack2(v[0], v[1]), pack2(v[2], v[3])};
}
__device__ __forceinline__ void lds_store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }

// What rounding to bfloat16 leaves of four values, itself rounded.
__device__ __forceinline__ void lds_store4_rest(uint16_t* p, f32x4 v) {
  uint32_t u0 = pack2(v[0], v[1]), u1 = pack2(v[2], v[3]);
  asm("" : "+v"(u0), "+v"(u1));
  *reinterpret_cast<uint2*>(p) = uint2{pack2(v[0] - low_half(u0), v[1] - high_half(u0)),
                                       pack2(v[2] - low_half(u1), v[3] - high_half(u1))};
}
// A fragment with 16 terms in half h and none in the other.  (Products of 16 terms,
// v_mfma_f32_16x16x16_bf16, would do half the work, but where one followed a product
// of 32 into the same registers its results were wrong now and then.)
__device__ __forceinline__ Frag<uint16_t> half_frag(uint2 u, int h) {
  const uint2 none = make_uint2(0, 0);
  return h ? frag_of(none, u) : frag_of(u, none);
}

// NT consecutive fours at byte offset `off`, rounded to V, as 8- or 16-byte stores.
template <typename V, int NT>
__device__ __forceinline__ void buf_store(buf_t to, uint32_t off, const f32x4 (&v)[NT]) {
  typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
  if constexpr (sizeof(V) == 4) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v[t]), to,
                                             static_cast<int>(off + 16 * t), 0, 0);
  } else if constexpr (NT == 1) {
    __builtin_amdgcn_raw_buffer_store_b64(
        u32x2{pack2(v[0][0], v[0][1]), pack2(v[0][2], v[0][3])}, to, static_cast<int>(off), 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b128(
        u32x4{pack2(v[0][0], v[0][1]), pack2(v[0][2], v[0][3]), pack2(v[1][0], v[1][1]),
              pack2(v[1][2], v[1][3])},
        to, static_cast<int>(off), 0, 0);
  }
}

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
// writes them to LDS.  Rows past n and columns past d load a valid piece
// instead and become zero when stashed: no branch stands around or between the
// loads, so that all are in flight at once and the wait for them counts what
// was issued since (where branches meet, it would wait for everything).  Pieces
// are read at any alignment.
//
// kHalves 2: the tile's columns are two heads' of D / 2 each, the second head's d
// values following the first's.
template <typename T, int C, int D, int kHalves = 1>
struct Tile {
  static constexpr int kPer = 16 / sizeof(T);              // values in a 16-byte piece
  static constexpr int kRowPieces = D / kPer;
  static constexpr int kPieces = C * kRowPieces / kThreads;
  static constexpr int kRowsApart = kThreads / kRowPieces;
  static_assert(C * kRowPieces % kThreads == 0 && kThreads % kRowPieces == 0, "whole pieces");
  uint4 v[kPieces];

  __device__ __forceinline__ void fetch(const T* base, uint32_t row, int n, int d) {
    const int r = threadIdx.x / kRowPieces;
    int c = static_cast<int>(threadIdx.x % kRowPieces) * kPer;
    if constexpr (kHalves == 2) c = (c >= D / 2 ? d : 0) + min(c % (D / 2), d - kPer);
    else c = min(c, d - kPer);
    const char* from = reinterpret_cast<const char*>(base);
    const uint32_t bytes = row * static_cast<uint32_t>(sizeof(T));   // below 2^24
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t off = __umul24(min(r + i * kRowsApart, n - 1), bytes) +
                           c * static_cast<uint32_t>(sizeof(T));
      __builtin_memcpy(&v[i], from + off, 16);
    }
  }
  __device__ __forceinline__ void stash(T* lds, int n, int d) const {
    const int r = threadIdx.x / kRowPieces, c = static_cast<int>(threadIdx.x % kRowPieces) * kPer;
    auto at = [&](int i) {
      return reinterpret_cast<uint4*>(lds + tile_at<T, D>(r + i * kRowsApart, c));
    };
    if (n == C && d == D / kHalves) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) *at(i) = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const bool in = r + i * kRowsApart < n && c % (D / kHalves) < d;
        *at(i) = in ? v[i] : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
};

// Decays of one chunk, in LDS.  Log decays are in powers of two.
template <int C>
struct Decay {
  float hi[C], lo[C];      // G, inclusive, as a float32 pair
  float ein[C];            // factor of the carried state at each token
  float w[C];              // factor of each token in the state's update
  float fac[C];            // forward: from the token to the end of its 16 tokens;
                           // backward: from the end of the 16 before to the token
  float all;               // exp(G_C)
};

// v of the lane a DPP control names, 0 where it names none.
template <int kCtrl, int kRows>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), kCtrl, kRows, 0xF, false);
  const uint32_t hi =
      __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), kCtrl, kRows, 0xF, false);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// 2^(hi + lo), lo below hi's last place: without it an argument near -100, say,
// would cost the result 4e-6 of itself.
__device__ __forceinline__ float exp2_of(float hi, float lo) {
  return fast_exp2(hi) * __builtin_fmaf(0.693147181f, lo, 1.0f);
}
__device__ __forceinline__ float exp2_of(double v) {
  const float hi = static_cast<float>(v);
  return exp2_of(hi, static_cast<float>(v - static_cast<double>(hi)));
}
// 2^(a + al - b - bl); kExact: with what the leading parts' difference loses in
// rounding (all of it where |a| >= |b|, as where the log decays are of one sign).
template <bool kExact>
__device__ __forceinline__ float exp2_diff(float a, float al, float b, float bl) {
  const float d = a - b;
  return kExact ? exp2_of(d, ((a - d) - b) + (al - bl)) : fast_exp2(d + (al - bl));
}

template <int C, bool kRev>
__device__ __forceinline__ void decays(Decay<C>& d, float g, float scale, int lane) {
  // far below what exp can represent, so that a decay to zero (minus infinity)
  // leaves the differences finite
  g = g < -1e4f ? -1e4f : g;
  // inclusive sums: shifts by 1, 2, 4, 8 inside rows of 16 lanes, then the last
  // lane of row 0 (and 2) to row 1 (and 3), then lane 31 to rows 2 and 3
  double s = static_cast<double>(g) * 1.4426950408889634074;
  s += dpp_f64<0x111, 0xF>(s);
  s += dpp_f64<0x112, 0xF>(s);
  s += dpp_f64<0x114, 0xF>(s);
  s += dpp_f64<0x118, 0xF>(s);
  const float fac = exp2_of(kRev ? s : dpp_f64<0x15F, 0xF>(s) - s);
  s += dpp_f64<0x142, 0xA>(s);
  s += dpp_f64<0x143, 0xC>(s);
  const uint64_t u = __builtin_bit_cast(uint64_t, s);
  const uint32_t tl = __builtin_amdgcn_readlane(static_cast<int>(u), C - 1);
  const uint32_t th = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), C - 1);
  const double total = __builtin_bit_cast(double, static_cast<uint64_t>(th) << 32 | tl);
  if (lane < C) {
    const float hi = static_cast<float>(s);
    d.hi[lane] = hi;
    const float lo = static_cast<float>(s - static_cast<double>(hi));
    d.lo[lane] = lo;
    const float in = exp2_of(hi, lo), out = exp2_of(total - s);
    d.ein[lane] = kRev ? out : scale * in;
    d.w[lane] = kRev ? scale * in : out;
    d.fac[lane] = fac;
    if (lane == 0) d.all = exp2_of(total);
  }
}

// Two wait states before a value is read through DPP, wherever a branch may have
// led here from (inside a block the compiler sees to them).
__device__ __forceinline__ float before_dpp(float v) {
  asm volatile("s_nop 1" : "+v"(v));
  return v;
}

// Inclusive sums over the wavefront, by the same steps as the decays'.
__device__ __forceinline__ float scan_f32(float v) {
  v = before_dpp(v);
#define MSSM_LA_SCAN(CTRL, ROWS) \
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
  MSSM_LA_SCAN(0x111, 0xF)
  MSSM_LA_SCAN(0x112, 0xF)
  MSSM_LA_SCAN(0x114, 0xF)
  MSSM_LA_SCAN(0x118, 0xF)
  MSSM_LA_SCAN(0x142, 0xA)
  MSSM_LA_SCAN(0x143, 0xC)
#undef MSSM_LA_SCAN
  return v;
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Sum over the 16 lanes of a row, in every one of them (rotations by 8, 4, 2, 1).
__device__ __forceinline__ float row16_sum(float v) {
  v = before_dpp(v);
#define MSSM_LA_ROT(CTRL) \
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
  MSSM_LA_ROT(0x128)
  MSSM_LA_ROT(0x124)
  MSSM_LA_ROT(0x122)
  MSSM_LA_ROT(0x121)
#undef MSSM_LA_ROT
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// ---- what a segment's state depends on ---------------------------------------------------------------

// How many tokens of a segment, from its end (in reverse its start) on, can reach
// its state.  Where the decays between a token and that end come to less than
// 2^-256, they take whatever the state held at the token, any finite float32, below
// the smallest normal number: the token and all on its other side add exactly
// nothing and need not be read, and nothing passes through the segment.  Each
// thread sums a run of log decays, the runs are scanned, and the answer is rounded
// up to whole runs.  (1 x 131072, 20 heads of 128, log decays of -0.02 times 1 to
// 16 on average: the state pass reads about a third of the tokens of segments of
// 5248 and takes 220 us; it took 326 over all of them in segments of 2624.)
constexpr int kReachFrom = 512;            // shorter segments are not looked over
struct Reach {
  float sum[4];
  int count[4];
};
template <bool kRev>
__device__ __forceinline__ int reach(Reach& m, const float* g, int64_t g_row, int len, int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  const int run = (len + kThreads - 1) / kThreads;
  float s = 0.0f;
#pragma unroll 8
  for (int r = 0; r < run; ++r) {
    const int u = min(tid * run + r, len - 1);     // (past the last token: never asked for)
    const float v = g[(kRev ? u : len - 1 - u) * g_row];
    s += v < -1e4f ? -1e4f : v;
  }
  s *= 1.44269504f;
  const float upto = scan_f32(s);
  if (lane == 63) m.sum[wave] = upto;
  block_sync();
  float before = upto - s;
#pragma unroll
  for (int w = 0; w < 3; ++w) before += w < wave ? m.sum[w] : 0.0f;
  const uint64_t out = __ballot(before <= -257.0f);         // (false for NaN)
  if (lane == 0) m.count[wave] = out ? __builtin_ctzll(out) : 64;
  block_sync();
  int runs = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) runs += runs == 64 * w ? m.count[w] : 0;
  return min(runs * run, len);
}

// ---- the pass ----------------------------------------------------------------------------------------

// V: the type the output is stored in.
// kHeads 2: two heads that share x and y in one block, two wavefronts for each;
// the products of x and y, and their tiles, then serve both.
// kOut false: only the state over the segment (no x, no output).
// kDot 0: nothing more.  1 (dq): also W and q . dqc, as one sum u for each
// token, and the state before some of the chunks.  2 (dk): also k . dkc, and dg
// from it, u and those states.
template <typename T, int C, int DA, int NT, int kHeads, bool kOut, int kDot>
struct Lds {
  static constexpr int TB = 64 * NT;                        // columns of z
  static constexpr int PP = C + 16 / sizeof(T);             // row pitch of p
  T x[kOut ? C * DA : 8];
  T y[C * DA];
  T z[C * TB];
  T e[kDot == 1 ? C * TB : 8];
  T p[kOut ? kHeads * C * PP : 8];
  Decay<C> d[2][kHeads];
  float dot[kDot ? 4 : 1][C];
  float rows[kDot == 1 ? 2 : 1][C];
  float cols[kDot == 1 ? 4 : 1][C];
  float edge[4];
};

// Of the chunks of a segment, those whose carried-through part of dg is computed
// from the two states themselves: the last and every kStride-th before it.  The
// others get it from the next chunk's, by what enters and leaves in between.
template <int C>
constexpr int kStride = 256 / C;

template <typename T, typename V, int C, int DA, int NT, int kHeads, bool kRev, bool kOut, int kDot>
__global__ __launch_bounds__(kThreads, 2) void la_pass(PassArgs p) {
  constexpr bool kBf16 = sizeof(T) == 2;
  constexpr int kStateParts = kBf16 && kDot != 0 ? 3 : 1;  // of the state as an operand
  constexpr bool kExact = !kBf16 || kDot != 0;             // float32 results depend on the scores
  constexpr int NR = C / 16, NK = C / 32, NM = DA / 16, TB = 64 * NT;
  constexpr int PP = Lds<T, C, DA, NT, kHeads, kOut, kDot>::PP;
  __shared__ __align__(16) Lds<T, C, DA, NT, kHeads, kOut, kDot> m;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;

  static_assert(kHeads == 1 || (NT == 2 && kDot == 0), "two heads of up to 64 columns");
  const uint32_t block = logical_block();
  const uint32_t groups = static_cast<uint32_t>(p.heads) / kHeads;
  const int64_t slot = block / groups;
  const int h = static_cast<int>(block % groups) * kHeads;
  const int hw = kHeads == 2 ? wave >> 1 : 0;              // this wavefront's head is h + hw
  Place at = place_of(p.grid, slot);
  if (!at.ok) {
    if constexpr (kDot == 2) {
      if (p.head_part && tid == 0) p.head_part[block] = 0.0f;
    }
    return;
  }
  // a state-only pass has nothing to do for the segment that no other follows
  const bool last_seg = kRev ? at.local == 0 : at.local == at.count - 1;
  if (!kOut && last_seg) return;
  bool whole = true;                       // nothing of the segment is out of reach
  if constexpr (!kOut) {
    if (at.len >= kReachFrom) {
      __shared__ Reach look[kHeads];
      int n = 0;
#pragma unroll
      for (int hh = 0; hh < kHeads; ++hh)
        n = max(n, reach<kRev>(look[hh], p.g + at.start * p.g_row + h + hh, p.g_row,
                               static_cast<int>(at.len), tid));
      const int64_t beyond = kRev ? max(at.len - int64_t(n + C - 1) / C * C, int64_t(0))
                                  : (at.len - n) / C * C;           // whole chunks
      whole = beyond == 0;
      if (!kRev) at.start += beyond;
      at.len -= beyond;
    }
  }

  // columns of this wavefront: with two tiles, lane group g4's rows 4 g4 + r of
  // both are the eight consecutive columns 8 g4 + 4 t + r (16-byte stores)
  constexpr int kStep = NT == 2 ? 8 : 4;
  const int c_wave = 16 * NT * wave;
  const int c_head = c_wave - 64 * hw;                     // of its head's columns
  auto col_of = [&](int t, int c) { return c_head + kStep * (c >> 2) + 4 * t + (c & 3); };

  const int64_t sh = (at.seq * p.heads + h + hw) * (int64_t(p.dA) * p.dB);        // per sequence
  const int64_t wh = (slot * p.heads + h + hw) * (int64_t(p.dA) * p.dB);          // per segment

  // the state: rows 16 mt + 4 g4 + r of dA, column col_of(t, l16)
  auto row_of = [&](int mt, int r) { return 16 * mt + 4 * g4 + r; };
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
          const int a = row_of(mt, r);
          s[mt][t][r] = init && a < p.dA && c < p.dB ? init[a * p.sA + c * p.sB] : 0.0f;
        }
      }
  }

  const int chunks = static_cast<int>((at.len + C - 1) / C);
  const float scale = p.scale;
  // A chunk's tiles on their way from memory.  The loads run one chunk ahead of
  // their use, or two, with a second set of registers where state, results and
  // both sets leave room for two blocks on a compute unit (256 registers).  The
  // log decays run two ahead: a chunk's factors are made while the one before is
  // worked on.
  struct Stage {
    Tile<T, C, DA> x, y;
    Tile<T, C, TB, kHeads> z;
    Tile<T, C, TB> e;
  };
  constexpr int kStage = (kOut ? Tile<T, C, DA>::kPieces : 0) * 4 + Tile<T, C, DA>::kPieces * 4 +
                         Tile<T, C, TB>::kPieces * 4 * (kDot == 1 ? 2 : 1);
  constexpr int kHeld = NM * NT * 4 + (kOut ? NR * NT * 4 : 0) + (kDot == 2 ? NR * NT * 4 : 0);
  constexpr int kSets = kHeld + 2 * kStage <= (kOut ? 112 : 128) ? 2 : 1;
  constexpr bool kLate = kOut && kHeld + kStage > 100;
  Stage sets[kSets];
  // Tokens of the it-th chunk worked on, and the pointers to the next chunk to load.
  const int len = static_cast<int>(at.len);
  auto tokens_of = [&](int it) { return min(len - (kRev ? chunks - 1 - it : it) * C, C); };
  const int64_t first = at.start + (kRev && chunks > 0 ? int64_t(chunks - 1) * C : 0);
  auto begin = [&](const View& v, int size) {
    return static_cast<const T*>(v.p) + first * v.row + int64_t(h / v.div) * size;
  };
  const T* X = kOut ? begin(p.x, p.dA) : nullptr;
  const T* Y = begin(p.y, p.dA);
  const T* Z = begin(p.z, p.dB);
  const T* E = kDot == 1 ? begin(p.e, p.dB) : nullptr;
  // (the wavefronts that make the decays load them: one for each head)
  const float* G = p.g + (p.g_row ? first * p.g_row : 0) + h + (kHeads == 2 ? wave & 1 : 0);
  constexpr int kAhead = kRev ? -C : C;                     // tokens from chunk to chunk
  const uint32_t x_row = static_cast<uint32_t>(p.x.row), y_row = static_cast<uint32_t>(p.y.row);
  const uint32_t z_row = static_cast<uint32_t>(p.z.row), e_row = static_cast<uint32_t>(p.e.row);
  const uint32_t g_row = static_cast<uint32_t>(p.g_row);
  // Past the last chunk these load it again (unused).
  auto fetch_g = [&](int it) __attribute__((always_inline)) {
    const float g = G[static_cast<uint32_t>(min(lane, tokens_of(it) - 1)) * g_row];
    if (it + 1 < chunks) G += kAhead * static_cast<int64_t>(g_row);
    return g;
  };
  auto fetch = [&](Stage& f, int it) __attribute__((always_inline)) {
    const int n = tokens_of(it);
    const int64_t next = it + 1 < chunks ? kAhead : 0;
    if constexpr (kOut) {
      f.x.fetch(X, x_row, n, p.dA);
      X += next * x_row;
    }
    f.y.fetch(Y, y_row, n, p.dA);
    Y += next * y_row;
    f.z.fetch(Z, z_row, n, p.dB);
    Z += next * z_row;
    if constexpr (kDot == 1) {
      f.e.fetch(E, e_row, n, p.dB);
      E += next * e_row;
    }
  };
  // The chunk being worked on: where its output, and what is dotted with it, begin.
  const uint32_t o_row = static_cast<uint32_t>(p.heads) * p.dB;
  V* out = kOut ? static_cast<V*>(p.out) + first * o_row + int64_t(h) * p.dB : nullptr;
  const T* dotted = kDot == 2 ? begin(p.e, p.dB) : nullptr;
  float* u_at = kDot != 0 ? p.u + first * p.heads + h : nullptr;
  float* dg_at = kDot == 2 && p.dg ? p.dg + first * p.heads + h : nullptr;

  constexpr int kDumpSize = DA * TB;
  // The second parts of the diagonal's scores lie in tiles of p that no product reads:
  // (0 and 1, 2 and 3), in reverse (2 and 3, 0 and 1).
  auto rest_at = [&](int rt) {
    return (16 * ((kRev ? 2 : 0) + (rt & 1)) + l16) * PP + 16 * ((kRev ? 0 : 2) + (rt >> 1)) + 4 * g4;
  };
  float edge = 0.0f, head_sum = 0.0f;      // dg's are wavefront 0's
  double decay_sum = 0.0;
  float g_next = 0.0f;                     // log decays of the next chunk

  auto step = [&](int it, Stage& f) __attribute__((always_inline)) {
    const int ck = kRev ? chunks - 1 - it : it;
    const int n = tokens_of(it);
    const Decay<C>& d = m.d[it & 1][hw];
    if constexpr (kOut) f.x.stash(m.x, n, p.dA);
    f.y.stash(m.y, n, p.dA);
    f.z.stash(m.z, n, p.dB);
    if constexpr (kDot == 1) f.e.stash(m.e, n, p.dB);
    block_sync();
    const float g_after = fetch_g(min(it + 2, chunks - 1));
    if constexpr (!kLate) fetch(f, min(it + kSets, chunks - 1));
    const int back = (chunks - 1 - ck) % kStride<C>;
    float* dump = nullptr;
    if constexpr (kDot != 0) {
      if (back == 0)
        dump = p.dumps + ((slot * p.dumps_per_slot + (chunks - 1 - ck) / kStride<C>) * p.heads + h) *
                             int64_t(kDumpSize) + tid * 4;
    }
    // (dk: the first half of the state that dq left there, loaded before the products
    // that stand between, into the registers of the tiles now in LDS)
    constexpr int kHalf = kDot == 2 ? NM * NT / 2 : 1;
    f32x4 left[kHalf];
    if constexpr (kDot == 2) {
      if (dump) {
#pragma unroll
        for (int u = 0; u < kHalf; ++u) left[u] = *reinterpret_cast<const f32x4*>(dump + u * (kThreads * 4));
      }
    }
    if constexpr (kDot == 1) {
      if (dump) {
#pragma unroll
        for (int mt = 0; mt < NM; ++mt)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            *reinterpret_cast<f32x4*>(dump + (mt * NT + t) * (kThreads * 4)) = s[mt][t];
      }
    }
    // the tensor that the carried part is dotted with, and u: used further on
    f32x4 ev[kDot == 2 ? NR : 1][NT];
    float uv = 0.0f, qs = 0.0f;
    if constexpr (kDot == 2) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint32_t i = min(16 * r + l16, n - 1), c = min(col_of(t, 4 * g4), p.dB - 4);
          T raw[4];
          __builtin_memcpy(raw, dotted + (i * e_row + c), sizeof(raw));
#pragma unroll
          for (int q = 0; q < 4; ++q) ev[r][t][q] = to_float(raw[q]);
        }
      uv = u_at[static_cast<uint32_t>(min(lane, n - 1) * p.heads)];
      const f32x4 q = *reinterpret_cast<const f32x4*>(p.q_sums + ((slot * p.chunks_per_slot + ck) * p.heads + h) * 4);
      qs = (q[0] + q[1]) + (q[2] + q[3]);
    }

    f32x4 acc[NR][NT];
    if constexpr (kOut) {
      // the C x C products of this wavefront's part: tiles (rows of x, rows of
      // y), each result a lane's column i (row of x) and four rows j of y
      constexpr int kWaveTiles = NR == 4 ? 4 : 1;
      const int rt = NR == 4 ? wave : wave >> 1;
      const int i = 16 * rt + l16;
      float row_sum = 0.0f;
      // All of a row tile's products are formed, also those that the mask then
      // drops: without branches between them the loads and products of one hide
      // the latency of the others.
      f32x4 as[kWaveTiles], bs[kDot == 1 ? kWaveTiles : 1];
      {
        Frag<T> xf[DA / 32];
#pragma unroll
        for (int k = 0; k < DA / 32; ++k) xf[k] = frag_row<DA>(m.x, i, 32 * k + 4 * g4);
#pragma unroll
        for (int u = 0; u < kWaveTiles; ++u) {
          const int ct = NR == 4 ? u : wave & 1;
          as[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < DA / 32; ++k)
            mma(as[u], frag_row<DA>(m.y, 16 * ct + l16, 32 * k + 4 * g4), xf[k]);
        }
      }
      if constexpr (kDot == 1) {
        Frag<T> ef[TB / 32];
#pragma unroll
        for (int k = 0; k < TB / 32; ++k) ef[k] = frag_row<TB>(m.e, i, 32 * k + 4 * g4);
#pragma unroll
        for (int u = 0; u < kWaveTiles; ++u) {
          const int ct = NR == 4 ? u : wave & 1;
          bs[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < TB / 32; ++k)
            mma(bs[u], frag_row<TB>(m.z, 16 * ct + l16, 32 * k + 4 * g4), ef[k]);
        }
      }
#pragma unroll
      for (int hh = 0; hh < kHeads; ++hh) {
        const Decay<C>& dh = m.d[it & 1][hh];
        T* const ph = m.p + hh * C * PP;
        const float gi = dh.hi[i], gil = dh.lo[i];
#pragma unroll
        for (int u = 0; u < kWaveTiles; ++u) {
          const int ct = NR == 4 ? u : wave & 1;
          const bool live = kRev ? ct >= rt : ct <= rt;
          const int j0 = 16 * ct + 4 * g4;
          if (live) {
            f32x4 a = as[u], b = bs[kDot == 1 ? u : 0];
            if (ct == rt) {
              const f32x4 gj = *reinterpret_cast<const f32x4*>(&dh.hi[j0]);
              const f32x4 gjl = *reinterpret_cast<const f32x4*>(&dh.lo[j0]);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const bool in = kRev ? j0 + r >= i : j0 + r <= i;
                const float f = kRev ? exp2_diff<kExact>(gj[r], gjl[r], gi, gil) : exp2_diff<kExact>(gi, gil, gj[r], gjl[r]);
                a[r] = in ? a[r] * (scale * f) : 0.0f;
                if constexpr (kDot == 1) b[r] = j0 + r != i ? a[r] * b[r] : 0.0f;
              }
            } else {
              // through the boundary between the 16 tokens and what is nearer to i
              const int edge16 = kRev ? 16 * ct - 1 : 16 * ct + 15;
              const float fi = scale * (kRev ? exp2_diff<kExact>(dh.hi[edge16], dh.lo[edge16], gi, gil)
                                             : exp2_diff<kExact>(gi, gil, dh.hi[edge16], dh.lo[edge16]));
              const f32x4 fj = *reinterpret_cast<const f32x4*>(&dh.fac[j0]);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                a[r] *= fi * fj[r];
                if constexpr (kDot == 1) b[r] *= a[r];
              }
            }
            lds_store4(ph + i * PP + j0, a);
            if constexpr (kBf16) {
              if (ct == rt) lds_store4_rest(ph + rest_at(rt), a);
            }
            if constexpr (kDot == 1) {
              row_sum += (b[0] + b[1]) + (b[2] + b[3]);
              // sums over this wavefront's 16 rows i, for each of the four j
#pragma unroll
              for (int r = 0; r < 4; ++r) b[r] = row16_sum(b[r]);
              if (l16 == 0) *reinterpret_cast<f32x4*>(&m.cols[rt][j0]) = b;
            }
          } else if ((ct ^ rt) == 1) {
            lds_store4(ph + i * PP + j0, f32x4{0.0f, 0.0f, 0.0f, 0.0f});   // read with its neighbour
          }
        }
      }
      // the wavefronts with the fewest scores prepare the next chunk's decays
      if ((kRev ? wave > 3 - kHeads : wave < kHeads) && it + 1 < chunks)
        decays<C, kRev>(m.d[(it + 1) & 1][wave & (kHeads - 1)], lane < tokens_of(it + 1) ? g_next : 0.0f, scale, lane);
      if constexpr (kDot == 1) {
        row_sum += __shfl_xor(row_sum, 16, 64);
        row_sum += __shfl_xor(row_sum, 32, 64);
        // with two row tiles, each of a row tile's two wavefronts has a part
        if (g4 == 0) m.rows[NR == 4 ? 0 : wave & 1][i] = row_sum;
      }

      // the carried part: x S
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < DA / 32; ++k) {
        Frag<T> part[NT][kStateParts];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float v[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = s[2 * k][t][r], v[4 + r] = s[2 * k + 1][t][r];
          split(v, part[t]);
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const Frag<T> xf = frag_row<DA>(m.x, 16 * r + l16, 32 * k + 4 * g4);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int q = 0; q < kStateParts; ++q) mma(acc[r][t], part[t][q], xf);
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float fe = d.ein[16 * r + l16];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] *= fe;
      }
      if constexpr (kDot != 0) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int i2 = 16 * r + l16;
          float dot = 0.0f;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            f32x4 e4;
            if constexpr (kDot == 1) e4 = lds_load4(m.e + tile_at<T, TB>(i2, col_of(t, 4 * g4)));
            else e4 = ev[r][t];       // past n or dB: acc is zero there, of finite values
#pragma unroll
            for (int q = 0; q < 4; ++q) dot = __builtin_fmaf(acc[r][t][q], e4[q], dot);
          }
          dot += __shfl_xor(dot, 16, 64);
          dot += __shfl_xor(dot, 32, 64);
          if (g4 == 0) m.dot[wave][i2] = dot;
        }
      }
      if constexpr (kDot == 2) {
        if (dump) {
          f32x4 right[kHalf];
#pragma unroll
          for (int u = 0; u < kHalf; ++u)
            right[u] = *reinterpret_cast<const f32x4*>(dump + (kHalf + u) * (kThreads * 4));
          float part = 0.0f;
#pragma unroll
          for (int u = 0; u < NM * NT; ++u) {
            const f32x4 q = u < kHalf ? left[u % kHalf] : right[u % kHalf];
#pragma unroll
            for (int r = 0; r < 4; ++r) part = __builtin_fmaf(q[r], s[u / NT][u % NT][r], part);
          }
          part = wave_sum(part);
          if (lane == 0) m.edge[wave] = part;
        }
      }
      block_sync();
    }
    if constexpr (kLate) fetch(f, min(it + 1, chunks - 1));

    // z by columns, for the scores' product and for the state
    Frag<T> zf[NK][NT];
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        zf[k][t] = frag_col<TB, kStep>(m.z, 32 * k, c_wave + 4 * t, lane);

    if constexpr (kOut) {
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          if (kRev ? k < r / 2 : k > r / 2) continue;
          const Frag<T> pf = frag_at(m.p + (hw * C + 16 * r + l16) * PP + 32 * k + 4 * g4);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma(acc[r][t], zf[k][t], pf);
        }
      if constexpr (kBf16) {
        static_assert(NR == 4, "tiles for the diagonal's second parts");
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const Frag<T> rest = half_frag(lds_read8(m.p + hw * C * PP + rest_at(r)), r & 1);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma(acc[r][t], zf[r / 2][t], rest);
        }
      }
      // Stores through a descriptor that ends with the chunk's last value: rows and
      // columns past it are dropped by the hardware, so no branch stands around them.
      // (Buffer accesses, too, take any alignment.)
      {
        const buf_t to = make_buf(out, ((n - 1) * o_row + kHeads * p.dB) * static_cast<uint32_t>(sizeof(V)));
        const uint32_t c = col_of(0, 4 * g4);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const uint32_t off = c < static_cast<uint32_t>(p.dB) ? (16 * r + l16) * o_row + hw * p.dB + c : 0x3ffffff0u;
          buf_store<V, NT>(to, off * static_cast<uint32_t>(sizeof(V)), acc[r]);
        }
      }
      if constexpr (kDot == 1) {
        // Each wavefront finishes 16 tokens, lane group g4 with its part of the sums,
        // and without branches, beside the products.
        const int w = NR == 4 ? wave : wave & 1, i2 = 16 * w + l16;
        float qd = m.dot[g4][i2];
        const float rows = m.rows[NR == 4 ? 0 : g4 & 1][i2], cols = m.cols[NR == 4 ? g4 : g4 & 1][i2];
        float u = (g4 < (NR == 4 ? 1 : w + 1) ? rows : 0.0f) - (g4 >= w && g4 < NR ? cols : 0.0f);
        qd += __shfl_xor(qd, 16, 64);
        u += __shfl_xor(u, 16, 64);
        qd += __shfl_xor(qd, 32, 64);
        u += __shfl_xor(u, 32, 64);
        const bool mine = wave < NR;
        const uint32_t heads = static_cast<uint32_t>(p.heads);
        __builtin_amdgcn_raw_buffer_store_b32(
            __float_as_uint(qd + u), make_buf(u_at, ((n - 1) * heads + 1) * 4),
            g4 == 0 && mine ? static_cast<int>(i2 * heads * 4) : 0x3ffffff0, 0, 0);
        const float sum = row16_sum(mine && i2 < n ? qd : 0.0f);
        __builtin_amdgcn_raw_buffer_store_b32(
            __float_as_uint(sum), make_buf(p.q_sums + ((slot * p.chunks_per_slot + ck) * p.heads + h) * 4, 16),
            lane == 0 ? wave * 4 : 0x3ffffff0, 0, 0);
      }
      if constexpr (kDot == 2) {
        if (wave == 0) {
          const bool in = lane < n;
          const int t = min(lane, C - 1);
          const float kd = in ? (m.dot[0][t] + m.dot[1][t]) + (m.dot[2][t] + m.dot[3][t]) : 0.0f;
          const float u = in ? uv : 0.0f;
          const float before = scan_f32(kd), u_before = scan_f32(u);     // up to this token
          const float after = u + (lane_value(u_before, 63) - u_before); // from it on
          // what passes through the whole chunk
          const float through = dump ? d.all * ((m.edge[0] + m.edge[1]) + (m.edge[2] + m.edge[3]))
                                     : edge - lane_value(before, 63);
          const float dg = after + (before - kd) + through;
          edge = through + qs;
          if (in) {
            if (p.dg) dg_at[static_cast<uint32_t>(lane * p.heads)] = dg;
            head_sum += dg;
          }
        }
      }
    }

    if constexpr (kOut) out += kAhead * static_cast<int64_t>(o_row);
    if constexpr (kDot == 2) {
      dotted += kAhead * static_cast<int64_t>(e_row);
      dg_at += kAhead * p.heads;
    }
    if constexpr (kDot != 0) u_at += kAhead * p.heads;

    // The state after the chunk.  Three parts of the weighted z where the state
    // itself is a result or dg depends on it; two where only outputs rounded to
    // bfloat16 do.
    if (it + 1 < chunks || !kOut || (last_seg && p.last)) {
      constexpr int kParts = !kBf16 ? 1 : kOut && kDot == 0 ? 2 : 3;
      const float all = d.all;
#pragma unroll
      for (int mt = 0; mt < NM; ++mt)
#pragma unroll
        for (int t = 0; t < NT; ++t) s[mt][t] *= all;
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        Frag<T> part[NT][kParts];
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(&d.w[32 * k + 4 * g4]);
        const f32x4 w1 = *reinterpret_cast<const f32x4*>(&d.w[32 * k + 16 + 4 * g4]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float v[8];
          unpack(zf[k][t], v);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] *= w0[e], v[4 + e] *= w1[e];
          split(v, part[t]);
        }
        // (two row tiles at once, so that products into the same registers, which wait
        // for one another, stand apart)
#pragma unroll
        for (int mt = 0; mt < NM; mt += 2) {
          const Frag<T> yf[2] = {frag_col<DA, 4>(m.y, 32 * k, 16 * mt, lane),
                                 frag_col<DA, 4>(m.y, 32 * k, 16 * mt + 16, lane)};
#pragma unroll
          for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int t = 0; t < NT; ++t) mma(s[mt + u][t], yf[u], part[t][q]);
        }
        if constexpr (kParts == 2) {
          if (last_seg && p.last) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              float v[8], v0[8], v1[8];
              unpack(zf[k][t], v);
              unpack(part[t][0], v0);
              unpack(part[t][1], v1);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                v[e] = __builtin_fmaf(v[e], e < 4 ? w0[e] : w1[e - 4], -v0[e]) - v1[e];
              split(v, reinterpret_cast<Frag<T>(&)[1]>(part[t][0]));
            }
#pragma unroll
            for (int mt = 0; mt < NM; ++mt) {
              const Frag<T> yf = frag_col<DA, 4>(m.y, 32 * k, 16 * mt, lane);
#pragma unroll
              for (int t = 0; t < NT; ++t) mma(s[mt][t], yf, part[t][0]);
            }
          }
        }
      }
    }
    if constexpr (!kOut) {
      decay_sum += static_cast<double>(d.hi[C - 1]) + d.lo[C - 1];   // the segment's
    }
    if (!kOut && wave < kHeads && it + 1 < chunks)
      decays<C, kRev>(m.d[(it + 1) & 1][wave & (kHeads - 1)], lane < tokens_of(it + 1) ? g_next : 0.0f, scale, lane);
    g_next = g_after;
    block_sync();
  };
  if (chunks > 0) {
    const float g_first = fetch_g(0);
    g_next = fetch_g(min(1, chunks - 1));
    // Each set's first loads are followed by as many stores as later ones (into an
    // empty buffer, dropped): the waits in the loop then leave that many in flight,
    // where for the sake of the first turn they would otherwise drain them.
    auto no_stores = [&](int k) __attribute__((always_inline)) {
      if constexpr (kOut) {
        const buf_t none = make_buf(out, 0);
        const f32x4 zero[NT] = {};
#pragma unroll
        for (int r = 0; r < NR; ++r) buf_store<V, NT>(none, 64 * (NR * k + r), zero);
      }
    };
    fetch(sets[0], 0);
    no_stores(0);
    if constexpr (kSets == 2) {
      fetch(sets[1], min(1, chunks - 1));
      no_stores(1);
    }
    if (wave < kHeads)
      decays<C, kRev>(m.d[0][wave & (kHeads - 1)], lane < tokens_of(0) ? g_first : 0.0f, scale, lane);
  }
  int it = 0;
  if constexpr (kSets == 2) {
    for (; it + 1 < chunks; it += 2) {
      step(it, sets[0]);
      step(it + 1, sets[1]);
    }
    if (it < chunks) step(it, sets[0]);
  } else {
    for (; it < chunks; ++it) step(it, sets[0]);
  }

  if constexpr (kDot == 2) {
    if (p.head_part && wave == 0) {
      head_sum = wave_sum(head_sum);
      if (lane == 0) p.head_part[slot * p.heads + h] = head_sum;
    }
  }
  float* dst = nullptr;
  if constexpr (kOut) {
    if (last_seg && p.last) dst = p.last + sh;
  } else {
    dst = p.seg_out + wh;
    if (lane == 0 && wave % (4 / kHeads) == 0)
      p.seg_decay[slot * p.heads + h + hw] = whole ? exp2_of(decay_sum) : 0.0f;
  }
  if (!dst) return;
#pragma unroll
  for (int mt = 0; mt < NM; ++mt)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = col_of(t, l16);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int a = row_of(mt, r);
        if (a < p.dA && c < p.dB) dst[a * p.sA + c * p.sB] = s[mt][t][r];
      }
    }
}

}  // namespace la
}  // namespace mssm
