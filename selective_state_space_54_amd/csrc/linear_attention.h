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
// Rounding.  Products of bfloat16 inputs accumulate in float32.  Float32 operands
// go through the bfloat16 products in parts, each the rounding of what the parts
// before it leave.  The decayed scores, and the state where it is an operand of
// an output that is rounded to bfloat16 itself, have two (16 bits, 2^-17.5 of
// them on average): an output then differs from the float32 formula rounded once
// by 1e-4 of the norm, a last place where the rounding is all but a tie.  (One part,
// but for the scores of the 16 x 16 tiles on the diagonal: 1.8e-3.  The second
// costs 1 x 131072 tokens of 20 heads of 128 930 us, not 874; packed prompts of
// 32768 tokens, 32 heads of 128 x 64 304, not 284; a gradient over 4 x 8192, 16
// heads of 128 756, not 748.)  Where float32 results depend on them (the state's
// own update, dg) the operand has three parts, 24 bits.  Decays, their sums (float64
// inside a chunk, kept as a float32 pair) and the state are 32 bits or more.
//
// What bounds it.  On long prompts memory, then what a wavefront issues between a
// chunk's barriers: 1 x 131072 tokens of 20 heads of 128, bf16, moves 2.75 GB in
// 715 us (3.9 TB/s; 256-byte rows reach 4.1 to 4.9 when only copied) with the
// matrix cores busy 37 % of the cycles.  dq and dk split the state in three
// parts: 4 x 8192, 16 heads of 128: 229 and 232 us at 3.8 TB/s, matrix cores 27 %,
// vector instructions as long again, two blocks a compute unit for 256 registers
// each, some spilled (20 and 28 bytes a lane).  float32: the 16x16x4 products and
// the LDS reads between them, 40 % of whose cycles meet bank conflicts (the
// swizzle of the tiles is made for values of two bytes): 8 x 2048, 24 heads of 64:
// 131 us, 56 % of the matrix cores' cycles.  Its gradient passes for heads of 128
// spill 160 to 250 bytes a lane: 4 x 2048, 16 heads: 177, 126 and 155 us.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
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
// v_mfma_f32_16x16x16_bf16, would do half the work.  But in a variant where one followed
// a product of 32 into the same registers, results were wrong now and then; why was not
// found.  So no kernel has matrix products of two kinds:
// tests/test_linear_attention_isa_cpu.py looks for them in the compiled code.)
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
__device__ __forceinline__ uint32_t logical_block(uint32_t n, uint32_t b) {
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
struct alignas(16) Decay {
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
// 5248 and takes 245 us; it took 326 over all of them in segments of 2624.)
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
  static constexpr int PR = C + (sizeof(T) == 2 ? 16 : 0);  // rows of p: a head's
  T x[kOut ? C * DA : 8];
  T y[C * DA];
  T z[C * TB];
  T e[kDot == 1 ? C * TB : 8];
  T p[kOut ? kHeads * PR * PP : 8];
  Decay<C> d[2][kHeads];
  float dot[kDot ? 4 : 1][C];
  float rows[kDot == 1 && C == 32 ? 2 : 1][kDot == 1 ? C : 4];
  alignas(16) float cols[kDot == 1 ? C / 32 * (C + 16) : 4];   // row tile rt's first 16 (rt + 1), on end
  float edge[kDot == 2 ? 4 : 1];
};

// Of the chunks of a segment, those whose carried-through part of dg is computed
// from the two states themselves: the last and every kStride-th before it.  The
// others get it from the next chunk's, by what enters and leaves in between.
template <int C>
constexpr int kStride = 256 / C;

template <typename T, typename V, int C, int DA, int NT, int kHeads, bool kRev, bool kOut, int kDot>
__device__ __forceinline__ void pass(const PassArgs& p, Lds<T, C, DA, NT, kHeads, kOut, kDot>& m,
                                     uint32_t blocks, uint32_t index) {
#include "la_pass_body.h"
}

template <typename T, typename V, int C, int DA, int NT, int kHeads, bool kRev, bool kOut, int kDot>
__global__ __launch_bounds__(kThreads, 2) void la_pass(PassArgs p) {
  __shared__ __align__(16) Lds<T, C, DA, NT, kHeads, kOut, kDot> m;
  const uint32_t blocks = gridDim.x, index = blockIdx.x;
#include "la_pass_body.h"
}

// Two passes that do not wait for each other in one launch.  The segments' own states
// in both directions (4 x 8192, 16 heads of 128: 137 us, 147 in two launches):
template <typename T, int C, int DA, int NT, int kHeads>
__global__ __launch_bounds__(kThreads, 2) void la_states(PassArgs fwd, PassArgs rev) {
  __shared__ __align__(16) Lds<T, C, DA, NT, kHeads, false, 0> m;
  if (blockIdx.y == 0) pass<T, T, C, DA, NT, kHeads, false, false, 0>(fwd, m, gridDim.x, blockIdx.x);
  else pass<T, T, C, DA, NT, kHeads, true, false, 0>(rev, m, gridDim.x, blockIdx.x);
}

// and dq (the first `n` blocks) and dv, for passes that leave compute units free.
template <typename T, typename V, int C, int DK, int DV, int kHeads>
__global__ __launch_bounds__(kThreads, 2) void la_dq_dv(PassArgs dq, PassArgs dv, uint32_t n) {
  constexpr int NQ = DK / 64, NV = kHeads == 2 ? 2 : DV / 64;
  using Q = Lds<T, C, DV, NQ, 1, true, 1>;
  using U = Lds<T, C, DK, NV, kHeads, true, 0>;
  __shared__ __align__(16) char m[sizeof(Q) > sizeof(U) ? sizeof(Q) : sizeof(U)];
  if (blockIdx.x < n)
    pass<T, V, C, DV, NQ, 1, false, true, 1>(dq, *reinterpret_cast<Q*>(m), n, blockIdx.x);
  else
    pass<T, T, C, DK, NV, kHeads, true, true, 0>(dv, *reinterpret_cast<U*>(m), gridDim.x - n,
                                                 blockIdx.x - n);
}

}  // namespace la
}  // namespace mssm
