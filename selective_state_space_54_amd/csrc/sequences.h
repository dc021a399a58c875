// Tokens in one row, sequence after sequence, and where sequences begin and end
// among a wavefront's few consecutive tokens (gfx950).
//
// Dense batches and packed sequences are the same thing here: `n` sequences whose
// tokens lie behind one another, each of `L` tokens, or from offsets[q] to
// offsets[q + 1].  A kernel walks the row in pieces of any position; most pieces
// hold no border, and one scalar search says so.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mssm {

struct Sequences {
  const int64_t* offsets = nullptr;   // [n + 1] on the device, or null
  int64_t n = 0;
  int64_t L = 0;                      // tokens of each, without offsets
  int64_t tokens = 0;                 // of all
};

#ifdef __HIP_DEVICE_COMPILE__
#define MSSM_UNIFORM(v) __builtin_amdgcn_readfirstlane(v)
#else
#define MSSM_UNIFORM(v) (v)
#endif

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = MSSM_UNIFORM(static_cast<uint32_t>(v));
  const uint32_t hi = MSSM_UNIFORM(static_cast<uint32_t>(static_cast<uint64_t>(v) >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// First token of sequence q (q = n: the end of the last one), kept inside the row
// whatever the offsets hold.
__device__ __forceinline__ int64_t seq_begin(const Sequences& s, int64_t q) {
  if (!s.offsets) return q * s.L;
  const int64_t v = s.offsets[q];
  return v < 0 ? 0 : v > s.tokens ? s.tokens : v;
}

// How many q of 0 .. n have seq_begin(q) <= t (t = -1: none): t lies in sequence
// (result - 1) where that is one of 0 .. n - 1.
__device__ __forceinline__ int64_t seq_after(const Sequences& s, int64_t t) {
  if (t < 0) return 0;
  if (!s.offsets) {
    if (s.L <= 0) return s.n + 1;
    const int64_t q = s.tokens <= INT32_MAX
                          ? static_cast<int64_t>(static_cast<uint32_t>(t) / static_cast<uint32_t>(s.L))
                          : t / s.L;
    return (q < s.n ? q : s.n) + 1;
  }
  int64_t lo = 0, hi = s.n + 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (seq_begin(s, mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// The tokens t0 .. t0 + S - 1 (S up to 32) of one wavefront.  Bit s of a mask stands for token
// t0 + s.  Without borders every token is in the same sequence (or in none) and neither
// its first nor its last.
struct Span {
  bool borders = false;
  uint32_t valid = 0, first = 0, last = 0;
  int owner = 0;              // in lane s: the sequence of token t0 + s
  __device__ __forceinline__ int64_t sequence(int s) const {
    return static_cast<int64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(owner, s)));
  }
};

template <int S>
__device__ __forceinline__ Span span_of(const Sequences& seqs, int64_t t0) {
  static_assert(S <= 32, "a mask's bits");
  Span p;
  const int64_t after = uniform64(seq_after(seqs, t0 - 1));   // the first border at or after t0
  // a border at t0 + S makes the last of these tokens its sequence's last
  const bool plain = after > seqs.n || uniform64(seq_begin(seqs, after)) > t0 + S;
  if (plain) {
    p.valid = after >= 1 && after <= seqs.n ? 0xffffffffu : 0u;
    return p;
  }
  p.borders = true;
  const int lane = static_cast<int>(threadIdx.x & 63);
  const int64_t t = t0 + lane;
  const int64_t q = seq_after(seqs, t) - 1;
  const bool valid = lane < S && q >= 0 && q < seqs.n && t < seqs.tokens;
  const int64_t at = valid ? q : 0;
  p.owner = static_cast<int>(at);
  p.valid = static_cast<uint32_t>(__ballot(valid));
  p.first = static_cast<uint32_t>(__ballot(valid && seq_begin(seqs, at) == t));
  p.last = static_cast<uint32_t>(__ballot(valid && seq_begin(seqs, at + 1) == t + 1));
  return p;
}

// The sequence that a wavefront's current token is in: q, or none (not valid) before the first
// and behind the last.  begin <= t < end at the token it was made for, also for offsets
// that decrease.
struct Cursor {
  int64_t q, begin, end;
  bool valid;
};
__device__ __forceinline__ Cursor cursor_at(const Sequences& s, int64_t t) {
  Cursor c;
  const int64_t after = uniform64(seq_after(s, t));
  c.q = after - 1;
  c.valid = c.q >= 0 && c.q < s.n;
  c.begin = c.q >= 0 ? uniform64(seq_begin(s, c.q)) : 0;
  c.end = after <= s.n ? uniform64(seq_begin(s, after)) : INT64_MAX;
  return c;
}

}  // namespace mssm
