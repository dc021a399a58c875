// Linear attention with a decay for each head: how a call is cut into
// segments, the pass that joins the segments' states, the single-token step,
// the sums over heads that share queries and keys, and the order of launches.
// The matrix products are in linear_attention.h.
#include <stdint.h>

#include <initializer_list>

#include "la_args.h"
#include "linear_attention.h"
#include "mssm_internal.h"

namespace mssm {

namespace la {
#define MSSM_LA_PASS(NAME)                                              \
  hipError_t pass_##NAME##_bf16(const PassArgs& p, hipStream_t stream); \
  hipError_t pass_##NAME##_fp32(const PassArgs& p, hipStream_t stream); \
  static hipError_t pass_##NAME(mssm_dtype t, const PassArgs& p, hipStream_t stream) { \
    return t == MSSM_BFLOAT16 ? pass_##NAME##_bf16(p, stream) : pass_##NAME##_fp32(p, stream); \
  }
MSSM_LA_PASS(fwd)
MSSM_LA_PASS(state)
MSSM_LA_PASS(dq)
MSSM_LA_PASS(dk)
MSSM_LA_PASS(dv)
#undef MSSM_LA_PASS
hipError_t pass_states_bf16(const PassArgs& fwd, const PassArgs& rev, hipStream_t stream);
hipError_t pass_states_fp32(const PassArgs& fwd, const PassArgs& rev, hipStream_t stream);
hipError_t pass_dq_dv_bf16(const PassArgs& dq, const PassArgs& dv, hipStream_t stream);
hipError_t pass_dq_dv_bf16_f32(const PassArgs& dq, const PassArgs& dv, hipStream_t stream);
hipError_t pass_dq_dv_fp32(const PassArgs& dq, const PassArgs& dv, hipStream_t stream);
}  // namespace la

namespace {

using la::Grid;
using la::PassArgs;
using la::View;

// ---- the state before each segment ---------------------------------------------------------------

// Runs over a sequence's segments in order (rev: from the last): `st` holds
// each segment's own state on entry and the state the segment starts from on
// return.  A thread owns four values of one
// head's state; the segments' loads do not depend on each other and run kAhead
// ahead of the chain of multiply-adds.  A gradient's two directions are one launch.
// Bound by memory (25 segments of 20 heads of 128 x 128: 65 MB in 15 us, 4.3 TB/s).
struct Carry {
  const float* init;
  const float* decay;
  float* st;
};
__global__ __launch_bounds__(256) void la_carry(Grid grid, int heads, int64_t size, Carry fwd,
                                                Carry back) {
  const bool rev = blockIdx.z != 0;
  const float* __restrict__ init = rev ? back.init : fwd.init;
  const float* __restrict__ decay = rev ? back.decay : fwd.decay;
  float* __restrict__ st = rev ? back.st : fwd.st;
  using la::f32x4;
  constexpr int kAhead = 8;
  const int64_t i = 4 * (int64_t(blockIdx.y) * 256 + threadIdx.x);
  if (i >= size) return;
  const int64_t seq = blockIdx.x / heads;
  const int h = blockIdx.x % heads;
  int64_t first, count;
  if (grid.offsets) {
    auto at = [&](int64_t s) {
      const int64_t o = grid.offsets[s];
      return o < 0 ? int64_t(0) : (o > grid.tokens ? grid.tokens : o);
    };
    const int64_t a = at(seq), b = max(at(seq + 1), a);
    first = a / grid.seg_len + seq;
    count = max((b - a + grid.seg_len - 1) / grid.seg_len, int64_t(1));
  } else {
    first = seq * grid.segs;
    count = grid.segs;
  }
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t sh = (seq * heads + h) * size + i;
  if (init) s = f32x4{init[sh], init[sh + 1], init[sh + 2], init[sh + 3]};
  const int64_t own = count - 1;            // nothing follows the one that comes last
  for (int64_t c0 = 0; c0 < count; c0 += kAhead) {
    f32x4 u[kAhead];
    float e[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t c = c0 + k;
      const int64_t slot = first + (rev ? count - 1 - c : c);
      u[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      e[k] = 1.0f;
      if (c < own) {
        u[k] = *reinterpret_cast<const f32x4*>(st + (slot * heads + h) * size + i);
        e[k] = decay[slot * heads + h];
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t c = c0 + k;
      if (c >= count) break;
      const int64_t slot = first + (rev ? count - 1 - c : c);
      *reinterpret_cast<f32x4*>(st + (slot * heads + h) * size + i) = s;
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] = __builtin_fmaf(e[k], s[r], u[k][r]);
    }
  }
}

hipError_t launch_carry(const Grid& grid, int heads, int64_t size, const Carry& fwd,
                        const Carry* back, hipStream_t stream) {
  const dim3 g(static_cast<uint32_t>(grid.seqs * heads),
               static_cast<uint32_t>((size / 4 + 255) / 256), back ? 2 : 1);
  hipLaunchKernelGGL(la_carry, g, dim3(256), 0, stream, grid, heads, size, fwd, back ? *back : fwd);
  return hipGetLastError();
}

// ---- sums --------------------------------------------------------------------------------------------

// out[t, hk, :] = the sum over the `rep` heads that share key head hk, in their order;
// for dq and dk.  One pass over memory, a launch's length at small sizes (3 x 333, 6
// heads of 48: 4 us).
template <typename T>
__global__ __launch_bounds__(256) void la_sum_heads(const float* part_q, const float* part_k,
                                                    T* out_q, T* out_k, int64_t quads, int d,
                                                    int rep) {
  const float* __restrict__ part = blockIdx.y ? part_k : part_q;
  T* out = blockIdx.y ? out_k : out_q;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= quads) return;
  const int per = d / 4;                               // quads of a head
  const int64_t head = i / per;                        // t * key_heads + hk
  const int c = static_cast<int>(i - head * per) * 4;
  la::f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int r = 0; r < rep; ++r)
    s += *reinterpret_cast<const la::f32x4*>(part + (head * rep + r) * d + c);
  la::store4(out + head * d + c, s);
}

hipError_t launch_sum_heads(const LaShape& s, const float* part_q, const float* part_k, void* dq,
                            void* dk, int rep, mssm_dtype dtype, hipStream_t stream) {
  const int64_t quads = s.tokens * s.key_heads * s.dk / 4;
  const dim3 grid(static_cast<uint32_t>((quads + 255) / 256), 2);
  const int d = static_cast<int>(s.dk);
  if (dtype == MSSM_BFLOAT16)
    hipLaunchKernelGGL(la_sum_heads<uint16_t>, grid, dim3(256), 0, stream, part_q, part_k,
                       static_cast<uint16_t*>(dq), static_cast<uint16_t*>(dk), quads, d, rep);
  else
    hipLaunchKernelGGL(la_sum_heads<float>, grid, dim3(256), 0, stream, part_q, part_k,
                       static_cast<float*>(dq), static_cast<float*>(dk), quads, d, rep);
  return hipGetLastError();
}

// out[h] = sum over slots of part[slot, h]; one block per head.
__global__ __launch_bounds__(256) void la_sum_slots(const float* __restrict__ part, float* out,
                                                    int64_t slots, int heads) {
  __shared__ float m[4];
  float s = 0.0f;
  for (int64_t i = threadIdx.x; i < slots; i += 256) s += part[i * heads + blockIdx.x];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) m[threadIdx.x >> 6] = s;
  block_sync();
  if (threadIdx.x == 0) out[blockIdx.x] = (m[0] + m[1]) + (m[2] + m[3]);
}

// ---- one token -----------------------------------------------------------------------------------------

struct StepLaunch {
  const void *q, *k, *v;
  int64_t q_row, k_row, v_row;
  const float* g;
  int64_t g_row;
  float* state;
  void* o;
  float scale;
  int heads, rep, dk, dv;
};

// S = exp(g) S + k v^T, o = scale S^T q for one (sequence, head) per block: the
// state is read and written once, which is all the time there is (HBM bound).
// A thread owns four columns of S and every (256 / (dv / 4))-th row; the rows'
// parts of o meet in LDS.  Bound by the state, read and written once: 256 sequences
// of 20 heads of 128: 671 MB in 132 us, 5.1 TB/s, a large copy's rate.  One sequence
// of 24 heads of 64: 3.7 us, less than the host takes for the call.
template <typename T>
__global__ __launch_bounds__(256) void la_step(StepLaunch p) {
  using la::f32x4;
  __shared__ float red[1024];                          // rows in flight * dv values
  __shared__ float sk[128], sq[128];
  const int64_t b = blockIdx.x / p.heads;
  const int h = blockIdx.x % p.heads;
  const int tid = threadIdx.x;
  const int quads = p.dv / 4, groups = 256 / quads;    // 4 .. 32, 64 .. 8
  const T* q = static_cast<const T*>(p.q) + b * p.q_row + (h / p.rep) * p.dk;
  const T* k = static_cast<const T*>(p.k) + b * p.k_row + (h / p.rep) * p.dk;
  const T* v = static_cast<const T*>(p.v) + b * p.v_row + h * p.dv;
  const int rg = tid / quads, c = (tid % quads) * 4;
  const bool on = rg < groups;
  float* s = p.state + (int64_t(blockIdx.x) * p.dk) * p.dv;
  for (int i = tid; i < p.dk; i += 256) {
    sk[i] = to_float(k[i]);
    sq[i] = p.scale * to_float(q[i]);
  }
  const float a = fast_exp2(p.g[b * p.g_row + h] * kLog2e);
  f32x4 vv = {0.0f, 0.0f, 0.0f, 0.0f}, o = vv;
  if (on)
#pragma unroll
    for (int r = 0; r < 4; ++r) vv[r] = to_float(v[c + r]);
  block_sync();
  if (on) {
    for (int i = rg; i < p.dk; i += groups) {
      f32x4 x;
      __builtin_memcpy(&x, s + i * p.dv + c, 16);
      const float kk = sk[i], qq = sq[i];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[r] = __builtin_fmaf(a, x[r], kk * vv[r]);
        o[r] = __builtin_fmaf(qq, x[r], o[r]);
      }
      __builtin_memcpy(s + i * p.dv + c, &x, 16);
    }
    *reinterpret_cast<f32x4*>(&red[rg * p.dv + c]) = o;
  }
  block_sync();
  if (tid < p.dv) {
    float t = 0.0f;
    for (int r = 0; r < groups; ++r) t += red[r * p.dv + tid];
    T* out = static_cast<T*>(p.o) + (b * p.heads + h) * int64_t(p.dv) + tid;
    if constexpr (sizeof(T) == 2) *out = static_cast<T>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(t)));
    else *out = t;
  }
}

View view_of(const void* p, int64_t row, int div) {
  View v;
  v.p = p;
  v.row = row;
  v.div = div;
  return v;
}

constexpr size_t kAlign = 256;
size_t round_up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

}  // namespace

// Segments.  One block runs a segment of one head in order.  Where sequences
// times heads do not fill the compute units, sequences are cut: each segment's
// own state is found first (reading k and v once more), the states are joined,
// then all segments run at once.
LaPlan plan_la(const LaShape& s, bool backward, bool bf16) {
  LaPlan p;
  Grid& g = p.grid;
  g.seqs = s.seqs;
  g.tokens = s.tokens;
  g.L = s.packed ? 0 : (s.seqs > 0 ? s.tokens / s.seqs : 0);
  // Blocks to aim for: two on each of the 256 compute units at once, once
  // (backward) or twice over; a few blocks more than a multiple of 512 would be a
  // round of their own (1 x 131072, 20 heads of 128: 1040 blocks take 12 %
  // longer than 1000).  Twice over is better for short segments (packed prompts of
  // 32768 tokens, 32 heads of 128 x 64: 302 us, once over 342), once for those of
  // 4096 tokens and more, whose states mostly depend on a part of them (1 x 131072:
  // 940 us, twice over 1004; where they depend on all of them, log decays of -1e-4, 1061
  // and 1079).
  // A segment costs its state four times through memory,
  // as much as the tiles of max(dk, dv) or so tokens: below twice that only to
  // reach 256 blocks, and never below two chunks (4 x 2048, 16 heads of 128: 87 us
  // in segments of 256 tokens, 92 of 512, 111 of 128; 3 x 333 float32 backward, 6
  // heads: 79 us in segments of 128, 55 of 64).  From 256 sequences times heads
  // on, one segment each.
  const int64_t chunk = bf16 ? 64 : 32;
  p.paired = s.dv <= 64 && s.heads / s.key_heads % 2 == 0;
  const int64_t units = p.paired && !backward ? s.heads / 2 : s.heads;
  const int64_t rows = s.seqs * units;
  const int64_t len = s.packed ? s.tokens : g.L;      // the longest a sequence can be
  auto cut = [&](int64_t blocks) {                    // tokens of a segment for so many blocks
    if (s.packed) return (s.tokens * units + blocks - 1) / blocks;
    return rows >= 256 ? len : (len + blocks / rows - 1) / (blocks / rows);
  };
  const int64_t least = 2 * (s.dk > s.dv ? s.dk : s.dv);
  int64_t seg = cut(512);
  if (!backward && seg < 4096) seg = cut(1024);
  if (seg < least) seg = cut(256) < least ? cut(256) : least;
  if (seg < 2 * chunk) seg = 2 * chunk;
  if (seg > len) seg = len;
  seg = (seg + chunk - 1) / chunk * chunk;
  if (seg < chunk) seg = chunk;
  g.seg_len = seg;
  g.segs = s.packed ? 0 : (len + seg - 1) / seg;
  if (!s.packed && g.segs < 1) g.segs = 1;
  g.slots = s.packed ? s.tokens / seg + s.seqs : s.seqs * g.segs;
  p.cut = len > seg;

  // as many values of four bytes as the factors' product, at an aligned place
  size_t at = 0;
  auto take = [&](std::initializer_list<int64_t> factors) {
    const size_t o = at;
    size_t n = 4;
    for (int64_t f : factors) p.overflow |= __builtin_mul_overflow(n, static_cast<size_t>(f), &n);
    p.overflow |= n > SIZE_MAX / 2 || __builtin_add_overflow(at, round_up(n), &at);
    return o;
  };
  if (p.cut) {
    p.states = take({g.slots, s.heads, s.dk, s.dv});
    p.decay = take({g.slots, s.heads});
  }
  if (backward) {
    if (p.cut) {
      p.rev_states = take({g.slots, s.heads, s.dk, s.dv});
      p.rev_decay = take({g.slots, s.heads});
    }
    // Room for a whole segment's chunks and kept states in every slot, or, where packed
    // sequences are many and a segment long, for what the tokens can fill: a segment of n
    // tokens from token a on writes ceil(n / 256) states, no more than lie between
    // a / 256 + slot and the next segment's (a + n) / 256 + slot + 1.  (512 sequences of
    // 131072 tokens, 20 heads of 128: 2.8 GB, 15.5 by slots.)
    const int64_t every = 256 / chunk;
    p.chunks_per_slot = seg / chunk;
    p.dumps_per_slot = (p.chunks_per_slot + every - 1) / every;
    int64_t chunks = p.chunks_per_slot, dumps = p.dumps_per_slot;
    const bool chunks_fit = !__builtin_mul_overflow(chunks, g.slots, &chunks);
    const bool dumps_fit = !__builtin_mul_overflow(dumps, g.slots, &dumps);
    const bool fit = chunks_fit && dumps_fit;
    p.by_token = s.packed && (!fit || s.tokens / 256 + g.slots < dumps);
    if (p.by_token) {
      p.chunks_per_slot = p.dumps_per_slot = 1;
      chunks = s.tokens / chunk + g.slots;
      dumps = s.tokens / 256 + g.slots;
    } else {
      p.overflow |= !fit;
    }
    p.dumps = take({dumps, s.heads, s.dk <= 64 ? 64 : 128, s.dv <= 64 ? 64 : 128});
    p.q_sums = take({chunks, s.heads, 4});
    p.u = take({s.tokens, s.heads});
    p.head_part = take({g.slots, s.heads});
    if (s.heads != s.key_heads) {
      p.dq = take({s.tokens, s.heads, s.dk});
      p.dk = take({s.tokens, s.heads, s.dk});
    }
  }
  p.bytes = at;
  return p;
}

hipError_t launch_la_fwd(const LaArgs& a, const LaPlan& plan, void* ws, hipStream_t stream) {
  const LaShape& s = a.shape;
  const int rep = static_cast<int>(s.heads / s.key_heads);
  char* w = static_cast<char*>(ws);
  PassArgs p;
  p.grid = plan.grid;
  p.grid.offsets = a.offsets;
  p.x = view_of(a.q, a.q_row, rep);
  p.y = view_of(a.k, a.k_row, rep);
  p.z = view_of(a.v, a.v_row, 1);
  p.g = a.g;
  p.g_row = a.per_token ? s.heads : 0;
  p.heads = static_cast<int>(s.heads);
  p.dA = static_cast<int>(s.dk);
  p.dB = static_cast<int>(s.dv);
  p.scale = a.scale;
  p.paired = plan.paired;
  p.sA = s.dv;
  p.sB = 1;
  hipError_t err;
  if (plan.cut) {
    float* st = reinterpret_cast<float*>(w + plan.states);
    float* dec = reinterpret_cast<float*>(w + plan.decay);
    PassArgs q = p;
    q.seg_out = st;
    q.seg_decay = dec;
    if ((err = la::pass_state(a.dtype, q, stream)) != hipSuccess) return err;
    if ((err = launch_carry(p.grid, p.heads, s.dk * s.dv, {a.state, dec, st}, nullptr, stream)) != hipSuccess)
      return err;
    p.seg_states = st;
  }
  p.init = a.state;
  p.last = a.last;
  p.out = a.o;
  return la::pass_fwd(a.dtype, p, stream);
}

hipError_t launch_la_bwd(const LaArgs& a, const LaGrads& d, const LaPlan& plan, void* ws,
                         hipStream_t stream) {
  const LaShape& s = a.shape;
  const bool bf16 = a.dtype == MSSM_BFLOAT16;
  const int rep = static_cast<int>(s.heads / s.key_heads);
  char* w = static_cast<char*>(ws);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(w + o); };
  const View q = view_of(a.q, a.q_row, rep), k = view_of(a.k, a.k_row, rep);
  const View v = view_of(a.v, a.v_row, 1);
  const View g = view_of(d.dout, s.heads * s.dv, 1);
  PassArgs c;
  c.grid = plan.grid;
  c.grid.offsets = a.offsets;
  c.g = a.g;
  c.g_row = a.per_token ? s.heads : 0;
  c.heads = static_cast<int>(s.heads);
  c.scale = a.scale;
  const int64_t size = s.dk * s.dv;
  hipError_t err;
  if (plan.cut) {
    PassArgs p = c;
    p.y = k, p.z = v;
    p.dA = static_cast<int>(s.dk), p.dB = static_cast<int>(s.dv);
    p.sA = s.dv, p.sB = 1;
    p.paired = plan.paired;
    p.seg_out = at(plan.states);
    p.seg_decay = at(plan.decay);
    PassArgs r = p;
    r.y = q, r.z = g;
    r.seg_out = at(plan.rev_states);
    r.seg_decay = at(plan.rev_decay);
    err = bf16 ? la::pass_states_bf16(p, r, stream) : la::pass_states_fp32(p, r, stream);
    if (err != hipSuccess) return err;
    const Carry back = {d.dlast, at(plan.rev_decay), at(plan.rev_states)};
    if ((err = launch_carry(c.grid, c.heads, size, {a.state, at(plan.decay), at(plan.states)}, &back,
                            stream)) != hipSuccess)
      return err;
  }
  c.u = at(plan.u);
  c.q_sums = at(plan.q_sums);
  c.dumps = at(plan.dumps);
  c.chunks_per_slot = plan.chunks_per_slot;
  c.dumps_per_slot = plan.dumps_per_slot;
  c.by_token = plan.by_token;
  {
    PassArgs p = c;
    p.x = g, p.y = v, p.z = k, p.e = q;
    p.dA = static_cast<int>(s.dv), p.dB = static_cast<int>(s.dk);
    p.sA = 1, p.sB = s.dv;
    p.init = a.state;
    p.seg_states = plan.cut ? at(plan.states) : nullptr;
    p.out = rep > 1 ? at(plan.dq) : d.dq;
    p.out_f32 = rep > 1;
    PassArgs r = c;
    r.x = k, r.y = q, r.z = g;
    r.dA = static_cast<int>(s.dk), r.dB = static_cast<int>(s.dv);
    r.sA = s.dv, r.sB = 1;
    r.init = d.dlast;
    r.seg_states = plan.cut ? at(plan.rev_states) : nullptr;
    r.paired = plan.paired;
    r.out = d.dv;
    // One launch where both fit on the chip at once (3 x 333 float32, 6 heads: the call
    // 56 us, 65 with two); larger ones are faster apart (4 x 8192, 16 heads of 128: 738
    // and 746 us), each with its own registers.
    if (plan.grid.slots * s.heads <= 256) {
      err = !bf16 ? la::pass_dq_dv_fp32(p, r, stream)
            : p.out_f32 ? la::pass_dq_dv_bf16_f32(p, r, stream)
                        : la::pass_dq_dv_bf16(p, r, stream);
    } else if ((err = la::pass_dq(a.dtype, p, stream)) == hipSuccess) {
      err = la::pass_dv(a.dtype, r, stream);
    }
    if (err != hipSuccess) return err;
  }
  {
    PassArgs p = c;
    p.x = v, p.y = g, p.z = q, p.e = k;
    p.dA = static_cast<int>(s.dv), p.dB = static_cast<int>(s.dk);
    p.sA = 1, p.sB = s.dv;
    p.init = d.dlast;
    p.seg_states = plan.cut ? at(plan.rev_states) : nullptr;
    // dstate is written here, where the adjoint is walked for the last time and the
    // states are no longer read: it may then be dlast (each block has read its own part)
    // or the state.
    p.last = d.dstate;
    p.out = rep > 1 ? at(plan.dk) : d.dk;
    p.out_f32 = rep > 1;
    p.dg = a.per_token ? d.dg : nullptr;
    p.head_part = a.per_token ? nullptr : at(plan.head_part);
    if ((err = la::pass_dk(a.dtype, p, stream)) != hipSuccess) return err;
  }
  if (rep > 1 && s.tokens > 0) {
    err = launch_sum_heads(s, at(plan.dq), at(plan.dk), d.dq, d.dk, rep, a.dtype, stream);
    if (err != hipSuccess) return err;
  }
  if (!a.per_token) {
    hipLaunchKernelGGL(la_sum_slots, dim3(static_cast<uint32_t>(s.heads)), dim3(256), 0, stream,
                       at(plan.head_part), d.dg, plan.grid.slots, c.heads);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t launch_la_no_heads(const LaShape& s, void* dq, void* dk, mssm_dtype dtype,
                              hipStream_t stream) {
  return launch_sum_heads(s, nullptr, nullptr, dq, dk, 0, dtype, stream);   // sums over none
}

hipError_t launch_la_step(const LaArgs& a, float* state, hipStream_t stream) {
  const LaShape& s = a.shape;
  StepLaunch p{a.q, a.k, a.v, a.q_row, a.k_row, a.v_row, a.g, a.per_token ? s.heads : 0,
               state, a.o, a.scale, static_cast<int>(s.heads),
               static_cast<int>(s.heads / s.key_heads), static_cast<int>(s.dk),
               static_cast<int>(s.dv)};
  const dim3 grid(static_cast<uint32_t>(s.seqs * s.heads));
  if (a.dtype == MSSM_BFLOAT16)
    hipLaunchKernelGGL(la_step<uint16_t>, grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(la_step<float>, grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace mssm
