// Gated linear recurrence: forward, one token, gradient (gfx950).
//
// Per channel with a rate A, for each token's x and gates i, r:
//   s = sigmoid(r), a = exp(A s), m = sqrt(1 - a^2), g = sigmoid(i)
//   h_t = a h_{t-1} + b_t,  b = m g x
// and backwards, with psi_t = a_t lambda_t the gradient that reaches h_{t-1}:
//   lambda_t = dh_t + psi_{t+1}
//   dx = lambda m g,   di = lambda b (1 - g),
//   e = lambda (a h_{t-1} - g x a^2 / m)      (the gradient of log a: dm / dlog a = -a^2 / m)
//   dr = e A s (1 - s),   dA = sum over tokens of e s.
//
// A wavefront takes a few tokens of 64 V channels (a lane holds V channels) and a block
// several wavefronts behind one another: a tile.  The affine map h -> P h + H of a wavefront's tokens
// is formed from registers and the wavefronts' maps are joined in LDS, so every input is read
// once.  Tiles of the same channels form a chain: a block publishes its tile's map, then
// looks back over the tiles before it for the nearest one whose state is known, takes that state
// through the maps in between, and publishes its own.  Blocks take their tiles in the order in which
// they start (a counter for each chain), so the tiles that one waits for are all being worked on, and the
// first of them waits for none.  A state is always made by the same operations from the one
// before it, wherever the look-back began: results do not depend on the timing.
//
// Memory is the floor (5.1 TB/s of a large copy), and how fast a state goes along a chain what bounds it:
// kLookBack tiles a poll, which one wavefront makes while its block's others wait.  With every compute
// unit loading and storing a poll takes near 4 us, and a chain goes on by some 1.6 tiles a microsecond,
// be it one of 20 (bfloat16, 1 x 131072 x 2560: 1024 tiles in 630 us, 4.3 TB/s; floor 522) or of 16 (packed
// 32768 x 2048 with states: 256 tiles in 170 us; floor 104).  With one to four chains a poll takes 1.4 us and
// the time follows the tokens, not the width: 131072 x 64, 128, 256, 512 162, 248, 249, 258 us (floors 13
// to 104).  The gradient alike, in tiles of 64 tokens: 4 x 8192 x 2048 280 us (3.4 TB/s; floor 183),
// 1 x 32768 x 128 85 us.  One token of 256 x 5120 6 us.
#include <type_traits>

#include "mssm_internal.h"
#include "recurrence_device.h"

namespace mssm {

namespace {

constexpr int kSavedTokens = 64;          // a saved state for every so many tokens
// Tiles looked at together (131072 x 2560 bf16, 645 us with 6 when these were tried: 8 and 10, which
// spill, 656 and 839).
constexpr int kLookBack = 6;
constexpr int kMaxPolls = 1 << 22;
constexpr int64_t kTicketStride = 32;     // counters on cache lines of their own

// A wavefront's tokens and a block's wavefronts.  Forward: tiles of 128 tokens (float32: 64) of 128
// channels, two blocks a compute unit.  A tile of 131072 x 2560 bf16 takes 15 us: ticket 1, loads 3, gates
// 3, its wavefronts 3, look-back 4.  Where that workload took 645 us, four wavefronts took 850, 8 tokens
// 887, sixteen wavefronts 1130, four channels a lane 1180, and one block that loads ahead 780.
template <typename T>
struct Forward {
  static constexpr int S = sizeof(T) == 2 ? 16 : 8, W = 8;
};
// All tokens in one tile: shorter chains of operations (45 x 1536 bf16: kernel 6.3 us, 10.4 with tiles of
// 128).
template <typename T>
struct Short {
  static constexpr int S = 4, W = 16;
};
// Backward: a tile for each saved state (training pass 4 x 8192 x 2048 bf16, 432 us when these were
// tried: 4 tokens by sixteen wavefronts 444, tiles and states of 32 tokens 523).
template <typename T>
struct Backward {
  static constexpr int S = 8, W = 8;
};

// Joins the affine map (P, H) behind state h.  P = 0 stands for a sequence's first token in between:
// what h was, infinite or NaN too, is forgotten.
__device__ __forceinline__ float join(float P, float H, float h) {
  return P == 0.0f ? H : __builtin_fmaf(P, h, H);
}

// A product of decays within a sequence.  Where float32 rounds it to zero it is the smallest number above
// instead, 2^-149, which adds at most 5e-7 to a state: what is infinite or NaN goes on through
// the sequence, as it does token by token.
__device__ __forceinline__ float within(float P) { return P == 0.0f ? __uint_as_float(1u) : P; }

// A chain's slots, [tiles, D]: a tile's map (P, H) in one word, or its state, marked by P = -1
// (decays are not negative), or nothing yet (all bits set, which no map is).  A word is written and
// read whole, so it needs no other order.
constexpr uint32_t kEmpty = 0xffffffffu, kState = 0xbf800000u, kNan = 0x7fc00000u;

__device__ __forceinline__ void publish(uint64_t* slot, uint32_t P, float H) {
  __hip_atomic_store(slot, static_cast<uint64_t>(__float_as_uint(H)) << 32 | P, __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}

// The state before the chain's tile j, whose map is (P, H): one wavefront, each lane its V channels
// from c on.  Also publishes the tile's map and its state.  (The tiles it waits for are being
// worked on, some microseconds each; should another call overwrite the workspace meanwhile, the
// wait still ends, seconds later, with NaN.)
template <int V>
__device__ __forceinline__ void look_back(uint64_t* slots, int64_t j, int64_t D, int c,
                                          const float (&P)[V], const float (&H)[V], float (&h)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = 0.0f;
  if (j > 0) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      publish(slots + j * D + c + v, P[v] == P[v] ? __float_as_uint(P[v]) : kNan, H[v]);
    for (int polls = 0;; ++polls) {
      uint64_t w[kLookBack][V];
#pragma unroll
      for (int i = 0; i < kLookBack; ++i) {
        const int64_t k = j - 1 - i > 0 ? j - 1 - i : 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
          w[i][v] = __hip_atomic_load(slots + k * D + c + v, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT);
      }
      bool known = true;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        bool found = false;
        h[v] = 0.0f;
#pragma unroll
        for (int i = kLookBack - 1; i >= 0; --i) {      // from the farthest on
          const uint32_t p = static_cast<uint32_t>(w[i][v]);
          const float u = __uint_as_float(static_cast<uint32_t>(w[i][v] >> 32));
          h[v] = p == kState ? u : join(__uint_as_float(p), u, h[v]);
          // (P = 0: a sequence begins in the tile, and H is the state)
          found = (found || p == kState || p == 0) && p != kEmpty;
        }
        known = known && found;
      }
      if (__all(known)) break;
      if (polls == kMaxPolls) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = __uint_as_float(kNan);
        break;
      }
      __builtin_amdgcn_s_sleep(1);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) publish(slots + j * D + c + v, kState, join(P[v], H[v], h[v]));
}

// Before a pass: the slots are set to "nothing yet" and the chains' counters to zero (by the first
// clear_blocks blocks), and sequences without tokens pass their state on, to = from or zero.
struct Prepare {
  uint4* slots;
  int64_t n;
  uint32_t* tickets;
  int64_t groups;
  int64_t clear_blocks;
  Sequences seqs;
  const float* from;
  float* to;
  int64_t D;
};
__global__ __launch_bounds__(256) void recurrence_prepare_kernel(Prepare a) {
  if (blockIdx.x < a.clear_blocks) {
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    for (int64_t k = i; k < a.n; k += a.clear_blocks * 256)
      a.slots[k] = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
    for (int64_t k = i; k < a.groups; k += a.clear_blocks * 256) a.tickets[k * kTicketStride] = 0;
    return;
  }
  for (int64_t q = blockIdx.x - a.clear_blocks; q < a.seqs.n; q += gridDim.x - a.clear_blocks) {
    if (seq_begin(a.seqs, q + 1) > seq_begin(a.seqs, q)) continue;
    for (int64_t c = threadIdx.x; c < a.D; c += 256) {
      const int64_t e = q * a.D + c;
      a.to[e] = a.from ? a.from[e] : 0.0f;
    }
  }
}

// A barrier for what lies in LDS alone: loads and stores in flight go on.
__device__ __forceinline__ void lds_sync() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

struct Place {
  int64_t link;           // the tile's place in its chain
  int64_t t0;             // the wavefront's first token
  int wave, lane;
  int c;                  // the lane's first channel
  bool active;            // not a copy of another lane
};

// tiles: how many a chain has; with one there is nothing to take a ticket for.  (Every block gets a
// tile; one beyond them, which only a workspace in use elsewhere could give, is not worked on.)
template <int V, int S, int W, bool kReverse>
__device__ __forceinline__ Place place_of(int64_t D, int64_t groups, int64_t tiles,
                                          uint32_t* tickets) {
  __shared__ uint32_t ticket;
  Place p;
  p.wave = MSSM_UNIFORM(static_cast<int>(threadIdx.x >> 6));
  p.lane = static_cast<int>(threadIdx.x & 63);
  const int64_t group = blockIdx.x % groups;
  p.link = 0;
  if (tiles > 1) {
    if (threadIdx.x == 0)
      ticket = __hip_atomic_fetch_add(tickets + group * kTicketStride, 1u, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT);
    lds_sync();
    p.link = MSSM_UNIFORM(ticket);
  }
  const int64_t c0 = group * (64 * V) + p.lane * V;
  p.active = c0 < D;
  p.c = static_cast<int>(c0 < D - V ? c0 : D - V);
  p.t0 = (kReverse ? tiles - 1 - p.link : p.link) * (W * S) + p.wave * S;
  return p;
}

// What the wavefronts of a block tell one another.
template <int V, int W>
struct Maps {
  float p[W][64 * V], h[W][64 * V], in[64 * V];
  __device__ __forceinline__ void put(const Place& at, const float (&P)[V], const float (&H)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) p[at.wave][at.lane * V + v] = P[v], h[at.wave][at.lane * V + v] = H[v];
  }
  // The map of all wavefronts' tokens, in the chain's order.
  template <bool kReverse>
  __device__ __forceinline__ void all(int lane, float (&P)[V], float (&H)[V]) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      P[v] = 1.0f, H[v] = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const int w = kReverse ? W - 1 - k : k;
        const float q = p[w][lane * V + v];
        H[v] = join(q, h[w][lane * V + v], H[v]);
        P[v] = q == 0.0f || P[v] == 0.0f ? 0.0f : within(P[v] * q);
      }
    }
  }
  // The state x before the block's tokens, taken to the wavefront's own.
  template <bool kReverse>
  __device__ __forceinline__ void take(const Place& at, float (&x)[V]) const {
#pragma unroll
    for (int v = 0; v < V; ++v)
      for (int k = 0; k < (kReverse ? W - 1 - at.wave : at.wave); ++k) {
        const int w = kReverse ? W - 1 - k : k;
        x[v] = join(p[w][at.lane * V + v], h[w][at.lane * V + v], x[v]);
      }
  }
};

// The state (backward: psi) before this wavefront's tokens.  P, H: its own map.
template <int V, int W, bool kReverse>
__device__ __forceinline__ void chain(const Place& at, Maps<V, W>& m, uint64_t* slots, int64_t tiles,
                                      int64_t D, const float (&P)[V], const float (&H)[V],
                                      float (&x)[V]) {
  m.put(at, P, H);
  lds_sync();
  if (tiles > 1) {
    if (at.wave == 0) {
      float tp[V], th[V];
      m.template all<kReverse>(at.lane, tp, th);
      look_back<V>(slots, at.link, D, at.c, tp, th, x);
#pragma unroll
      for (int v = 0; v < V; ++v) m.in[at.lane * V + v] = x[v];
    }
    lds_sync();
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = m.in[at.lane * V + v];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = 0.0f;
  }
  m.template take<kReverse>(at, x);
}

// h (kOut) and the last and saved states.
template <typename T, int V, int S, int W, bool kOut>
__global__ __launch_bounds__(64 * W, 4) void recurrence_kernel(RecurrenceArgs a, int64_t groups,
                                                               int64_t tiles, uint32_t* tickets,
                                                               uint64_t* slots) {
  __shared__ Maps<V, W> maps;
  const int64_t D = a.D;
  const Place p = place_of<V, S, W, false>(D, groups, tiles, tickets);
  if (p.link >= tiles) return;
  Raw<T, V> x[S], gi[S], gr[S];
  load_rows<T, V, S>(a.r, a.r_row, D, p.t0, a.seqs.tokens, p.c, gr);
  load_rows<T, V, S>(a.i, a.i_row, D, p.t0, a.seqs.tokens, p.c, gi);
  load_rows<T, V, S>(a.x, a.x_row, D, p.t0, a.seqs.tokens, p.c, x);
  float rate[V];
  bool near = true;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    rate[v] = a.A[p.c + v];
    near = near && rate[v] > kSeries;
  }
  const Span span = span_of<S>(a.seqs, p.t0);

  float da[S][V], b[S][V];
  auto gates = [&](auto near_) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        constexpr bool kNear = decltype(near_)::value;
        const float q = decay_of<kNear>(rate[v] * sigmoid(gr[s].get(v)));
        da[s][v] = decay<kNear>(q);
        b[s][v] = sqrt_(one_minus_square<kNear>(q)) * (sigmoid(gi[s].get(v)) * x[s].get(v));
      }
  };
  if (__all(near)) gates(std::true_type());
  else gates(std::false_type());

  float P[V], H[V], h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) P[v] = 1.0f, H[v] = 0.0f;
  if (!span.borders) {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int v = 0; v < V; ++v) H[v] = __builtin_fmaf(da[s][v], H[v], b[s][v]), P[v] *= da[s][v];
  } else {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (span.first >> s & 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (a.state)
            b[s][v] = __builtin_fmaf(da[s][v], a.state[span.sequence(s) * D + p.c + v], b[s][v]);
          P[v] = 0.0f, H[v] = b[s][v];
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) H[v] = __builtin_fmaf(da[s][v], H[v], b[s][v]), P[v] *= da[s][v];
      }
    }
  }
  if (!span.first) {
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = within(P[v]);
  }
  chain<V, W, false>(p, maps, slots, tiles, D, P, H, h);
  if (!p.active) return;
  if (a.saved && p.t0 % kSavedTokens == 0 && p.t0 < a.seqs.tokens) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.saved[p.t0 / kSavedTokens * D + p.c + v] = h[v];
  }
  if constexpr (!kOut) return;
  const int step = static_cast<int>(D * sizeof(T));
  const buf_t out = rows_from<S>(a.h, p.t0, step, step);
  const int at = p.c * static_cast<int>(sizeof(T));
  if (!span.borders) {
    if (!span.valid) return;
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(da[s][v], h[v], b[s][v]);
      Raw<T, V>::store(out, at, s * step, h);
    }
  } else {
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        h[v] = span.first >> s & 1 ? b[s][v] : __builtin_fmaf(da[s][v], h[v], b[s][v]);
      if (span.valid >> s & 1) Raw<T, V>::store(out, at, s * step, h);
      if (a.last && (span.last >> s & 1)) {
        float* to = a.last + span.sequence(s) * D + p.c;
#pragma unroll
        for (int v = 0; v < V; ++v) to[v] = h[v];
      }
    }
  }
}

// saved: the state before each tile (null: zero); part: [tiles, D] the tiles' sums of dA.
template <typename T, int V>
__global__ __launch_bounds__(64 * Backward<T>::W, 4) void recurrence_bwd_kernel(
    RecurrenceArgs a, RecurrenceGrads d, int64_t groups, int64_t tiles, uint32_t* tickets,
    uint64_t* slots, const float* saved, float* part) {
  constexpr int S = Backward<T>::S, W = Backward<T>::W;
  static_assert(S * W == kSavedTokens, "a saved state for each tile");
  __shared__ Maps<V, W> fwd, rev;
  const int64_t D = a.D;
  const Place p = place_of<V, S, W, true>(D, groups, tiles, tickets);
  if (p.link >= tiles) return;
  const int64_t tile = tiles - 1 - p.link;
  float rate[V], h[V], psi[V], sum[V];
  Raw<T, V> x[S], dh[S], gi[S], gr[S];
  load_rows<T, V, S>(a.r, a.r_row, D, p.t0, a.seqs.tokens, p.c, gr);
  load_rows<T, V, S>(a.i, a.i_row, D, p.t0, a.seqs.tokens, p.c, gi);
  load_rows<T, V, S>(a.x, a.x_row, D, p.t0, a.seqs.tokens, p.c, x);
  load_rows<T, V, S>(d.dh, D, D, p.t0, a.seqs.tokens, p.c, dh);
  bool near = true;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    rate[v] = a.A[p.c + v];
    near = near && rate[v] > kSeries;
    h[v] = saved ? saved[tile * D + p.c + v] : 0.0f;
    sum[v] = 0.0f;
  }
  const Span span = span_of<S>(a.seqs, p.t0);
  auto state = [&](int s, int v) {
    return a.state ? a.state[span.sequence(s) * D + p.c + v] : 0.0f;
  };
  auto dlast = [&](int s, int v) {
    return d.dlast ? d.dlast[span.sequence(s) * D + p.c + v] : 0.0f;
  };

  // (the wavefronts of a block have the same channels: all of them take the same branch)
  auto work = [&](auto near_) __attribute__((always_inline)) {
    constexpr bool kNear = decltype(near_)::value;
    // sigmoid(r), a, sigmoid(i) and that times x, m; the input term, then h_{t-1}
    Gate sg[S][V], g[S][V];
    float k[S][V], gx[S][V], m[S][V], bb[S][V];
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float open = sg[s][v].make(gr[s].get(v));
        const float q = decay_of<kNear>(rate[v] * open);
        k[s][v] = decay<kNear>(q);
        m[s][v] = sqrt_(one_minus_square<kNear>(q));
        gx[s][v] = g[s][v].make(gi[s].get(v)) * x[s].get(v);
        bb[s][v] = m[s][v] * gx[s][v];
      }

    // The wavefront's maps: of the state, and of psi (from behind its tokens to before them).
    float P[V], H[V], Pf[V], Hf[V];
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = Pf[v] = 1.0f, H[v] = Hf[v] = 0.0f;
    if (!span.borders) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          Hf[v] = __builtin_fmaf(k[s][v], Hf[v], bb[s][v]), Pf[v] *= k[s][v];
          H[v] = k[S - 1 - s][v] * (dh[S - 1 - s].get(v) + H[v]);
        }
#pragma unroll
      for (int v = 0; v < V; ++v) P[v] = Pf[v];
    } else {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (span.first >> s & 1) Pf[v] = 0.0f, Hf[v] = __builtin_fmaf(k[s][v], state(s, v), bb[s][v]);
          else Hf[v] = __builtin_fmaf(k[s][v], Hf[v], bb[s][v]), Pf[v] *= k[s][v];
        }
#pragma unroll
      for (int s = S - 1; s >= 0; --s)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (span.last >> s & 1) P[v] = 0.0f, H[v] = dlast(s, v);
          H[v] = k[s][v] * (dh[s].get(v) + H[v]);
          P[v] = P[v] == 0.0f ? 0.0f : P[v] * k[s][v];
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!span.first) Pf[v] = within(Pf[v]);
      if (!span.last) P[v] = within(P[v]);
    }
    fwd.put(p, Pf, Hf);
    chain<V, W, true>(p, rev, slots, tiles, D, P, H, psi);     // (its barrier is fwd's too)
    fwd.template take<false>(p, h);
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (span.borders && (span.first >> s & 1)) h[v] = state(s, v);
        const float b = bb[s][v];
        bb[s][v] = h[v];
        h[v] = __builtin_fmaf(k[s][v], h[v], b);
      }
    const int step = static_cast<int>(D * sizeof(T));
    const buf_t to_x = rows_from<S>(d.dx, p.t0, step, step), to_i = rows_from<S>(d.di, p.t0, step, step),
                to_r = rows_from<S>(d.dr, p.t0, step, step);
    // (lanes that copy another's channels write out of bounds, which is dropped)
    const int at = p.active ? p.c * static_cast<int>(sizeof(T)) : S * step;
    // Gradients of token s; psi goes from behind it to before it.
    auto token = [&](int s) __attribute__((always_inline)) {
      float dx[V], di[V], dr[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float lam = dh[s].get(v) + psi[v], a = k[s][v];
        const float w = m[s][v] > 0.0f ? __builtin_amdgcn_rcpf(m[s][v]) : 0.0f;
        const float lm = lam * m[s][v], li = lm * gx[s][v];
        dx[v] = lm * g[s][v].value();
        di[v] = li * g[s][v].rest();
        psi[v] = a * lam;
        const float es = psi[v] * __builtin_fmaf(-gx[s][v] * a, w, bb[s][v]) * sg[s][v].value();
        dr[v] = es * rate[v] * sg[s][v].rest();
        sum[v] += es;
      }
      Raw<T, V>::store(to_x, at, s * step, dx);
      Raw<T, V>::store(to_i, at, s * step, di);
      Raw<T, V>::store(to_r, at, s * step, dr);
    };
    if (!span.borders) {
      if (span.valid) {
#pragma unroll
        for (int s = S - 1; s >= 0; --s) token(s);
      }
    } else {
#pragma unroll
      for (int s = S - 1; s >= 0; --s) {
        if (!(span.valid >> s & 1)) continue;
        if (span.last >> s & 1) {
#pragma unroll
          for (int v = 0; v < V; ++v) psi[v] = dlast(s, v);
        }
        token(s);
        if (d.dstate && p.active && (span.first >> s & 1)) {
          float* to = d.dstate + span.sequence(s) * D + p.c;
#pragma unroll
          for (int v = 0; v < V; ++v) to[v] = psi[v];
        }
      }
    }
  };
  if (__all(near)) work(std::true_type());
  else work(std::false_type());
  block_sync();
#pragma unroll
  for (int v = 0; v < V; ++v) rev.p[p.wave][p.lane * V + v] = sum[v];
  block_sync();
  if (p.wave == 0 && p.active) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float t = 0.0f;
      for (int w = 0; w < W; ++w) t += rev.p[w][p.lane * V + v];
      part[tile * D + p.c + v] = t;
    }
  }
}

// out[c] = the sum over the rows of part, in a fixed order.
__global__ __launch_bounds__(1024) void recurrence_sum_kernel(const float* __restrict__ part,
                                                              int64_t rows, int64_t D, float* out) {
  __shared__ double m[16][64];
  const int col = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = int64_t(blockIdx.x) * 64 + col;
  double s = 0.0;
  if (c < D) {
#pragma unroll 8
    for (int64_t r = w; r < rows; r += 16) s += part[r * D + c];
  }
  m[w][col] = s;
  block_sync();
  if (w == 0 && c < D) {
    for (int k = 1; k < 16; ++k) s += m[k][col];
    out[c] = static_cast<float>(s);
  }
}

template <typename T, int V>
__global__ __launch_bounds__(256) void recurrence_step_kernel(RecurrenceArgs a, float* state) {
  const int64_t groups = (a.D + V - 1) / V;
  const int64_t n = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t q = n / groups;
  if (q >= a.seqs.n) return;
  const int64_t c0 = (n - q * groups) * V;
  const int64_t c = c0 < a.D - V ? c0 : a.D - V;
  Raw<T, V> x, gi, gr;
  x.load(static_cast<const T*>(a.x) + q * a.x_row + c);
  gi.load(static_cast<const T*>(a.i) + q * a.i_row + c);
  gr.load(static_cast<const T*>(a.r) + q * a.r_row + c);
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float k = decay_of<false>(a.A[c + v] * sigmoid(gr.get(v)));
    const float b = sqrt_(one_minus_square<false>(k)) * (sigmoid(gi.get(v)) * x.get(v));
    h[v] = __builtin_fmaf(decay<false>(k), state[q * a.D + c + v], b);
  }
  // (where V does not divide D, the last thread's first channels are another's)
  if (c == c0) {
#pragma unroll
    for (int v = 0; v < V; ++v) state[q * a.D + c + v] = h[v];
    Raw<T, V>::store(static_cast<T*>(a.h) + q * a.D + c, h);
  } else {
    state[q * a.D + a.D - 1] = h[V - 1];
    const float last[1] = {h[V - 1]};
    Raw<T, 1>::store(static_cast<T*>(a.h) + q * a.D + a.D - 1, last);
  }
}

__global__ __launch_bounds__(256) void recurrence_zero_kernel(float* p, int64_t n) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

int64_t fwd_tile(mssm_dtype dtype) {
  return dtype == MSSM_BFLOAT16 ? Forward<uint16_t>::S * Forward<uint16_t>::W
                                : Forward<float>::S * Forward<float>::W;
}
size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Channels a lane holds: two, or one for up to 64 channels, which fill a wavefront only so.  The
// backward kernel keeps more numbers a channel and takes one (two spill registers: training
// pass 4 x 8192 x 2048 bf16 480 us, 445 with one).
constexpr int kBackwardChannels = 1;
int lane_channels(int64_t D) { return D > 64 ? 2 : 1; }

// Calls f with the element type and the channels a lane holds.
template <typename F>
hipError_t with_type(mssm_dtype dtype, int V, F f) {
  if (dtype == MSSM_BFLOAT16)
    return V == 2 ? f(uint16_t(), std::integral_constant<int, 2>())
                  : f(uint16_t(), std::integral_constant<int, 1>());
  return V == 2 ? f(float(), std::integral_constant<int, 2>())
                : f(float(), std::integral_constant<int, 1>());
}

}  // namespace

RecurrencePlan plan_recurrence(int64_t tokens, int64_t D, bool backward, bool saved,
                               mssm_dtype dtype) {
  RecurrencePlan p;
  p.tiles = (tokens + fwd_tile(dtype) - 1) / fwd_tile(dtype);
  p.bwd_tiles = (tokens + kSavedTokens - 1) / kSavedTokens;
  auto groups = [&](bool back) {
    const int64_t wide = 64 * (back ? kBackwardChannels : lane_channels(D));
    return (D + wide - 1) / wide;
  };
  p.groups = groups(false);
  p.bwd_groups = groups(true);
  const size_t states = static_cast<size_t>(p.bwd_tiles) * D * sizeof(float);
  p.saved_bytes = states;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  // the two directions follow one another and share the counters and slots
  const int64_t links = backward ? p.bwd_tiles : p.tiles;
  if (links > 1) {
    p.tickets = take(static_cast<size_t>(backward ? p.bwd_groups : p.groups) * kTicketStride *
                     sizeof(uint32_t));
    p.slots = take(static_cast<size_t>(links) * D * sizeof(uint64_t));
  }
  if (backward) {
    if (p.bwd_tiles > 1 && !saved) p.states = take(states);
    p.part = take(states);
  }
  p.bytes = off;
  return p;
}

namespace {

// links: of a chain, to be cleared where there are several; from, to: what sequences without tokens
// pass on, with to.
hipError_t prepare(const RecurrencePlan& p, int64_t links, int64_t groups, const Sequences& seqs,
                   const float* from, float* to, int64_t D, char* ws, hipStream_t stream) {
  Prepare a;
  const bool clear = links > 1, states = to && seqs.n > 0 && (seqs.offsets || seqs.L == 0);
  if (!clear && !states) return hipSuccess;
  a.slots = reinterpret_cast<uint4*>(ws + p.slots);
  a.n = (links * D + 1) / 2;                         // (slots end at a multiple of 256 bytes)
  a.tickets = reinterpret_cast<uint32_t*>(ws + p.tickets);
  a.groups = groups;
  a.clear_blocks = !clear ? 0 : a.n < 2048 * 256 ? (a.n + 255) / 256 : 2048;
  a.seqs = seqs;
  a.from = from;
  a.to = to;
  a.D = D;
  const int64_t more = !states ? 0 : seqs.n < 65536 ? seqs.n : 65536;
  hipLaunchKernelGGL(recurrence_prepare_kernel, dim3(static_cast<uint32_t>(a.clear_blocks + more)),
                     dim3(256), 0, stream, a);
  return hipGetLastError();
}

// h, last and saved states; kOut false: the saved states alone.
template <bool kOut>
hipError_t forward(const RecurrenceArgs& a, const RecurrencePlan& p, char* ws, hipStream_t stream) {
  const hipError_t e = prepare(p, p.tiles, p.groups, a.seqs, a.state, a.last, a.D, ws, stream);
  if (e != hipSuccess || a.seqs.tokens == 0) return e;
  return with_type(a.dtype, lane_channels(a.D), [&](auto t, auto v) {
    using T = decltype(t);
    auto go = [&](auto shape) {
      using Shape = decltype(shape);
      hipLaunchKernelGGL((recurrence_kernel<T, decltype(v)::value, Shape::S, Shape::W, kOut>),
                         dim3(static_cast<uint32_t>(p.tiles * p.groups)), dim3(64 * Shape::W), 0,
                         stream, a, p.groups, p.tiles, reinterpret_cast<uint32_t*>(ws + p.tickets),
                         reinterpret_cast<uint64_t*>(ws + p.slots));
      return hipGetLastError();
    };
    if constexpr (kOut)
      if (a.seqs.tokens <= Short<T>::S * Short<T>::W) return go(Short<T>());
    return go(Forward<T>());
  });
}

}  // namespace

hipError_t launch_recurrence(const RecurrenceArgs& a, const RecurrencePlan& p, void* ws,
                             hipStream_t stream) {
  return forward<true>(a, p, static_cast<char*>(ws), stream);
}

hipError_t launch_recurrence_bwd(const RecurrenceArgs& a, const RecurrenceGrads& d,
                                 const RecurrencePlan& p, void* ws_, hipStream_t stream) {
  char* ws = static_cast<char*>(ws_);
  const float* saved = nullptr;
  hipError_t e;
  if (p.bwd_tiles > 1) {
    saved = a.saved;
    if (!saved) {
      RecurrenceArgs f = a;
      f.saved = reinterpret_cast<float*>(ws + p.states);
      f.last = nullptr;
      if ((e = forward<false>(f, p, ws, stream)) != hipSuccess) return e;
      saved = f.saved;
    }
  }
  e = prepare(p, p.bwd_tiles, p.bwd_groups, a.seqs, d.dlast, d.dstate, a.D, ws, stream);
  if (e != hipSuccess) return e;
  if (a.seqs.tokens == 0) {
    hipLaunchKernelGGL(recurrence_zero_kernel, dim3(static_cast<uint32_t>((a.D + 255) / 256)),
                       dim3(256), 0, stream, d.dA, a.D);
    return hipGetLastError();
  }
  float* part = reinterpret_cast<float*>(ws + p.part);
  const dim3 grid(static_cast<uint32_t>(p.bwd_tiles * p.bwd_groups));
  auto go = [&](auto t) {
    using T = decltype(t);
    hipLaunchKernelGGL((recurrence_bwd_kernel<T, kBackwardChannels>), grid,
                       dim3(64 * Backward<T>::W), 0, stream, a, d, p.bwd_groups, p.bwd_tiles,
                       reinterpret_cast<uint32_t*>(ws + p.tickets),
                       reinterpret_cast<uint64_t*>(ws + p.slots), saved, part);
    return hipGetLastError();
  };
  e = a.dtype == MSSM_BFLOAT16 ? go(uint16_t()) : go(float());
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(recurrence_sum_kernel, dim3(static_cast<uint32_t>((a.D + 63) / 64)),
                     dim3(1024), 0, stream, part, p.bwd_tiles, a.D, d.dA);
  return hipGetLastError();
}

hipError_t launch_recurrence_step(const RecurrenceArgs& a, float* state, hipStream_t stream) {
  return with_type(a.dtype, lane_channels(a.D), [&](auto t, auto v) {
    constexpr int V = decltype(v)::value;
    const int64_t threads = a.seqs.n * ((a.D + V - 1) / V);
    hipLaunchKernelGGL((recurrence_step_kernel<decltype(t), V>),
                       dim3(static_cast<uint32_t>((threads + 255) / 256)), dim3(256), 0, stream, a,
                       state);
    return hipGetLastError();
  });
}

}  // namespace mssm
