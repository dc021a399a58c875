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
// A wavefront takes kSteps tokens of 64 V channels (a lane holds V channels) and a block kWaves
// wavefronts behind one another: a tile.  Every affine map h -> P h + H of a wavefront's
// tokens is formed from registers; the wavefronts' maps are joined in LDS, the tiles'
// by a pass over them.
#include <type_traits>

#include "mssm_internal.h"
#include "recurrence_device.h"

namespace mssm {

namespace {

constexpr int kWaves = 8;
constexpr int kBlock = 64 * kWaves;

template <typename T>
constexpr int kSteps = sizeof(T) == 2 ? 16 : 8;   // tokens of a wavefront
template <typename T>
constexpr int kTile = kWaves * kSteps<T>;

// Joins the affine map (P, H) behind state h.  P = 0 stands for a sequence's first token in between
// (or a decay of nothing): what h was, infinite or NaN too, is forgotten.
__device__ __forceinline__ float join(float P, float H, float h) {
  return P == 0.0f ? H : __builtin_fmaf(P, h, H);
}

struct Place {
  int64_t tile, t0;       // t0: the wavefront's first token
  int wave, lane;
  int c;                  // the lane's first channel
  bool active;            // not a copy of another lane
};

template <typename T, int V>
__device__ __forceinline__ Place place_of(int64_t D, int64_t groups, int64_t block) {
  Place p;
  p.wave = MSSM_UNIFORM(static_cast<int>(threadIdx.x >> 6));
  p.lane = static_cast<int>(threadIdx.x & 63);
  p.tile = block / groups;
  const int64_t c0 = (block % groups) * (64 * V) + p.lane * V;
  p.active = c0 < D;
  p.c = static_cast<int>(c0 < D - V ? c0 : D - V);
  p.t0 = p.tile * kTile<T> + p.wave * kSteps<T>;
  return p;
}

// kSteps rows of a tensor from token t0 on, each lane its V channels.
template <typename T, int V, int S>
__device__ __forceinline__ void load_rows(const void* base, int64_t row, int64_t t0, int64_t tokens,
                                          int c, Raw<T, V> (&v)[S]) {
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int64_t t = t0 + s < tokens ? t0 + s : tokens - 1;
    v[s].load(static_cast<const T*>(base) + t * row + c);
  }
}

// agg: [tiles, D] (P, H) of each tile, written without kOut; carry: [tiles, D] the state
// before each tile, read with kOut (null: zero, for a single tile).
template <typename T, int V, bool kOut>
__global__ __launch_bounds__(kBlock) void recurrence_kernel(RecurrenceArgs a, int64_t groups,
                                                            float2* agg, const float* carry) {
  constexpr int S = kSteps<T>;
  __shared__ float sp[kWaves][64 * V], sh[kWaves][64 * V];
  const int64_t D = a.D;
  const Place p = place_of<T, V>(D, groups, blockIdx.x);
  Raw<T, V> x[S], gi[S], gr[S];
  load_rows<T, V, S>(a.r, a.r_row, p.t0, a.seqs.tokens, p.c, gr);
  load_rows<T, V, S>(a.i, a.i_row, p.t0, a.seqs.tokens, p.c, gi);
  load_rows<T, V, S>(a.x, a.x_row, p.t0, a.seqs.tokens, p.c, x);
  float rate[V];
#pragma unroll
  for (int v = 0; v < V; ++v) rate[v] = a.A[p.c + v];
  const Span span = span_of<S>(a.seqs, p.t0);

  float da[S][V], b[S][V];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Decay d = decay_of(rate[v], gr[s].get(v));
      da[s][v] = d.a;
      b[s][v] = sqrt_(d.m2) * sigmoid(gi[s].get(v)) * x[s].get(v);
    }
  if (span.borders && a.state) {
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (span.first >> s & 1) {
        const float* h0 = a.state + span.sequence(s) * D + p.c;
#pragma unroll
        for (int v = 0; v < V; ++v) b[s][v] = __builtin_fmaf(da[s][v], h0[v], b[s][v]);
      }
  }
  float P[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) P[v] = 1.0f, H[v] = 0.0f;
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (span.first >> s & 1) P[v] = 0.0f, H[v] = b[s][v];
      else H[v] = __builtin_fmaf(da[s][v], H[v], b[s][v]), P[v] *= da[s][v];
    }
#pragma unroll
  for (int v = 0; v < V; ++v) sp[p.wave][p.lane * V + v] = P[v], sh[p.wave][p.lane * V + v] = H[v];
  block_sync();
  if constexpr (!kOut) {
    if (p.wave == 0 && p.active) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float pp = 1.0f, hh = 0.0f;
        for (int w = 0; w < kWaves; ++w) {
          const float q = sp[w][p.lane * V + v];
          hh = join(q, sh[w][p.lane * V + v], hh);
          pp = q == 0.0f ? 0.0f : pp * q;
        }
        agg[p.tile * D + p.c + v] = make_float2(pp, hh);
      }
    }
    return;
  }
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = carry ? carry[p.tile * D + p.c + v] : 0.0f;
    for (int w = 0; w < p.wave; ++w)
      h[v] = join(sp[w][p.lane * V + v], sh[w][p.lane * V + v], h[v]);
  }
  if (!p.active) return;
  T* out = static_cast<T*>(a.h) + p.t0 * D + p.c;
#pragma unroll
  for (int s = 0; s < S; ++s) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      h[v] = span.first >> s & 1 ? b[s][v] : __builtin_fmaf(da[s][v], h[v], b[s][v]);
    if ((span.valid >> s & 1) && p.t0 + s < a.seqs.tokens) Raw<T, V>::store(out + s * D, h);
    if (a.last && (span.last >> s & 1)) {
      float* to = a.last + span.sequence(s) * D + p.c;
#pragma unroll
      for (int v = 0; v < V; ++v) to[v] = h[v];
    }
  }
}

// carry[tile] = the state before it, over the tiles in order (backward: behind it, from
// the last one back).
__global__ __launch_bounds__(64) void recurrence_carry_kernel(const float2* __restrict__ agg,
                                                              float* __restrict__ carry,
                                                              int64_t tiles, int64_t D,
                                                              int backward) {
  const int64_t c = int64_t(blockIdx.x) * 64 + threadIdx.x;
  if (c >= D) return;
  float h = 0.0f;
  for (int64_t j0 = 0; j0 < tiles; j0 += 16) {
    float2 u[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int64_t k = j0 + j < tiles ? j0 + j : tiles - 1;
      u[j] = agg[(backward ? tiles - 1 - k : k) * D + c];
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int64_t k = j0 + j;
      if (k < tiles) {
        carry[(backward ? tiles - 1 - k : k) * D + c] = h;
        h = join(u[j].x, u[j].y, h);
      }
    }
  }
}

// Sequences without tokens: to = from, or zero.
__global__ __launch_bounds__(256) void empty_states_kernel(Sequences seqs, const float* from,
                                                           float* to, int64_t D) {
  const int64_t q = blockIdx.x;
  if (seq_begin(seqs, q + 1) > seq_begin(seqs, q)) return;
  for (int64_t c = threadIdx.x; c < D; c += 256) to[q * D + c] = from ? from[q * D + c] : 0.0f;
}

// ragg: [tiles, D] (P, H) of each tile's map of psi, written without kOut; rcarry: psi behind
// each tile (null: zero); saved: the state before each tile (null: zero); part: [tiles, D]
// the tiles' sums of dA.
template <typename T, int V, bool kOut>
__global__ __launch_bounds__(kBlock) void recurrence_bwd_kernel(RecurrenceArgs a, RecurrenceGrads d,
                                                                int64_t groups, float2* ragg,
                                                                const float* rcarry,
                                                                const float* saved, float* part) {
  constexpr int S = kSteps<T>;
  __shared__ float sp[kWaves][64 * V], sh[kWaves][64 * V], sq[kWaves][64 * V];
  const int64_t D = a.D;
  const Place p = place_of<T, V>(D, groups, blockIdx.x);
  Raw<T, V> x[S], gi[S], gr[S], dh[S];
  load_rows<T, V, S>(a.r, a.r_row, p.t0, a.seqs.tokens, p.c, gr);
  load_rows<T, V, S>(d.dh, D, p.t0, a.seqs.tokens, p.c, dh);
  if constexpr (kOut) {
    load_rows<T, V, S>(a.i, a.i_row, p.t0, a.seqs.tokens, p.c, gi);
    load_rows<T, V, S>(a.x, a.x_row, p.t0, a.seqs.tokens, p.c, x);
  }
  float rate[V];
#pragma unroll
  for (int v = 0; v < V; ++v) rate[v] = a.A[p.c + v];
  const Span span = span_of<S>(a.seqs, p.t0);
  auto dstate = [&](int s, int v) {
    return d.dlast ? d.dlast[span.sequence(s) * D + p.c + v] : 0.0f;
  };

  float P[V], H[V];      // psi before the wavefront's tokens = P psi behind them + H
#pragma unroll
  for (int v = 0; v < V; ++v) P[v] = 1.0f, H[v] = 0.0f;
  float da[S][V];
#pragma unroll
  for (int s = S - 1; s >= 0; --s)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      da[s][v] = decay_of(rate[v], gr[s].get(v)).a;
      if (p.t0 + s >= a.seqs.tokens) continue;
      if (span.last >> s & 1) P[v] = 0.0f, H[v] = dstate(s, v);
      H[v] = da[s][v] * (dh[s].get(v) + H[v]);
      P[v] = P[v] == 0.0f ? 0.0f : P[v] * da[s][v];
    }
#pragma unroll
  for (int v = 0; v < V; ++v) sp[p.wave][p.lane * V + v] = P[v], sh[p.wave][p.lane * V + v] = H[v];
  if constexpr (!kOut) {
    block_sync();
    if (p.wave == 0 && p.active) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float pp = 1.0f, hh = 0.0f;
        for (int w = kWaves - 1; w >= 0; --w) {
          const float q = sp[w][p.lane * V + v];
          hh = join(q, sh[w][p.lane * V + v], hh);
          pp = q == 0.0f ? 0.0f : pp * q;
        }
        ragg[p.tile * D + p.c + v] = make_float2(pp, hh);
      }
    }
    return;
  }
  // the states: the wavefront's own map first, joined behind the earlier ones'
  float hp[S][V];        // h_{t-1}
  float Pf[V], Hf[V];
  {
#pragma unroll
    for (int v = 0; v < V; ++v) Pf[v] = 1.0f, Hf[v] = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const Decay k = decay_of(rate[v], gr[s].get(v));
        const float b = sqrt_(k.m2) * sigmoid(gi[s].get(v)) * x[s].get(v);
        if (span.first >> s & 1) {
          const float h0 = a.state ? a.state[span.sequence(s) * D + p.c + v] : 0.0f;
          Pf[v] = 0.0f, Hf[v] = __builtin_fmaf(da[s][v], h0, b);
        } else {
          Hf[v] = __builtin_fmaf(da[s][v], Hf[v], b), Pf[v] *= da[s][v];
        }
        hp[s][v] = b;    // for now: the input term
      }
  }
  float psi[V], h[V];
  block_sync();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    psi[v] = rcarry ? rcarry[p.tile * D + p.c + v] : 0.0f;
    for (int w = kWaves - 1; w > p.wave; --w)
      psi[v] = join(sp[w][p.lane * V + v], sh[w][p.lane * V + v], psi[v]);
  }
  block_sync();
#pragma unroll
  for (int v = 0; v < V; ++v) sp[p.wave][p.lane * V + v] = Pf[v], sh[p.wave][p.lane * V + v] = Hf[v];
  block_sync();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = saved ? saved[p.tile * D + p.c + v] : 0.0f;
    for (int w = 0; w < p.wave; ++w)
      h[v] = join(sp[w][p.lane * V + v], sh[w][p.lane * V + v], h[v]);
  }
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (span.first >> s & 1) h[v] = a.state ? a.state[span.sequence(s) * D + p.c + v] : 0.0f;
      const float b = hp[s][v];
      hp[s][v] = h[v];
      h[v] = __builtin_fmaf(da[s][v], h[v], b);
    }
  float sum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) sum[v] = 0.0f;
#pragma unroll
  for (int s = S - 1; s >= 0; --s) {
    if (p.t0 + s >= a.seqs.tokens) continue;
    const bool valid = span.valid >> s & 1;
    float dx[V], di[V], dr[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (span.last >> s & 1) psi[v] = dstate(s, v);
      const float lam = dh[s].get(v) + psi[v];
      const Decay k = decay_of(rate[v], gr[s].get(v));
      const float w = k.m2 > 0.0f ? rsqrt_(k.m2) : 0.0f;          // 1 / m
      const float m = k.m2 * w;
      const float g = sigmoid(gi[s].get(v)), gx = g * x[s].get(v);
      dx[v] = lam * m * g;
      di[v] = lam * m * gx * (1.0f - g);
      const float e = lam * k.a * (hp[s][v] - gx * k.a * w);
      const float es = e * k.s;
      dr[v] = es * rate[v] * (1.0f - k.s);
      if (valid) sum[v] += es;
      psi[v] = k.a * lam;
    }
    if (p.active && valid) {
      const int64_t at = (p.t0 + s) * D + p.c;
      Raw<T, V>::store(static_cast<T*>(d.dx) + at, dx);
      Raw<T, V>::store(static_cast<T*>(d.di) + at, di);
      Raw<T, V>::store(static_cast<T*>(d.dr) + at, dr);
      if (d.dstate && (span.first >> s & 1)) {
        float* to = d.dstate + span.sequence(s) * D + p.c;
#pragma unroll
        for (int v = 0; v < V; ++v) to[v] = psi[v];
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) sq[p.wave][p.lane * V + v] = sum[v];
  block_sync();
  if (p.wave == 0 && p.active) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float t = 0.0f;
      for (int w = 0; w < kWaves; ++w) t += sq[w][p.lane * V + v];
      part[p.tile * D + p.c + v] = t;
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
  if (c < D)
    for (int64_t r = w; r < rows; r += 16) s += part[r * D + c];
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
    const Decay d = decay_of(a.A[c + v], gr.get(v));
    const float b = sqrt_(d.m2) * sigmoid(gi.get(v)) * x.get(v);
    h[v] = __builtin_fmaf(d.a, state[q * a.D + c + v], b);
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

int64_t tile_of(mssm_dtype dtype) {
  return dtype == MSSM_BFLOAT16 ? kTile<uint16_t> : kTile<float>;
}
size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Calls f with the element type and the channels a lane holds: two, or one for up to 64 channels,
// which fill a wavefront only so.
template <typename F>
hipError_t with_type(mssm_dtype dtype, int64_t D, F f) {
  if (dtype == MSSM_BFLOAT16)
    return D > 64 ? f(uint16_t(), std::integral_constant<int, 2>())
                  : f(uint16_t(), std::integral_constant<int, 1>());
  return D > 64 ? f(float(), std::integral_constant<int, 2>())
                : f(float(), std::integral_constant<int, 1>());
}

}  // namespace

RecurrencePlan plan_recurrence(int64_t tokens, int64_t D, bool backward, bool saved,
                               mssm_dtype dtype) {
  RecurrencePlan p;
  p.tiles = (tokens + tile_of(dtype) - 1) / tile_of(dtype);
  p.groups = (D + (D > 64 ? 127 : 63)) / (D > 64 ? 128 : 64);
  const size_t states = static_cast<size_t>(p.tiles) * D;
  p.saved_bytes = states * sizeof(float);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  if (p.tiles > 1) p.agg = take(states * sizeof(float2));
  if (p.tiles > 1 && !saved) p.states = take(states * sizeof(float));
  if (backward) {
    if (p.tiles > 1) p.rcarry = take(states * sizeof(float));
    p.part = take(states * sizeof(float));
  }
  p.bytes = off;
  return p;
}

namespace {

hipError_t empty_states(const Sequences& s, const float* from, float* to, int64_t D,
                        hipStream_t stream) {
  for (int64_t q = 0; q < s.n; q += 1 << 22) {       // a launch's blocks
    const int64_t n = s.n - q < (1 << 22) ? s.n - q : 1 << 22;
    Sequences part = s;
    if (part.offsets) part.offsets += q;
    part.n = n;
    hipLaunchKernelGGL(empty_states_kernel, dim3(static_cast<uint32_t>(n)), dim3(256), 0, stream,
                       part, from ? from + q * D : nullptr, to + q * D, D);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The states before every tile, into carry.
hipError_t tile_states(const RecurrenceArgs& a, const RecurrencePlan& p, char* ws, float* carry,
                       hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(p.tiles * p.groups));
  float2* agg = reinterpret_cast<float2*>(ws + p.agg);
  const hipError_t e = with_type(a.dtype, a.D, [&](auto t, auto v) {
    hipLaunchKernelGGL((recurrence_kernel<decltype(t), decltype(v)::value, false>), grid,
                       dim3(kBlock), 0, stream, a, p.groups, agg, nullptr);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(recurrence_carry_kernel, dim3(static_cast<uint32_t>((a.D + 63) / 64)), dim3(64),
                     0, stream, agg, carry, p.tiles, a.D, 0);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_recurrence(const RecurrenceArgs& a, const RecurrencePlan& p, void* ws_,
                             hipStream_t stream) {
  char* ws = static_cast<char*>(ws_);
  if (a.last && (a.seqs.offsets || a.seqs.L == 0)) {
    const hipError_t e = empty_states(a.seqs, a.state, a.last, a.D, stream);
    if (e != hipSuccess) return e;
  }
  if (a.seqs.tokens == 0) return hipSuccess;
  float* carry = nullptr;
  if (p.tiles > 1) {
    carry = a.saved ? a.saved : reinterpret_cast<float*>(ws + p.states);
    const hipError_t e = tile_states(a, p, ws, carry, stream);
    if (e != hipSuccess) return e;
  } else if (a.saved) {
    hipLaunchKernelGGL(recurrence_zero_kernel, dim3(static_cast<uint32_t>((a.D + 255) / 256)),
                       dim3(256), 0, stream, a.saved, a.D);
  }
  const dim3 grid(static_cast<uint32_t>(p.tiles * p.groups));
  return with_type(a.dtype, a.D, [&](auto t, auto v) {
    hipLaunchKernelGGL((recurrence_kernel<decltype(t), decltype(v)::value, true>), grid,
                       dim3(kBlock), 0, stream, a, p.groups, nullptr, carry);
    return hipGetLastError();
  });
}

hipError_t launch_recurrence_bwd(const RecurrenceArgs& a, const RecurrenceGrads& d,
                                 const RecurrencePlan& p, void* ws_, hipStream_t stream) {
  char* ws = static_cast<char*>(ws_);
  if (d.dstate && (a.seqs.offsets || a.seqs.L == 0)) {
    const hipError_t e = empty_states(a.seqs, d.dlast, d.dstate, a.D, stream);
    if (e != hipSuccess) return e;
  }
  if (a.seqs.tokens == 0) {
    hipLaunchKernelGGL(recurrence_zero_kernel, dim3(static_cast<uint32_t>((a.D + 255) / 256)),
                       dim3(256), 0, stream, d.dA, a.D);
    return hipGetLastError();
  }
  const dim3 grid(static_cast<uint32_t>(p.tiles * p.groups));
  const float* states = nullptr;
  float* rcarry = nullptr;
  float* part = reinterpret_cast<float*>(ws + p.part);
  if (p.tiles > 1) {
    float2* agg = reinterpret_cast<float2*>(ws + p.agg);
    states = a.saved;
    if (!states) {
      float* to = reinterpret_cast<float*>(ws + p.states);
      const hipError_t e = tile_states(a, p, ws, to, stream);
      if (e != hipSuccess) return e;
      states = to;
    }
    rcarry = reinterpret_cast<float*>(ws + p.rcarry);
    const hipError_t e = with_type(a.dtype, a.D, [&](auto t, auto v) {
      hipLaunchKernelGGL((recurrence_bwd_kernel<decltype(t), decltype(v)::value, false>), grid,
                         dim3(kBlock), 0, stream, a, d, p.groups, agg, nullptr, nullptr, nullptr);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(recurrence_carry_kernel, dim3(static_cast<uint32_t>((a.D + 63) / 64)),
                       dim3(64), 0, stream, agg, rcarry, p.tiles, a.D, 1);
  }
  const hipError_t e = with_type(a.dtype, a.D, [&](auto t, auto v) {
    hipLaunchKernelGGL((recurrence_bwd_kernel<decltype(t), decltype(v)::value, true>), grid,
                       dim3(kBlock), 0, stream, a, d, p.groups, nullptr, rcarry, states, part);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(recurrence_sum_kernel, dim3(static_cast<uint32_t>((a.D + 63) / 64)),
                     dim3(1024), 0, stream, part, p.tiles, a.D, d.dA);
  return hipGetLastError();
}

hipError_t launch_recurrence_step(const RecurrenceArgs& a, float* state, hipStream_t stream) {
  return with_type(a.dtype, a.D, [&](auto t, auto v) {
    constexpr int V = decltype(v)::value;
    const int64_t threads = a.seqs.n * ((a.D + V - 1) / V);
    hipLaunchKernelGGL((recurrence_step_kernel<decltype(t), V>),
                       dim3(static_cast<uint32_t>((threads + 255) / 256)), dim3(256), 0, stream, a,
                       state);
    return hipGetLastError();
  });
}

}  // namespace mssm
