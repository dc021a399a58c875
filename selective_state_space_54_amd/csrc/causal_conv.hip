// Causal depthwise convolution with sequence states: forward, one token, gradient (gfx950).
//
//   c_t = bias + sum_i w_i u_{t - (k - 1) + i},   y_t = c_t or SiLU(c_t)
// where the k - 1 places before a sequence's first token are its state's rows (or zero).  With
// dz_t = dy_t (times SiLU'(c_t)):
//   du_t = sum_i w_i dz_{t + (k - 1) - i}   over the sequence's own tokens, for the state's rows
//          too; the last k - 1 places also get the last state's gradient
//   dw_i = sum_t dz_t u_{t - (k - 1) + i},   dbias = sum_t dz_t.
//
// A wavefront takes a run of consecutive tokens of 64 V channels, the last k - 1 inputs in
// registers.  Bound by memory: a run reads k - 1 rows beside its own (the gradient 2 (k - 1)).  Two
// batches of rows take turns in registers, the next on its way while one is worked on, and no
// branch stands around their loads and stores: what is not to be written goes to a buffer
// of no bytes.  A batch with a border between sequences goes token by token instead.
// One of 8 tokens is then read again, k rows a token: 2048 sequences of 16 x 2048 in bfloat16, every second
// batch of which has one, take 100 us (floor 62) and their gradient 176 (93); 512 of 64 50 and 114.
// The gradient in bfloat16 keeps 4 channels a lane, which spills 17, 95 and 163 registers at 6, 7 and 8
// taps: 16 x 2048 x 5120 296, 726 and 1102 us, 224 at 5.
// bfloat16, k = 4: packed 32768 x 5120 in 23 sequences 135 to 141 us (4.9 TB/s; 184 with branches and a
// launch of its own for the last states), the gradient of 16 x 2048 x 5120 219 us (4.6 TB/s; 250), one token
// of 256 x 5120 6 us.
#include <type_traits>

#include "mssm_internal.h"
#include "recurrence_device.h"

namespace mssm {

namespace {

constexpr int kWaves = 4;
constexpr int kBlock = 64 * kWaves;
constexpr int kBatch = 8;             // tokens loaded together
// Bytes a lane holds and tokens a run at most, forward and backward.  Packed 32768 x 5120 bf16: 4 bytes
// and runs of 32 tokens 135 us, 64 tokens 138, 128 tokens 143; 8 bytes and 64 tokens 141.  The gradient of
// 16 x 2048 x 5120: 8 bytes and runs of 64 or 128 tokens 219 us, 256 tokens 231, 32 tokens 255.
constexpr int kFwdBytes = 4, kBwdBytes = 8;
constexpr int64_t kFwdRun = 32, kBwdRun = 128;
constexpr int64_t kWavesWanted = 4096;

struct Lane {
  int64_t group, run;
  int lane, c;
  bool active;
};

// Wavefronts in the order of their groups; the wavefronts of a backward block share a group.
template <int V>
__device__ __forceinline__ Lane lane_of(int64_t D, int64_t group, int64_t run) {
  Lane p;
  p.group = group, p.run = run;
  p.lane = static_cast<int>(threadIdx.x & 63);
  const int64_t c0 = group * (64 * V) + p.lane * V;
  p.active = c0 < D;
  p.c = static_cast<int>(c0 < D - V ? c0 : D - V);
  return p;
}

template <typename T, int V>
__device__ __forceinline__ void widen(const Raw<T, V>& r, float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = r.get(j);
}

// The input at place `at` of the cursor's sequence (valid, at < end): a token's, or one of the state's
// K - 1 rows before it.
template <typename T, int V, int K>
__device__ __forceinline__ void load_place(const ConvArgs& a, const Cursor& q, int64_t at, int c,
                                           float (&v)[V]) {
  Raw<T, V> r;
  r.clear();
  if (at >= q.begin)
    r.load(static_cast<const T*>(a.u) + at * a.u_row + c);
  else if (a.state)
    r.load(static_cast<const T*>(a.state) + (q.q * (K - 1) + (at - q.begin) + (K - 1)) * a.D + c);
  r.keep();
  widen(r, v);
}

// win[j] = the input K - 1 - j places before token t of the cursor's sequence (zero outside of one).
template <typename T, int V, int K>
__device__ __forceinline__ void load_window(const ConvArgs& a, const Cursor& q, int64_t t, int c,
                                            float (&win)[K > 1 ? K - 1 : 1][V]) {
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    if (q.valid) {
      load_place<T, V, K>(a, q, t - (K - 1) + j, c, win[j]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) win[j][v] = 0.0f;
    }
  }
}

template <typename T, int V, int K>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int c, float (&w)[K][V], float (&b)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    b[v] = a.bias ? a.bias[c + v] : 0.0f;
#pragma unroll
    for (int i = 0; i < K; ++i) w[i][v] = a.weight[int64_t(c + v) * K + i];
  }
}

// The last k - 1 places of each sequence, as they are: block `block` of `blocks`.
template <typename T>
__device__ __forceinline__ void copy_last(const ConvArgs& a, int64_t block, int64_t blocks) {
  constexpr int64_t kPiece = 2048;
  const int64_t K1 = a.k - 1, pieces = (K1 * a.D + kPiece - 1) / kPiece;
  const T* u = static_cast<const T*>(a.u);
  const T* state = static_cast<const T*>(a.state);
  for (int64_t w = block; w < a.seqs.n * pieces; w += blocks) {
    const int64_t q = w / pieces, e0 = (w - q * pieces) * kPiece;
    const int64_t begin = seq_begin(a.seqs, q), end = seq_begin(a.seqs, q + 1);
    const int64_t n = end > begin ? end - begin : 0;
    T* last = static_cast<T*>(a.last) + q * K1 * a.D;
    for (int64_t e = e0 + threadIdx.x; e < e0 + kPiece && e < K1 * a.D; e += kBlock) {
      const int64_t j = e / a.D, c = e - j * a.D;
      const int64_t at = n + j - K1;                 // token of the sequence, or before it
      last[e] = at >= 0 ? u[(begin + at) * a.u_row + c]
                        : state ? state[(q * K1 + n + j) * a.D + c] : T();
    }
  }
}

// A buffer that takes what is written at rows of a batch, or nothing.
__device__ __forceinline__ buf_t when(bool open, const char* base, int bytes) {
  return make_buf(base, open ? static_cast<uint32_t>(bytes) : 0u);
}

// Blocks past the first `main` copy the last states.
template <typename T, int V, int K>
__global__ __launch_bounds__(kBlock, 2) void conv_kernel(ConvArgs a, int64_t groups, int64_t len,
                                                      int64_t main) {
  if (blockIdx.x >= main) {
    copy_last<T>(a, blockIdx.x - main, gridDim.x - main);
    return;
  }
  const int64_t id = int64_t(blockIdx.x) * kWaves + MSSM_UNIFORM(static_cast<int>(threadIdx.x >> 6));
  const Lane p = lane_of<V>(a.D, id % groups, id / groups);
  const int64_t T0 = a.seqs.tokens;
  const int64_t t0 = p.run * len;
  if (t0 >= T0) return;                       // no barriers in this kernel
  const int64_t t1 = t0 + len < T0 ? t0 + len : T0;
  using Batch = Raw<T, V>[kBatch];
  Batch u[2];
  auto load = [&](Batch& to, int64_t tb) __attribute__((always_inline)) {
    load_rows<T, V, kBatch>(a.u, a.u_row, a.D, tb, t1, p.c, to);    // (no rows past the run's)
  };
  load(u[0], t0);
  float w[K][V], bias[V], win[K > 1 ? K - 1 : 1][V];
  load_taps<T, V, K>(a, p.c, w, bias);
  Cursor q = cursor_at(a.seqs, t0);
  load_window<T, V, K>(a, q, t0, p.c, win);
  const int step = static_cast<int>(a.D * sizeof(T));
  // (lanes that copy another's channels write out of bounds, which is dropped)
  const int at = p.active ? p.c * static_cast<int>(sizeof(T)) : kBatch * step;
  auto work = [&](Batch& now, int64_t tb) __attribute__((always_inline)) {
    const char* y = static_cast<const char*>(a.y) + tb * step;
    if (tb + kBatch <= q.end) {
      const buf_t to = when(q.valid, y, kBatch * step);
#pragma unroll
      for (int s = 0; s < kBatch; ++s) {
        float cur[V], out[V];
        widen(now[s], cur);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float c = bias[v];
#pragma unroll
          for (int i = 0; i < K - 1; ++i) c = __builtin_fmaf(w[i][v], win[i][v], c);
          c = __builtin_fmaf(w[K - 1][v], cur[v], c);
          out[v] = a.silu ? silu(c) : c;
        }
        Raw<T, V>::store(to, at, s * step, out);
        if constexpr (K > 1) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int i = 0; i < K - 2; ++i) win[i][v] = win[i + 1][v];
            win[K - 2][v] = cur[v];
          }
        }
      }
      return;
    }
    const int64_t te = tb + kBatch < t1 ? tb + kBatch : t1;
#pragma unroll 1
    for (int64_t t = tb; t < te; ++t) {
      if (t >= q.end) q = cursor_at(a.seqs, t);
      if (!q.valid) continue;
      float c[V];
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = bias[v];
#pragma unroll
      for (int i = 0; i < K; ++i) {
        float cur[V];
        load_place<T, V, K>(a, q, t - (K - 1) + i, p.c, cur);
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = __builtin_fmaf(w[i][v], cur[v], c[v]);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = a.silu ? silu(c[v]) : c[v];
      Raw<T, V>::store(when(true, y, kBatch * step), at, static_cast<int>(t - tb) * step, c);
    }
    if (te < t1) {
      if (te >= q.end) q = cursor_at(a.seqs, te);
      load_window<T, V, K>(a, q, te, p.c, win);
    }
  };
  for (int64_t tb = t0; tb < t1;) {
    load(u[1], tb + kBatch);
    work(u[0], tb);
    tb += kBatch;
    if (tb >= t1) break;
    load(u[0], tb + kBatch);
    work(u[1], tb);
    tb += kBatch;
  }
}

// part: [rows of blocks, K + 1, D]: the blocks' sums for the taps and the bias.
template <typename T, int V, int K>
__global__ __launch_bounds__(kBlock, 2) void conv_bwd_kernel(ConvArgs a, ConvGrads d, int64_t groups,
                                                             int64_t len, float* part) {
  __shared__ float m[kWaves][(K + 1) * V][64];
  const int wave = MSSM_UNIFORM(static_cast<int>(threadIdx.x >> 6));
  const int64_t brow = blockIdx.x / groups;
  const Lane p = lane_of<V>(a.D, blockIdx.x % groups, brow * kWaves + wave);
  const int64_t T0 = a.seqs.tokens;
  const int64_t t0 = p.run * len;
  const int64_t t1 = t0 + len < T0 ? t0 + len : T0;
  float dw[K][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.0f;
#pragma unroll
    for (int i = 0; i < K; ++i) dw[i][v] = 0.0f;
  }
  if (t0 < T0) {
    using Batch = Raw<T, V>[kBatch];
    Batch u[2], g[2];
    const int64_t stop = t1 + K - 1;            // tokens up to t1 + K - 2 reach back into the run
    const int64_t end = stop < T0 ? stop : T0;
    auto load = [&](int k, int64_t tb) __attribute__((always_inline)) {
      load_rows<T, V, kBatch>(a.u, a.u_row, a.D, tb, end, p.c, u[k]);
      load_rows<T, V, kBatch>(d.dy, a.D, a.D, tb, end, p.c, g[k]);
    };
    load(0, t0);
    float w[K][V], bias[V], win[K > 1 ? K - 1 : 1][V];
    load_taps<T, V, K>(a, p.c, w, bias);
    Cursor q = cursor_at(a.seqs, t0);
    load_window<T, V, K>(a, q, t0, p.c, win);
    const int step = static_cast<int>(a.D * sizeof(T));
    const int at = p.active ? p.c * static_cast<int>(sizeof(T)) : kBatch * step;
    float acc[K][V];              // du of the places t - (K - 1) .. t, so far
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[j][v] = 0.0f;
    // du of a state's row is complete: written by the run that has the sequence's first token.
    auto emit_state = [&](int64_t place, const float (&val)[V]) __attribute__((always_inline)) {
      if (d.dstate && q.begin >= t0 && q.begin < t1 && p.active)
        Raw<T, V>::store(static_cast<T*>(d.dstate) +
                             (q.q * (K - 1) + (place - q.begin) + (K - 1)) * a.D + p.c, val);
    };
    // The sequence ends before token t: the K - 1 places before t are complete.
    auto flush = [&](int64_t t) __attribute__((always_inline)) {
      if (!q.valid) return;
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        float val[V];
#pragma unroll
        for (int v = 0; v < V; ++v) val[v] = acc[j][v];
        if (d.dlast) {
          Raw<T, V> r;
          r.load(static_cast<const T*>(d.dlast) + (q.q * (K - 1) + j) * a.D + p.c);
#pragma unroll
          for (int v = 0; v < V; ++v) val[v] += r.get(v);
        }
        const int64_t place = t - (K - 1) + j;
        if (place < q.begin) emit_state(place, val);
        else if (place >= t0 && place < t1 && p.active)
          Raw<T, V>::store(static_cast<T*>(d.du) + place * a.D + p.c, val);
      }
    };
    // Token t of the cursor's sequence with its input and gradient: the sums for the taps, and what it
    // adds to the places it reaches; the oldest of them is complete then, in acc[0].
    auto token = [&](int64_t t, const float (&cur)[V], float (&dz)[V]) __attribute__((always_inline)) {
      if (a.silu) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float c = bias[v];
#pragma unroll
          for (int i = 0; i < K - 1; ++i) c = __builtin_fmaf(w[i][v], win[i][v], c);
          c = __builtin_fmaf(w[K - 1][v], cur[v], c);
          const float e = sigmoid(c);
          dz[v] *= e * __builtin_fmaf(c, 1.0f - e, 1.0f);
        }
      }
      if (t < t1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
          for (int i = 0; i < K - 1; ++i) dw[i][v] = __builtin_fmaf(dz[v], win[i][v], dw[i][v]);
          dw[K - 1][v] = __builtin_fmaf(dz[v], cur[v], dw[K - 1][v]);
          db[v] += dz[v];
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < K; ++j)             // place t - (K - 1) + j meets tap j
          acc[j][v] = __builtin_fmaf(w[j][v], dz[v], acc[j][v]);
    };
    auto move_on = [&](const float (&cur)[V]) __attribute__((always_inline)) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) acc[j][v] = acc[j + 1][v];
        acc[K - 1][v] = 0.0f;
        if constexpr (K > 1) {
#pragma unroll
          for (int i = 0; i < K - 2; ++i) win[i][v] = win[i + 1][v];
          win[K - 2][v] = cur[v];
        }
      }
    };
    auto work = [&](int k, int64_t tb) __attribute__((always_inline)) {
      // the row that token tb completes
      const char* du = static_cast<const char*>(d.du) + (tb - (K - 1)) * step;
      if (tb + kBatch <= q.end && tb - (K - 1) >= q.begin) {
        if (!q.valid) return;
#pragma unroll
        for (int s = 0; s < kBatch; ++s) {
          const int64_t t = tb + s, place = t - (K - 1);
          float cur[V], dz[V];
          widen(u[k][s], cur);
          widen(g[k][s], dz);
          token(t, cur, dz);
          Raw<T, V>::store(when(place >= t0 && place < t1, du, kBatch * step), at, s * step, acc[0]);
          move_on(cur);
        }
        return;
      }
      const int64_t te = tb + kBatch < stop ? tb + kBatch : stop;
#pragma unroll 1
      for (int64_t t = tb; t < te; ++t) {
        if (t >= q.end) {                       // (past the last token: no sequence)
          flush(t);
#pragma unroll
          for (int j = 0; j < K; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) acc[j][v] = 0.0f;
          q = cursor_at(a.seqs, t);
          load_window<T, V, K>(a, q, t, p.c, win);
        }
        if (!q.valid) continue;
        const int64_t place = t - (K - 1);
        float cur[V], dz[V];
        Raw<T, V> r;
        load_place<T, V, K>(a, q, t, p.c, cur);
        r.load(static_cast<const T*>(d.dy) + t * a.D + p.c);
        r.keep();
        widen(r, dz);
        token(t, cur, dz);
        if (place < q.begin) emit_state(place, acc[0]);
        else
          Raw<T, V>::store(when(place >= t0 && place < t1, du, kBatch * step), at,
                           static_cast<int>(t - tb) * step, acc[0]);
        move_on(cur);
      }
    };
    for (int64_t tb = t0; tb < stop;) {
      load(1, tb + kBatch);
      work(0, tb);
      tb += kBatch;
      if (tb >= stop) break;
      load(0, tb + kBatch);
      work(1, tb);
      tb += kBatch;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int i = 0; i < K; ++i) m[wave][i * V + v][p.lane] = dw[i][v];
    m[wave][K * V + v][p.lane] = db[v];
  }
  block_sync();
  if (!p.active) return;
  for (int e = wave; e < (K + 1) * V; e += kWaves) {
    float s = 0.0f;
    for (int k = 0; k < kWaves; ++k) s += m[k][e][p.lane];
    part[(brow * (K + 1) + e / V) * a.D + p.c + e % V] = s;
  }
}

// dweight [D, K] and dbias [D] = the sums over the rows of part, in a fixed order.
__global__ __launch_bounds__(1024) void conv_sum_kernel(const float* __restrict__ part, int64_t rows,
                                                        int64_t D, int K, float* dweight,
                                                        float* dbias) {
  __shared__ double m[16][64];
  const int col = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = int64_t(blockIdx.x) * 64 + col;
  const int i = blockIdx.y;
  double s = 0.0;
  if (c < D) {
#pragma unroll 8
    for (int64_t r = w; r < rows; r += 16) s += part[(r * (K + 1) + i) * D + c];
  }
  m[w][col] = s;
  block_sync();
  if (w != 0 || c >= D) return;
  for (int k = 1; k < 16; ++k) s += m[k][col];
  if (i < K) dweight[c * K + i] = static_cast<float>(s);
  else if (dbias) dbias[c] = static_cast<float>(s);
}

__global__ __launch_bounds__(256) void conv_zero_kernel(float* p, int64_t n) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// The gradient of the state of a sequence without tokens is its last state's.
template <typename T>
__global__ __launch_bounds__(256) void conv_empty_kernel(ConvArgs a, ConvGrads d, int64_t q0) {
  const int64_t q = q0 + blockIdx.x;
  if (seq_begin(a.seqs, q + 1) > seq_begin(a.seqs, q)) return;
  const int64_t n = (a.k - 1) * a.D;
  const T* from = static_cast<const T*>(d.dlast);
  for (int64_t e = threadIdx.x; e < n; e += 256)
    static_cast<T*>(d.dstate)[q * n + e] = from ? from[q * n + e] : T();
}

template <typename T, int K>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a, T* state) {
  const int64_t n = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t q = n / a.D, c = n - q * a.D;
  if (q >= a.seqs.n) return;
  T* s = state + q * (K - 1) * a.D + c;
  const T cur = static_cast<const T*>(a.u)[q * a.u_row + c];
  T win[K];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) win[i] = s[i * a.D];
  win[K - 1] = cur;
  float v = a.bias ? a.bias[c] : 0.0f;
#pragma unroll
  for (int i = 0; i < K; ++i) v = __builtin_fmaf(a.weight[c * K + i], to_float(win[i]), v);
#pragma unroll
  for (int i = 0; i < K - 1; ++i) s[i * a.D] = win[i + 1];
  const float out[1] = {a.silu ? silu(v) : v};
  Raw<T, 1>::store(static_cast<T*>(a.y) + q * a.D + c, out);
}

template <typename T, int kBytes>
constexpr int kVec = kBytes / static_cast<int>(sizeof(T));

// Calls f(type, channels a lane holds, taps).  kBytes: of a lane's load where the row is as long.
template <int kBytes, typename F>
hipError_t with_taps(mssm_dtype dtype, int64_t D, int64_t k, F f) {
  auto taps = [&](auto t, auto v) -> hipError_t {
    switch (k) {
      case 1: return f(t, v, std::integral_constant<int, 1>());
      case 2: return f(t, v, std::integral_constant<int, 2>());
      case 3: return f(t, v, std::integral_constant<int, 3>());
      case 4: return f(t, v, std::integral_constant<int, 4>());
      case 5: return f(t, v, std::integral_constant<int, 5>());
      case 6: return f(t, v, std::integral_constant<int, 6>());
      case 7: return f(t, v, std::integral_constant<int, 7>());
      case 8: return f(t, v, std::integral_constant<int, 8>());
      default: return hipErrorInvalidValue;
    }
  };
  if (dtype == MSSM_BFLOAT16) {
    constexpr int V = kVec<uint16_t, kBytes>;
    return D >= V ? taps(uint16_t(), std::integral_constant<int, V>())
                  : taps(uint16_t(), std::integral_constant<int, 1>());
  }
  constexpr int V = kVec<float, kBytes>;
  return D >= V ? taps(float(), std::integral_constant<int, V>())
                : taps(float(), std::integral_constant<int, 1>());
}

struct ConvGrid {
  int64_t groups, len, runs;
};
// Runs long enough that the rows read twice are few, but with 4096 wavefronts where there are so many.
ConvGrid conv_grid(int64_t tokens, int64_t D, int V, int64_t longest) {
  ConvGrid g;
  g.groups = (D + 64 * V - 1) / (64 * V);
  int64_t len = tokens / (kWavesWanted / (g.groups < kWavesWanted ? g.groups : kWavesWanted));
  len = (len + kBatch - 1) / kBatch * kBatch;
  g.len = len < kBatch ? kBatch : len > longest ? longest : len;
  g.runs = (tokens + g.len - 1) / g.len;
  return g;
}
int vec_of(mssm_dtype dtype, int64_t D, int bytes) {
  const int V = bytes / (dtype == MSSM_BFLOAT16 ? 2 : 4);
  return D >= V ? V : 1;
}
ConvGrid fwd_grid(int64_t tokens, int64_t D, mssm_dtype dtype) {
  return conv_grid(tokens, D, vec_of(dtype, D, kFwdBytes), kFwdRun);
}
ConvGrid bwd_grid(int64_t tokens, int64_t D, mssm_dtype dtype) {
  return conv_grid(tokens, D, vec_of(dtype, D, kBwdBytes), kBwdRun);
}

constexpr int64_t kMaxSequences = 1 << 22;      // of one launch

}  // namespace

int64_t conv_blocks(int64_t tokens, int64_t D, bool backward, mssm_dtype dtype) {
  if (tokens == 0 || D == 0) return 0;
  const ConvGrid g = backward ? bwd_grid(tokens, D, dtype) : fwd_grid(tokens, D, dtype);
  return backward ? g.groups * ((g.runs + kWaves - 1) / kWaves)
                  : (g.groups * g.runs + kWaves - 1) / kWaves;
}

size_t conv_bwd_workspace(int64_t tokens, int64_t D, int64_t k, mssm_dtype dtype) {
  if (tokens == 0 || D == 0) return 0;
  const ConvGrid g = bwd_grid(tokens, D, dtype);
  return static_cast<size_t>((g.runs + kWaves - 1) / kWaves) * (k + 1) * D * sizeof(float);
}

hipError_t launch_conv(const ConvArgs& a, hipStream_t stream) {
  int64_t main = 0, last = 0;
  ConvGrid g{1, kBatch, 0};
  if (a.seqs.tokens > 0) {
    g = fwd_grid(a.seqs.tokens, a.D, a.dtype);
    main = (g.groups * g.runs + kWaves - 1) / kWaves;
  }
  if (a.last && a.k > 1) {
    last = a.seqs.n * ((a.k * a.D + 2047) / 2048);
    if (last > 4096) last = 4096;
  }
  if (main + last == 0) return hipSuccess;
  return with_taps<kFwdBytes>(a.dtype, a.D, a.k, [&](auto t, auto v, auto k) {
    hipLaunchKernelGGL((conv_kernel<decltype(t), decltype(v)::value, decltype(k)::value>),
                       dim3(static_cast<uint32_t>(main + last)), dim3(kBlock), 0, stream, a,
                       g.groups, g.len, main);
    return hipGetLastError();
  });
}

hipError_t launch_conv_bwd(const ConvArgs& a, const ConvGrads& d, void* ws, hipStream_t stream) {
  if (d.dstate && a.k > 1 && (a.seqs.offsets || a.seqs.L == 0)) {
    for (int64_t q = 0; q < a.seqs.n; q += kMaxSequences) {
      const dim3 grid(static_cast<uint32_t>(a.seqs.n - q < kMaxSequences ? a.seqs.n - q
                                                                         : kMaxSequences));
      if (a.dtype == MSSM_BFLOAT16)
        hipLaunchKernelGGL(conv_empty_kernel<uint16_t>, grid, dim3(256), 0, stream, a, d, q);
      else
        hipLaunchKernelGGL(conv_empty_kernel<float>, grid, dim3(256), 0, stream, a, d, q);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  if (a.seqs.tokens == 0) {
    auto zero = [&](float* p, int64_t n) {
      hipLaunchKernelGGL(conv_zero_kernel, dim3(static_cast<uint32_t>((n + 255) / 256)), dim3(256),
                         0, stream, p, n);
      return hipGetLastError();
    };
    const hipError_t e = zero(d.dweight, a.D * a.k);
    return e != hipSuccess || !d.dbias ? e : zero(d.dbias, a.D);
  }
  const ConvGrid g = bwd_grid(a.seqs.tokens, a.D, a.dtype);
  const int64_t rows = (g.runs + kWaves - 1) / kWaves;
  float* part = static_cast<float*>(ws);
  const hipError_t e = with_taps<kBwdBytes>(a.dtype, a.D, a.k, [&](auto t, auto v, auto k) {
    hipLaunchKernelGGL((conv_bwd_kernel<decltype(t), decltype(v)::value, decltype(k)::value>),
                       dim3(static_cast<uint32_t>(g.groups * rows)), dim3(kBlock), 0, stream, a, d,
                       g.groups, g.len, part);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(conv_sum_kernel,
                     dim3(static_cast<uint32_t>((a.D + 63) / 64), static_cast<uint32_t>(a.k + 1)),
                     dim3(1024), 0, stream, part, rows, a.D, static_cast<int>(a.k), d.dweight,
                     d.dbias);
  return hipGetLastError();
}

hipError_t launch_conv_step(const ConvArgs& a, void* state, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>((a.seqs.n * a.D + 255) / 256));
  // one channel a lane: the calls are small
  return with_taps<0>(a.dtype, a.D, a.k, [&](auto t, auto, auto k) {
    using T = decltype(t);
    hipLaunchKernelGGL((conv_step_kernel<T, decltype(k)::value>), grid, dim3(256), 0, stream, a,
                       static_cast<T*>(state));
    return hipGetLastError();
  });
}

}  // namespace mssm
