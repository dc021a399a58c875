// C-ABI front end of the gated linear recurrence, the causal convolution with states and the
// residual norm: argument checks, which all run before the first HIP call, and dispatch.
#include "api_checks.h"

namespace {

using mssm::bad_dtype;
using mssm::check_workspace;
using mssm::done;
using mssm::product;
using mssm::same_address;

// A row of values, or from one token's to the next one's: sixteen of them are reached in 31 bits.
constexpr int64_t kMaxRow = int64_t(1) << 24;
constexpr int64_t kMaxSeqs = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxThreads = int64_t(1) << 32;       // of a launch, in one dimension

mssm_status sequences_of(const int64_t* offsets, bool packed, int64_t seqs, int64_t L, int64_t D,
                         mssm_dtype dtype, mssm::Sequences* s) {
  if (seqs < 0 || L < 0 || D < 0 || bad_dtype(dtype)) return MSSM_ERROR_INVALID_VALUE;
  int64_t tokens = L, n;
  if (!packed && !product({seqs, L}, &tokens)) return MSSM_ERROR_SIZE_OVERFLOW;
  if (!product({tokens, D, 64}, &n) || !product({seqs, D, 64}, &n)) return MSSM_ERROR_SIZE_OVERFLOW;
  if (D >= kMaxRow || seqs > kMaxSeqs) return MSSM_ERROR_NOT_SUPPORTED;
  s->offsets = offsets;
  s->n = seqs;
  s->L = packed ? 0 : L;
  s->tokens = seqs == 0 ? 0 : tokens;
  return MSSM_SUCCESS;
}

// Token rows hold their channels.  (A single token's are reached in 64 bits, whatever lies
// between them.)
mssm_status check_rows(const mssm::Sequences& s, int64_t D, std::initializer_list<int64_t> rows,
                       bool single = false) {
  for (int64_t row : rows) {
    int64_t n;
    if (row < D) return MSSM_ERROR_INVALID_VALUE;
    if (!single && row >= kMaxRow) return MSSM_ERROR_NOT_SUPPORTED;
    if (!product({s.tokens, row, 8}, &n)) return MSSM_ERROR_SIZE_OVERFLOW;
  }
  return MSSM_SUCCESS;
}

mssm_status recurrence_plan(const mssm::Sequences& s, int64_t D, bool backward, bool saved,
                            mssm_dtype dtype, mssm::RecurrencePlan* p) {
  *p = mssm::plan_recurrence(s.tokens, D, backward, saved, dtype);
  int64_t n;
  if (!product({p->bwd_tiles, p->bwd_groups, 512}, &n)) return MSSM_ERROR_SIZE_OVERFLOW;
  return n < kMaxThreads ? MSSM_SUCCESS : MSSM_ERROR_NOT_SUPPORTED;
}

// Whether a dense output lies over an input whose rows lie otherwise, so that a row is written while
// another one is still to be read there.
bool overwritten(const void* out, int64_t D, const void* x, int64_t x_row, const void* i,
                 int64_t i_row, const void* r, int64_t r_row) {
  return (out == x && x_row != D) || (out == i && i_row != D) || (out == r && r_row != D);
}

mssm_status check_saved(const void* saved, size_t have, size_t need) {
  return check_workspace(saved, have, need);
}

}  // namespace

extern "C" {

mssm_status mssm_gated_recurrence_saved_size(int64_t seqs, int64_t L, int64_t D, int packed,
                                             mssm_dtype dtype, size_t* bytes) {
  if (!bytes) return MSSM_ERROR_INVALID_VALUE;
  mssm::Sequences s;
  mssm::RecurrencePlan p;
  mssm_status st = sequences_of(nullptr, packed != 0, seqs, L, D, dtype, &s);
  if (st != MSSM_SUCCESS) return st;
  if ((st = recurrence_plan(s, D, false, true, dtype, &p)) != MSSM_SUCCESS) return st;
  *bytes = p.saved_bytes;
  return MSSM_SUCCESS;
}

mssm_status mssm_gated_recurrence_workspace_size(int64_t seqs, int64_t L, int64_t D, int packed,
                                                 int backward, int saved, mssm_dtype dtype,
                                                 size_t* bytes) {
  if (!bytes) return MSSM_ERROR_INVALID_VALUE;
  mssm::Sequences s;
  mssm::RecurrencePlan p;
  mssm_status st = sequences_of(nullptr, packed != 0, seqs, L, D, dtype, &s);
  if (st != MSSM_SUCCESS) return st;
  if ((st = recurrence_plan(s, D, backward != 0, saved != 0, dtype, &p)) != MSSM_SUCCESS) return st;
  *bytes = D == 0 ? 0 : p.bytes;
  return MSSM_SUCCESS;
}

mssm_status mssm_gated_recurrence_fwd(const void* x, const void* input_gate,
                                      const void* decay_gate, const float* A,
                                      const int64_t* seq_offsets, const float* state, void* h,
                                      float* last_state, float* saved, size_t saved_bytes,
                                      void* workspace, size_t workspace_bytes, int64_t seqs,
                                      int64_t L, int64_t D, int64_t x_row, int64_t i_row,
                                      int64_t r_row, mssm_dtype dtype, void* stream) {
  mssm::RecurrenceArgs a;
  mssm::RecurrencePlan p;
  mssm_status st = sequences_of(seq_offsets, seq_offsets != nullptr, seqs, L, D, dtype, &a.seqs);
  if (st != MSSM_SUCCESS) return st;
  if (seqs == 0 || D == 0) return MSSM_SUCCESS;
  if (last_state && last_state == state) return MSSM_ERROR_INVALID_VALUE;
  if (a.seqs.tokens > 0) {
    if (!x || !input_gate || !decay_gate || !A || !h) return MSSM_ERROR_INVALID_VALUE;
    if ((st = check_rows(a.seqs, D, {x_row, i_row, r_row})) != MSSM_SUCCESS) return st;
  } else if (!last_state) {
    return MSSM_SUCCESS;
  }
  if ((st = recurrence_plan(a.seqs, D, false, saved != nullptr, dtype, &p)) != MSSM_SUCCESS)
    return st;
  if (saved && (st = check_saved(saved, saved_bytes, p.saved_bytes)) != MSSM_SUCCESS) return st;
  if ((st = check_workspace(workspace, workspace_bytes, p.bytes)) != MSSM_SUCCESS) return st;
  if (a.seqs.tokens > 0 &&
      same_address({h, last_state, saved}, {x, input_gate, decay_gate, A, state}))
    return MSSM_ERROR_INVALID_VALUE;
  a.D = D;
  a.x = x, a.i = input_gate, a.r = decay_gate, a.A = A;
  a.x_row = x_row, a.i_row = i_row, a.r_row = r_row;
  a.state = state, a.h = h, a.last = last_state, a.saved = saved;
  a.dtype = dtype;
  return done(mssm::launch_recurrence(a, p, workspace, static_cast<hipStream_t>(stream)),
              "gated recurrence launch");
}

mssm_status mssm_gated_recurrence_step(const void* x, const void* input_gate,
                                       const void* decay_gate, const float* A, float* state,
                                       void* h, int64_t seqs, int64_t D, int64_t x_row,
                                       int64_t i_row, int64_t r_row, mssm_dtype dtype,
                                       void* stream) {
  mssm::RecurrenceArgs a;
  mssm_status st = sequences_of(nullptr, false, seqs, 1, D, dtype, &a.seqs);
  if (st != MSSM_SUCCESS) return st;
  if (seqs == 0 || D == 0) return MSSM_SUCCESS;
  if (!x || !input_gate || !decay_gate || !A || !state || !h) return MSSM_ERROR_INVALID_VALUE;
  if ((st = check_rows(a.seqs, D, {x_row, i_row, r_row}, true)) != MSSM_SUCCESS) return st;
  int64_t n;
  if (!product({seqs, D}, &n)) return MSSM_ERROR_SIZE_OVERFLOW;
  if (n >= kMaxThreads - 256) return MSSM_ERROR_NOT_SUPPORTED;
  if (same_address({h, state}, {A}) || same_address({state}, {x, input_gate, decay_gate}) ||
      overwritten(h, D, x, x_row, input_gate, i_row, decay_gate, r_row))
    return MSSM_ERROR_INVALID_VALUE;
  a.D = D;
  a.x = x, a.i = input_gate, a.r = decay_gate, a.A = A;
  a.x_row = x_row, a.i_row = i_row, a.r_row = r_row;
  a.h = h, a.dtype = dtype;
  return done(mssm::launch_recurrence_step(a, state, static_cast<hipStream_t>(stream)),
              "gated recurrence step launch");
}

mssm_status mssm_gated_recurrence_bwd(const void* x, const void* input_gate,
                                      const void* decay_gate, const float* A,
                                      const int64_t* seq_offsets, const float* state,
                                      const float* saved, size_t saved_bytes, const void* dh,
                                      const float* dlast, void* dx, void* dinput_gate,
                                      void* ddecay_gate, float* dA, float* dstate,
                                      void* workspace, size_t workspace_bytes, int64_t seqs,
                                      int64_t L, int64_t D, int64_t x_row, int64_t i_row,
                                      int64_t r_row, mssm_dtype dtype, void* stream) {
  mssm::RecurrenceArgs a;
  mssm::RecurrencePlan p;
  mssm_status st = sequences_of(seq_offsets, seq_offsets != nullptr, seqs, L, D, dtype, &a.seqs);
  if (st != MSSM_SUCCESS) return st;
  if (D == 0) return MSSM_SUCCESS;
  if (!dA) return MSSM_ERROR_INVALID_VALUE;
  if (dstate && (dstate == state || dstate == dlast)) return MSSM_ERROR_INVALID_VALUE;
  if (a.seqs.tokens > 0) {
    if (!x || !input_gate || !decay_gate || !A || !dh || !dx || !dinput_gate || !ddecay_gate)
      return MSSM_ERROR_INVALID_VALUE;
    if ((st = check_rows(a.seqs, D, {x_row, i_row, r_row})) != MSSM_SUCCESS) return st;
  }
  if ((st = recurrence_plan(a.seqs, D, true, saved != nullptr, dtype, &p)) != MSSM_SUCCESS)
    return st;
  if (saved && (st = check_saved(saved, saved_bytes, p.saved_bytes)) != MSSM_SUCCESS) return st;
  if ((st = check_workspace(workspace, workspace_bytes, p.bytes)) != MSSM_SUCCESS) return st;
  if (a.seqs.tokens > 0) {
    if (same_address({dx, dinput_gate, ddecay_gate, dA, dstate}, {A, state, saved, dlast}))
      return MSSM_ERROR_INVALID_VALUE;
    for (const void* out : {dx, dinput_gate, ddecay_gate})
      if (overwritten(out, D, x, x_row, input_gate, i_row, decay_gate, r_row))
        return MSSM_ERROR_INVALID_VALUE;
  }
  a.D = D;
  a.x = x, a.i = input_gate, a.r = decay_gate, a.A = A;
  a.x_row = x_row, a.i_row = i_row, a.r_row = r_row;
  a.state = state;
  a.saved = const_cast<float*>(saved);    // read only
  a.dtype = dtype;
  mssm::RecurrenceGrads d;
  d.dh = dh, d.dlast = dlast;
  d.dx = dx, d.di = dinput_gate, d.dr = ddecay_gate, d.dA = dA, d.dstate = dstate;
  return done(mssm::launch_recurrence_bwd(a, d, p, workspace, static_cast<hipStream_t>(stream)),
              "gated recurrence backward launch");
}

}  // extern "C"

namespace {

mssm_status check_conv(mssm_activation act, int64_t k) {
  if (act != MSSM_ACT_NONE && act != MSSM_ACT_SILU) return MSSM_ERROR_INVALID_VALUE;
  if (k < 1) return MSSM_ERROR_INVALID_VALUE;
  return k <= 8 ? MSSM_SUCCESS : MSSM_ERROR_NOT_SUPPORTED;
}

mssm_status conv_sizes(const mssm::Sequences& s, int64_t D, bool backward, mssm_dtype dtype) {
  int64_t n;
  if (!product({mssm::conv_blocks(s.tokens, D, backward, dtype), 256}, &n))
    return MSSM_ERROR_SIZE_OVERFLOW;
  return n < kMaxThreads ? MSSM_SUCCESS : MSSM_ERROR_NOT_SUPPORTED;
}

}  // namespace

extern "C" {

mssm_status mssm_causal_conv1d_fwd(const void* u, const float* weight, const float* bias,
                                   const int64_t* seq_offsets, const void* state, void* y,
                                   void* last_state, mssm_activation act, int64_t seqs, int64_t L,
                                   int64_t D, int64_t k, int64_t u_row, mssm_dtype dtype,
                                   void* stream) {
  mssm::ConvArgs a;
  mssm_status st = sequences_of(seq_offsets, seq_offsets != nullptr, seqs, L, D, dtype, &a.seqs);
  if (st != MSSM_SUCCESS) return st;
  if ((st = check_conv(act, k)) != MSSM_SUCCESS) return st;
  if (seqs == 0 || D == 0) return MSSM_SUCCESS;
  if (last_state && last_state == state) return MSSM_ERROR_INVALID_VALUE;
  if (a.seqs.tokens > 0) {
    if (!u || !weight || !y) return MSSM_ERROR_INVALID_VALUE;
    if ((st = check_rows(a.seqs, D, {u_row})) != MSSM_SUCCESS) return st;
  } else if (!last_state) {
    return MSSM_SUCCESS;
  }
  if ((st = conv_sizes(a.seqs, D, false, dtype)) != MSSM_SUCCESS) return st;
  if (same_address({a.seqs.tokens > 0 ? y : nullptr, k > 1 ? last_state : nullptr},
                   {u, weight, bias, state}))
    return MSSM_ERROR_INVALID_VALUE;
  a.D = D, a.k = k;
  a.u = u, a.u_row = u_row, a.weight = weight, a.bias = bias;
  a.silu = act == MSSM_ACT_SILU;
  a.state = state, a.y = y, a.last = last_state;
  a.dtype = dtype;
  return done(mssm::launch_conv(a, static_cast<hipStream_t>(stream)), "causal convolution launch");
}

mssm_status mssm_causal_conv1d_step(const void* u, const float* weight, const float* bias,
                                    void* state, void* y, mssm_activation act, int64_t seqs,
                                    int64_t D, int64_t k, int64_t u_row, mssm_dtype dtype,
                                    void* stream) {
  mssm::ConvArgs a;
  mssm_status st = sequences_of(nullptr, false, seqs, 1, D, dtype, &a.seqs);
  if (st != MSSM_SUCCESS) return st;
  if ((st = check_conv(act, k)) != MSSM_SUCCESS) return st;
  if (seqs == 0 || D == 0) return MSSM_SUCCESS;
  if (!u || !weight || !y || (k > 1 && !state)) return MSSM_ERROR_INVALID_VALUE;
  if ((st = check_rows(a.seqs, D, {u_row}, true)) != MSSM_SUCCESS) return st;
  int64_t n;
  if (!product({seqs, D}, &n)) return MSSM_ERROR_SIZE_OVERFLOW;
  if (n >= kMaxThreads - 256) return MSSM_ERROR_NOT_SUPPORTED;
  const void* kept = k > 1 ? state : nullptr;
  // (a thread reads its own value of a dense u before it writes that of y)
  if (same_address({y, kept}, {weight, bias}) || (kept && kept == u) || (y == u && u_row != D))
    return MSSM_ERROR_INVALID_VALUE;
  a.D = D, a.k = k;
  a.u = u, a.u_row = u_row, a.weight = weight, a.bias = bias;
  a.silu = act == MSSM_ACT_SILU;
  a.y = y, a.dtype = dtype;
  return done(mssm::launch_conv_step(a, state, static_cast<hipStream_t>(stream)),
              "causal convolution step launch");
}

mssm_status mssm_causal_conv1d_bwd_workspace_size(int64_t seqs, int64_t L, int64_t D, int64_t k,
                                                  int packed, mssm_dtype dtype, size_t* bytes) {
  if (!bytes) return MSSM_ERROR_INVALID_VALUE;
  mssm::Sequences s;
  mssm_status st = sequences_of(nullptr, packed != 0, seqs, L, D, dtype, &s);
  if (st != MSSM_SUCCESS) return st;
  if ((st = check_conv(MSSM_ACT_NONE, k)) != MSSM_SUCCESS) return st;
  if ((st = conv_sizes(s, D, true, dtype)) != MSSM_SUCCESS) return st;
  *bytes = mssm::conv_bwd_workspace(s.tokens, D, k, dtype);
  return MSSM_SUCCESS;
}

mssm_status mssm_causal_conv1d_bwd(const void* u, const float* weight, const float* bias,
                                   const int64_t* seq_offsets, const void* state, const void* dy,
                                   const void* dlast, void* du, float* dweight, float* dbias,
                                   void* dstate, mssm_activation act, void* workspace,
                                   size_t workspace_bytes, int64_t seqs, int64_t L, int64_t D,
                                   int64_t k, int64_t u_row, mssm_dtype dtype, void* stream) {
  mssm::ConvArgs a;
  mssm_status st = sequences_of(seq_offsets, seq_offsets != nullptr, seqs, L, D, dtype, &a.seqs);
  if (st != MSSM_SUCCESS) return st;
  if ((st = check_conv(act, k)) != MSSM_SUCCESS) return st;
  if (D == 0) return MSSM_SUCCESS;
  if (!dweight) return MSSM_ERROR_INVALID_VALUE;
  if (dstate && (dstate == state || dstate == dlast)) return MSSM_ERROR_INVALID_VALUE;
  if (a.seqs.tokens > 0) {
    if (!u || !weight || !dy || !du) return MSSM_ERROR_INVALID_VALUE;
    if ((st = check_rows(a.seqs, D, {u_row})) != MSSM_SUCCESS) return st;
  }
  if ((st = conv_sizes(a.seqs, D, true, dtype)) != MSSM_SUCCESS) return st;
  st = check_workspace(workspace, workspace_bytes,
                       mssm::conv_bwd_workspace(a.seqs.tokens, D, k, dtype));
  if (st != MSSM_SUCCESS) return st;
  if (same_address({a.seqs.tokens > 0 ? du : nullptr, dweight, dbias,
                    k > 1 && seqs > 0 ? dstate : nullptr},
                   {u, weight, bias, state, dy, dlast}))
    return MSSM_ERROR_INVALID_VALUE;
  a.D = D, a.k = k;
  a.u = u, a.u_row = u_row, a.weight = weight, a.bias = bias;
  a.silu = act == MSSM_ACT_SILU;
  a.state = state, a.dtype = dtype;
  mssm::ConvGrads d;
  d.dy = dy, d.dlast = dlast, d.du = du, d.dweight = dweight, d.dbias = dbias, d.dstate = dstate;
  return done(mssm::launch_conv_bwd(a, d, workspace, static_cast<hipStream_t>(stream)),
              "causal convolution backward launch");
}

}  // extern "C"

namespace {

mssm_status check_residual_norm(int64_t rows, int64_t D, int64_t gate_rows, mssm_activation form,
                                mssm_dtype dtype) {
  if (rows < 0 || D < 0 || bad_dtype(dtype)) return MSSM_ERROR_INVALID_VALUE;
  if (form != MSSM_ACT_NONE && form != MSSM_ACT_SILU) return MSSM_ERROR_INVALID_VALUE;
  if (gate_rows < 1 || rows % gate_rows != 0) return MSSM_ERROR_INVALID_VALUE;
  if (!mssm::norm_size_supported(D)) return MSSM_ERROR_NOT_SUPPORTED;
  int64_t n;
  if (!product({rows, D, 8}, &n)) return MSSM_ERROR_SIZE_OVERFLOW;
  if (rows >> 32 != 0) return MSSM_ERROR_NOT_SUPPORTED;
  return MSSM_SUCCESS;
}

}  // namespace

extern "C" {

mssm_status mssm_residual_norm_fwd(const void* y, const void* residual, const float* weight,
                                   const float* post_weight, const void* gate, const float* scale,
                                   void* out, void* total, float* rstd, float* post_rstd,
                                   mssm_activation gate_form, int64_t gate_rows, float eps,
                                   int64_t rows, int64_t D, mssm_dtype dtype, void* stream) {
  const mssm_status st = check_residual_norm(rows, D, gate_rows, gate_form, dtype);
  if (st != MSSM_SUCCESS) return st;
  if (!(eps >= 0.0f)) return MSSM_ERROR_INVALID_VALUE;
  if (rows == 0 || D == 0) return MSSM_SUCCESS;
  if (!y || !residual || !weight || !out || !total) return MSSM_ERROR_INVALID_VALUE;
  if (post_rstd && (!rstd || !post_weight)) return MSSM_ERROR_INVALID_VALUE;
  if (same_address({out, total, rstd, post_rstd}, {y, residual, weight, post_weight, gate, scale}))
    return MSSM_ERROR_INVALID_VALUE;
  mssm::ResidualNormArgs a;
  a.y = y, a.residual = residual, a.weight = weight, a.post_weight = post_weight;
  a.gate = gate, a.gate_rows = gate ? gate_rows : 1, a.silu = gate_form == MSSM_ACT_SILU;
  a.scale = scale, a.out = out, a.total = total, a.rstd = rstd, a.post_rstd = post_rstd;
  a.eps = eps, a.rows = rows, a.D = D, a.dtype = dtype;
  return done(mssm::launch_residual_norm(a, static_cast<hipStream_t>(stream)),
              "residual norm launch");
}

mssm_status mssm_residual_norm_bwd_workspace_size(int64_t rows, int64_t D, int64_t gate_rows,
                                                  mssm_dtype dtype, size_t* bytes) {
  if (!bytes) return MSSM_ERROR_INVALID_VALUE;
  const mssm_status st = check_residual_norm(rows, D, gate_rows, MSSM_ACT_NONE, dtype);
  if (st != MSSM_SUCCESS) return st;
  *bytes = mssm::residual_norm_bwd_workspace(rows, D, gate_rows, dtype);
  return MSSM_SUCCESS;
}

mssm_status mssm_residual_norm_bwd(const void* dout, const void* dtotal, const void* y,
                                   const void* total, const float* weight,
                                   const float* post_weight, const void* gate, const float* scale,
                                   const float* rstd, const float* post_rstd, void* dy,
                                   void* dresidual, void* dgate, float* dweight,
                                   float* dpost_weight, float* dscale, mssm_activation gate_form,
                                   int64_t gate_rows, void* workspace, size_t workspace_bytes,
                                   int64_t rows, int64_t D, mssm_dtype dtype, void* stream) {
  mssm_status st = check_residual_norm(rows, D, gate_rows, gate_form, dtype);
  if (st != MSSM_SUCCESS) return st;
  if (D == 0) return MSSM_SUCCESS;
  if (!gate) gate_rows = 1;
  if (!dweight || !post_weight != !dpost_weight || !scale != !dscale)
    return MSSM_ERROR_INVALID_VALUE;
  if (rows > 0) {
    if (!dout || !y || !total || !weight || !rstd || !dy || !dresidual ||
        !post_weight != !post_rstd || !gate != !dgate)
      return MSSM_ERROR_INVALID_VALUE;
    st = check_workspace(workspace, workspace_bytes,
                         mssm::residual_norm_bwd_workspace(rows, D, gate_rows, dtype));
    if (st != MSSM_SUCCESS) return st;
    if (same_address({dy, dresidual, dgate, dweight, dpost_weight, dscale},
                     {dout, dtotal, y, total, weight, post_weight, gate, scale, rstd, post_rstd}))
      return MSSM_ERROR_INVALID_VALUE;
  }
  mssm::ResidualNormArgs a;
  a.y = y, a.weight = weight, a.post_weight = post_weight;
  a.gate = gate, a.gate_rows = gate_rows, a.silu = gate_form == MSSM_ACT_SILU;
  a.scale = scale, a.total = const_cast<void*>(total);
  a.rstd = const_cast<float*>(rstd), a.post_rstd = const_cast<float*>(post_rstd);
  a.rows = rows, a.D = D, a.dtype = dtype;
  mssm::ResidualNormGrads d;
  d.dout = dout, d.dtotal = dtotal, d.dy = dy, d.dresidual = dresidual, d.dgate = dgate;
  d.dweight = dweight, d.dpost_weight = dpost_weight, d.dscale = dscale;
  return done(mssm::launch_residual_norm_bwd(a, d, workspace, static_cast<hipStream_t>(stream)),
              "residual norm backward launch");
}

}  // extern "C"
