// C-ABI front end of linear attention and layer norm: argument checks, which
// all run before the first HIP call, and dispatch.
#include <initializer_list>
#include <limits>

#include "mssm_internal.h"

namespace {

// A token's values in any tensor: its bytes fit 24 bits, a chunk's 32, which is
// how the kernels reach them.
constexpr int64_t kMaxRow = int64_t(1) << 22;
constexpr int64_t kMaxBlocks = (int64_t(1) << 32) / 256 - 1;   // blocks of 256 threads

bool product(std::initializer_list<int64_t> f, int64_t* out) {
  int64_t n = 1;
  for (int64_t v : f) {
    if (v == 0) { *out = 0; return true; }
  }
  for (int64_t v : f) {
    if (n > std::numeric_limits<int64_t>::max() / v) return false;
    n *= v;
  }
  *out = n;
  return true;
}

bool bad_dtype(mssm_dtype t) { return t != MSSM_FLOAT32 && t != MSSM_BFLOAT16; }

mssm_status shape_of(int64_t seqs, int64_t L, int64_t key_heads, int64_t heads, int64_t dk,
                     int64_t dv, bool packed, mssm_dtype dtype, mssm::LaShape* s) {
  if (seqs < 0 || L < 0 || key_heads < 0 || heads < 0 || dk < 0 || dv < 0 || bad_dtype(dtype))
    return MSSM_ERROR_INVALID_VALUE;
  if (heads > 0 && (key_heads == 0 || heads % key_heads != 0)) return MSSM_ERROR_INVALID_VALUE;
  if (!mssm_linear_attention_supports(dk, dv)) return MSSM_ERROR_NOT_SUPPORTED;
  int64_t tokens = L, n;
  if (!packed && !product({seqs, L}, &tokens)) return MSSM_ERROR_SIZE_OVERFLOW;
  if (heads >= kMaxRow) return MSSM_ERROR_NOT_SUPPORTED;
  if (!product({tokens, heads, dk, 8}, &n) || !product({tokens, heads, dv, 8}, &n) ||
      !product({seqs, heads, dk, dv, 8}, &n))
    return MSSM_ERROR_SIZE_OVERFLOW;
  if (heads * dk >= kMaxRow || heads * dv >= kMaxRow) return MSSM_ERROR_NOT_SUPPORTED;
  s->seqs = seqs;
  s->tokens = tokens;
  s->packed = packed;
  s->key_heads = key_heads;
  s->heads = heads;
  s->dk = dk;
  s->dv = dv;
  return MSSM_SUCCESS;
}

// A plan whose workspace and grids fit their types.
mssm_status plan_of(const mssm::LaShape& s, bool backward, mssm_dtype dtype,
                    mssm::LaPlan* plan) {
  *plan = mssm::plan_la(s, backward, dtype == MSSM_BFLOAT16);
  if (plan->overflow) return MSSM_ERROR_SIZE_OVERFLOW;
  int64_t n;
  if (!product({plan->grid.slots, s.heads}, &n) || n > kMaxBlocks / (backward ? 2 : 1))
    return MSSM_ERROR_NOT_SUPPORTED;
  if (backward && s.heads != s.key_heads &&
      (!product({s.tokens, s.key_heads, s.dk}, &n) || n / 1024 > kMaxBlocks - 1))
    return MSSM_ERROR_NOT_SUPPORTED;
  return MSSM_SUCCESS;
}

// Rows hold their heads.  (A single token's are reached in 64 bits, whatever lies
// between them.)
mssm_status check_rows(const mssm::LaArgs& a, bool single) {
  const mssm::LaShape& s = a.shape;
  if (a.q_row < s.key_heads * s.dk || a.k_row < s.key_heads * s.dk || a.v_row < s.heads * s.dv)
    return MSSM_ERROR_INVALID_VALUE;
  for (int64_t row : {a.q_row, a.k_row, a.v_row}) {
    int64_t n;
    if (!single && row >= kMaxRow) return MSSM_ERROR_NOT_SUPPORTED;
    if (!product({s.tokens, row, 8}, &n)) return MSSM_ERROR_SIZE_OVERFLOW;
  }
  return MSSM_SUCCESS;
}

mssm_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MSSM_SUCCESS;
  if (!ws || have < need || reinterpret_cast<uintptr_t>(ws) % 256 != 0) return MSSM_ERROR_WORKSPACE;
  return MSSM_SUCCESS;
}

mssm_status done(hipError_t e, const char* where) {
  if (e == hipSuccess) return MSSM_SUCCESS;
  mssm::set_hip_error(e, where);
  return MSSM_ERROR_HIP;
}

}  // namespace

extern "C" {

int mssm_linear_attention_supports(int64_t dk, int64_t dv) {
  return dk >= 16 && dk <= 128 && dk % 16 == 0 && dv >= 16 && dv <= 128 && dv % 16 == 0 ? 1 : 0;
}

mssm_status mssm_linear_attention_workspace_size(int64_t seqs, int64_t L, int64_t key_heads,
                                                 int64_t heads, int64_t dk, int64_t dv, int packed,
                                                 int backward, mssm_dtype dtype, size_t* bytes) {
  if (!bytes) return MSSM_ERROR_INVALID_VALUE;
  mssm::LaShape s;
  mssm::LaPlan plan;
  mssm_status st = shape_of(seqs, L, key_heads, heads, dk, dv, packed != 0, dtype, &s);
  if (st != MSSM_SUCCESS) return st;
  *bytes = 0;
  if (seqs == 0 || heads == 0) return MSSM_SUCCESS;
  st = plan_of(s, backward != 0, dtype, &plan);
  if (st == MSSM_SUCCESS) *bytes = plan.bytes;
  return st;
}

mssm_status mssm_linear_attention_fwd(const void* q, const void* k, const void* v,
                                      const float* log_decay, const int64_t* seq_offsets,
                                      const float* state, void* o, float* last_state, float scale,
                                      mssm_decay decay, void* workspace, size_t workspace_bytes,
                                      int64_t seqs, int64_t L, int64_t key_heads, int64_t heads,
                                      int64_t dk, int64_t dv, int64_t q_row, int64_t k_row,
                                      int64_t v_row, mssm_dtype dtype, void* stream) {
  mssm::LaArgs a;
  mssm::LaPlan plan;
  mssm_status st = shape_of(seqs, L, key_heads, heads, dk, dv, seq_offsets != nullptr, dtype,
                            &a.shape);
  if (st != MSSM_SUCCESS) return st;
  if (decay != MSSM_DECAY_PER_HEAD && decay != MSSM_DECAY_PER_TOKEN)
    return MSSM_ERROR_INVALID_VALUE;
  if (seqs == 0 || heads == 0) return MSSM_SUCCESS;
  a.q_row = q_row, a.k_row = k_row, a.v_row = v_row;
  if (a.shape.tokens > 0) {
    if (!q || !k || !v || !log_decay || !o) return MSSM_ERROR_INVALID_VALUE;
    if ((st = check_rows(a, false)) != MSSM_SUCCESS) return st;
  } else if (!last_state) {
    return MSSM_SUCCESS;
  }
  if ((st = plan_of(a.shape, false, dtype, &plan)) != MSSM_SUCCESS) return st;
  if ((st = check_workspace(workspace, workspace_bytes, plan.bytes)) != MSSM_SUCCESS) return st;
  a.q = q, a.k = k, a.v = v, a.g = log_decay;
  a.per_token = decay == MSSM_DECAY_PER_TOKEN;
  a.offsets = seq_offsets;
  a.state = state, a.last = last_state, a.o = o;
  a.scale = scale, a.dtype = dtype;
  return done(mssm::launch_la_fwd(a, plan, workspace, static_cast<hipStream_t>(stream)),
              "linear attention launch");
}

mssm_status mssm_linear_attention_step(const void* q, const void* k, const void* v,
                                       const float* log_decay, float* state, void* o, float scale,
                                       mssm_decay decay, int64_t seqs, int64_t key_heads,
                                       int64_t heads, int64_t dk, int64_t dv, int64_t q_row,
                                       int64_t k_row, int64_t v_row, mssm_dtype dtype,
                                       void* stream) {
  mssm::LaArgs a;
  mssm_status st = shape_of(seqs, 1, key_heads, heads, dk, dv, false, dtype, &a.shape);
  if (st != MSSM_SUCCESS) return st;
  if (decay != MSSM_DECAY_PER_HEAD && decay != MSSM_DECAY_PER_TOKEN)
    return MSSM_ERROR_INVALID_VALUE;
  if (seqs == 0 || heads == 0) return MSSM_SUCCESS;
  if (!q || !k || !v || !log_decay || !state || !o) return MSSM_ERROR_INVALID_VALUE;
  a.q_row = q_row, a.k_row = k_row, a.v_row = v_row;
  if ((st = check_rows(a, true)) != MSSM_SUCCESS) return st;
  int64_t blocks;
  if (!product({seqs, heads}, &blocks)) return MSSM_ERROR_SIZE_OVERFLOW;
  if (blocks > kMaxBlocks) return MSSM_ERROR_NOT_SUPPORTED;
  a.q = q, a.k = k, a.v = v, a.g = log_decay;
  a.per_token = decay == MSSM_DECAY_PER_TOKEN;
  a.o = o, a.scale = scale, a.dtype = dtype;
  return done(mssm::launch_la_step(a, state, static_cast<hipStream_t>(stream)),
              "linear attention step launch");
}

mssm_status mssm_linear_attention_bwd(const void* q, const void* k, const void* v,
                                      const float* log_decay, const int64_t* seq_offsets,
                                      const float* state, const void* dout, const float* dlast,
                                      void* dq, void* dk_out, void* dv_out, float* dlog_decay,
                                      float* dstate, float scale, mssm_decay decay,
                                      void* workspace, size_t workspace_bytes, int64_t seqs,
                                      int64_t L, int64_t key_heads, int64_t heads, int64_t dk,
                                      int64_t dv, int64_t q_row, int64_t k_row, int64_t v_row,
                                      mssm_dtype dtype, void* stream) {
  mssm::LaArgs a;
  mssm::LaPlan plan;
  mssm_status st = shape_of(seqs, L, key_heads, heads, dk, dv, seq_offsets != nullptr, dtype,
                            &a.shape);
  if (st != MSSM_SUCCESS) return st;
  if (decay != MSSM_DECAY_PER_HEAD && decay != MSSM_DECAY_PER_TOKEN)
    return MSSM_ERROR_INVALID_VALUE;
  if (heads == 0) {
    // no head reads the queries and keys there may be: their gradients are zero
    int64_t n;
    if (!product({a.shape.tokens, key_heads, dk, 8}, &n)) return MSSM_ERROR_SIZE_OVERFLOW;
    if (n == 0) return MSSM_SUCCESS;
    if (!dq || !dk_out) return MSSM_ERROR_INVALID_VALUE;
    if (n / 8 / 1024 > kMaxBlocks - 1) return MSSM_ERROR_NOT_SUPPORTED;
    return done(mssm::launch_la_no_heads(a.shape, dq, dk_out, dtype, static_cast<hipStream_t>(stream)),
                "linear attention backward launch");
  }
  const bool per_token = decay == MSSM_DECAY_PER_TOKEN;
  a.q_row = q_row, a.k_row = k_row, a.v_row = v_row;
  if (a.shape.tokens > 0 && seqs > 0) {
    if (!q || !k || !v || !log_decay || !dout || !dq || !dk_out || !dv_out || !dlog_decay)
      return MSSM_ERROR_INVALID_VALUE;
    if ((st = check_rows(a, false)) != MSSM_SUCCESS) return st;
  } else {
    // nothing to differentiate but the decays (zero) and the states that pass through
    if (!per_token && !dlog_decay) return MSSM_ERROR_INVALID_VALUE;
    if (seqs == 0) {
      if (per_token) return MSSM_SUCCESS;
      return done(mssm::launch_state_init(dlog_decay, nullptr, heads,
                                          static_cast<hipStream_t>(stream)),
                  "linear attention backward launch");
    }
  }
  if ((st = plan_of(a.shape, true, dtype, &plan)) != MSSM_SUCCESS) return st;
  if ((st = check_workspace(workspace, workspace_bytes, plan.bytes)) != MSSM_SUCCESS) return st;
  a.q = q, a.k = k, a.v = v, a.g = log_decay;
  a.per_token = per_token;
  a.offsets = seq_offsets;
  a.state = state;
  a.scale = scale, a.dtype = dtype;
  mssm::LaGrads d;
  d.dout = dout, d.dlast = dlast;
  d.dq = dq, d.dk = dk_out, d.dv = dv_out, d.dg = dlog_decay, d.dstate = dstate;
  return done(mssm::launch_la_bwd(a, d, plan, workspace, static_cast<hipStream_t>(stream)),
              "linear attention backward launch");
}

}  // extern "C"

namespace {

mssm_status check_norm(int64_t rows, int64_t D, mssm_dtype dtype) {
  if (rows < 0 || D < 0 || bad_dtype(dtype)) return MSSM_ERROR_INVALID_VALUE;
  if (!mssm::norm_size_supported(D)) return MSSM_ERROR_NOT_SUPPORTED;
  int64_t n;
  if (!product({rows, D, 8}, &n)) return MSSM_ERROR_SIZE_OVERFLOW;
  if (rows >> 32 != 0) return MSSM_ERROR_NOT_SUPPORTED;
  return MSSM_SUCCESS;
}

}  // namespace

extern "C" {

mssm_status mssm_layer_norm_fwd(const void* x, const void* residual, const float* weight,
                                const float* bias, void* y, void* sum, float* mean, float* rstd,
                                float eps, int64_t rows, int64_t D, mssm_dtype dtype,
                                void* stream) {
  const mssm_status st = check_norm(rows, D, dtype);
  if (st != MSSM_SUCCESS) return st;
  if (!(eps >= 0.0f)) return MSSM_ERROR_INVALID_VALUE;
  if (rows == 0 || D == 0) return MSSM_SUCCESS;
  if (!x || !weight || !y || !residual != !sum || !mean != !rstd) return MSSM_ERROR_INVALID_VALUE;
  mssm::NormArgs a;
  a.x = x, a.residual = residual, a.weight = weight, a.bias = bias;
  a.y = y, a.sum = sum, a.mean = mean, a.rstd = rstd;
  a.eps = eps, a.rows = rows, a.D = D, a.dtype = dtype;
  return done(mssm::launch_norm(a, static_cast<hipStream_t>(stream)), "layer norm launch");
}

mssm_status mssm_layer_norm_bwd_workspace_size(int64_t rows, int64_t D, mssm_dtype dtype,
                                               size_t* bytes) {
  if (!bytes) return MSSM_ERROR_INVALID_VALUE;
  const mssm_status st = check_norm(rows, D, dtype);
  if (st != MSSM_SUCCESS) return st;
  *bytes = rows == 0 || D == 0 ? 0 : mssm::norm_bwd_workspace(rows, D, dtype);
  return MSSM_SUCCESS;
}

mssm_status mssm_layer_norm_bwd(const void* dy, const void* dsum, const void* x,
                                const float* weight, const float* mean, const float* rstd,
                                void* dx, float* dweight, float* dbias, void* workspace,
                                size_t workspace_bytes, int64_t rows, int64_t D,
                                mssm_dtype dtype, void* stream) {
  mssm_status st = check_norm(rows, D, dtype);
  if (st != MSSM_SUCCESS) return st;
  if (D == 0) return MSSM_SUCCESS;
  if (!dweight) return MSSM_ERROR_INVALID_VALUE;
  if (rows > 0) {
    if (!dy || !x || !weight || !mean || !rstd || !dx) return MSSM_ERROR_INVALID_VALUE;
    st = check_workspace(workspace, workspace_bytes, mssm::norm_bwd_workspace(rows, D, dtype));
    if (st != MSSM_SUCCESS) return st;
  }
  mssm::NormBwdArgs a;
  a.dy = dy, a.dsum = dsum, a.x = x, a.weight = weight, a.mean = mean, a.rstd = rstd;
  a.dx = dx, a.dweight = dweight, a.dbias = dbias;
  a.rows = rows, a.D = D, a.dtype = dtype;
  return done(mssm::launch_norm_bwd(a, workspace, static_cast<hipStream_t>(stream)),
              "layer norm backward launch");
}

}  // extern "C"
