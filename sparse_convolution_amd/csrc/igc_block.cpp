// extern "C" entry points of the operators between convolutions: layer norm, 8-bit activation
// checkpoints, cross and window attention, norm and rotation of queries and keys, dropout. Every check runs on the host before any launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "igc_host.h"

using namespace igc;

namespace {

// Rows, channels and type of a feature array (fn names the call).
int check_rows(const char* fn, int64_t n, int32_t c, int32_t dtype) {
  const std::string f(fn);
  if (dtype != IGC_F32 && dtype != IGC_BF16) return set_error(IGC_ERR_INVALID_ARG, f + ": bad dtype");
  if (n < 0) return set_error(IGC_ERR_INVALID_ARG, f + ": n is negative");
  if (c < 1) return set_error(IGC_ERR_INVALID_ARG, f + ": c must be positive");
  if (n > INT32_MAX) return set_error(IGC_ERR_RANGE, f + ": n exceeds 2^31-1");
  if (c > kNormMaxChannels)
    return set_error(IGC_ERR_UNSUPPORTED, f + ": at most " + std::to_string(kNormMaxChannels) + " channels");
  return IGC_OK;
}

int norm_forward(const NormArgs& a, int32_t wdtype, hipStream_t s) {
  clear_error();
  int rc = check_rows(a.fn, a.n, a.c, a.dtype);
  if (rc) return rc;
  const std::string f(a.fn);
  if (wdtype != IGC_F32 && wdtype != a.dtype)
    return set_error(IGC_ERR_INVALID_ARG, f + ": weight and bias must be fp32 or of the features' type");
  if (!(a.eps >= 0.f) || std::isinf(a.eps)) return set_error(IGC_ERR_INVALID_ARG, f + ": eps must be finite and >= 0");
  if (a.n == 0) return IGC_OK;
  if (!a.x || !a.y || !a.rstd) return set_error(IGC_ERR_INVALID_ARG, f + ": d_x, d_y or d_rstd is null");
  if (a.x == a.y) return set_error(IGC_ERR_INVALID_ARG, f + ": d_y aliases d_x");
  return launch_norm(a, s);
}

int norm_backward(const NormArgs& a, int32_t wdtype, void* ws, size_t ws_bytes, hipStream_t s) {
  clear_error();
  int rc = check_rows(a.fn, a.n, a.c, a.dtype);
  if (rc) return rc;
  const std::string f(a.fn);
  if (wdtype != IGC_F32 && wdtype != a.dtype)
    return set_error(IGC_ERR_INVALID_ARG, f + ": weight must be fp32 or of the features' type");
  if (!a.dw != !a.db) return set_error(IGC_ERR_INVALID_ARG, f + ": d_dw and d_db come together");
  if (a.n == 0) {
    if (a.dw && (rc = fill_u32((uint32_t*)a.dw, a.c, 0u, s))) return rc;
    return a.db ? fill_u32((uint32_t*)a.db, a.c, 0u, s) : IGC_OK;
  }
  if (!a.dy || !a.y || !a.rstd) return set_error(IGC_ERR_INVALID_ARG, f + ": d_dy, d_dx or d_rstd is null");
  if (a.y == a.dy || a.y == a.x) return set_error(IGC_ERR_INVALID_ARG, f + ": d_dx aliases an input");
  if (a.dw) {
    size_t need = 0;
    if ((rc = igc_layer_norm_workspace(a.n, a.c, &need))) return rc;
    if (!ws || ws_bytes < need)
      return set_error(IGC_ERR_CAPACITY, f + ": the weight gradient needs " + std::to_string(need) +
                                             " bytes of workspace (igc_layer_norm_workspace)");
  }
  return launch_norm_bwd(a, ws, s);
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

// Checks the problem's description and fills the device arguments (fn names the call).
int attention_args(const char* fn, const igc_attention_t* p, AttnArgs& a) {
  clear_error();
  const std::string f(fn);
  if (!p) return set_error(IGC_ERR_INVALID_ARG, f + ": the problem is null");
  if (p->dtype != IGC_F32 && p->dtype != IGC_BF16) return set_error(IGC_ERR_INVALID_ARG, f + ": bad dtype");
  if (p->n_q < 0 || p->n_k < 0) return set_error(IGC_ERR_INVALID_ARG, f + ": n_q or n_k is negative");
  if (p->batch < 1 || p->heads < 1 || p->kv_heads < 1 || p->dim < 1)
    return set_error(IGC_ERR_INVALID_ARG, f + ": batch, heads, kv_heads and dim must be positive");
  if (p->heads % p->kv_heads)
    return set_error(IGC_ERR_INVALID_ARG, f + ": heads must be a multiple of kv_heads");
  if (p->dim > kAttnMaxDim)
    return set_error(IGC_ERR_UNSUPPORTED, f + ": at most " + std::to_string(kAttnMaxDim) + " channels a head");
  if (p->batch > 1 && (!p->d_q_offsets || !p->d_kv_offsets))
    return set_error(IGC_ERR_INVALID_ARG, f + ": several sequences need d_q_offsets and d_kv_offsets");
  // The kernels exponentiate in base 2, with scale * log2(e).
  if (!(p->scale > 0.f) || std::isinf(p->scale * 1.4426950408889634f))
    return set_error(IGC_ERR_INVALID_ARG, f + ": scale must be positive, and finite times log2(e)");
  const int64_t group = p->heads / p->kv_heads;
  if (p->n_k > kAttnMaxRows || p->n_q > kAttnMaxRows / group)
    return set_error(IGC_ERR_RANGE, f + ": n_q times heads per key head, and n_k, can be at most 2^31 - 1024");
  // Workgroups: at most 128 parts of each tile (of 128 rows, or of a few where sequences have only those).
  if ((std::min(p->n_q * group / 128, INT64_C(1) << 31) + (int64_t)p->batch * 9) * p->kv_heads > INT32_MAX / 128 ||
      (p->n_k / 128 + p->batch) * (int64_t)p->kv_heads > INT32_MAX / 128)
    return set_error(IGC_ERR_RANGE, f + ": too many rows and heads for one launch");
  a.fn = fn;
  a.qo = p->d_q_offsets, a.ko = p->d_kv_offsets, a.mask = p->d_key_mask;
  a.nq = p->n_q, a.nk = p->n_k;
  for (int i = 0; i < 2; ++i) a.qs[i] = p->q_stride[i], a.ks[i] = p->k_stride[i], a.vs[i] = p->v_stride[i];
  a.batch = p->batch, a.heads = p->heads, a.kv_heads = p->kv_heads, a.group = (int)group, a.dim = p->dim;
  a.scale = p->scale;
  return IGC_OK;
}

// Which operands may be read 16 bytes at a time.
void attention_alignment(const igc_attention_t* p, AttnArgs& a, const void* dense) {
  const int64_t e = p->dtype == IGC_BF16 ? 8 : 4;
  const bool d = p->dim % 8 == 0;
  // A tile of at most 64 rows (and the group's heads) is addressed with 32-bit byte offsets from its start.
  auto strides = [&](const int64_t* s) {
    return s[0] % e == 0 && s[1] % e == 0 && s[0] >= 0 && s[1] >= 0 && s[0] < (1 << 22) && s[1] < (1 << 28) / a.group;
  };
  a.qvec = d && aligned16(a.q) && strides(a.qs);
  a.kvec = d && aligned16(a.k) && aligned16(a.v) && strides(a.ks) && strides(a.vs);
  a.ovec = d && aligned16(dense) && (int64_t)a.heads * a.dim < (1 << 22);
}

// Floats before the statistics in the forward workspace: the partial results, up to the next 16 bytes.
size_t forward_results(const AttnArgs& a) { return ((size_t)a.splits * a.nq * a.heads * a.dim + 3) / 4 * 4; }
size_t forward_bytes(const AttnArgs& a) {
  return a.splits > 1 ? (forward_results(a) + (size_t)a.splits * a.nq * a.heads * 2) * sizeof(float) : 0;
}

// Checks a workspace of which `need` bytes are used.
int check_workspace(const char* fn, bool windowed, const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return IGC_OK;
  const std::string family = windowed ? "igc_window_attention" : "igc_cross_attention";
  if (!ws || ws_bytes < need)
    return set_error(IGC_ERR_CAPACITY, std::string(fn) + ": needs " + std::to_string(need) +
                                           " bytes of workspace (" + family + "_workspace)");
  if (!aligned16(ws)) return set_error(IGC_ERR_INVALID_ARG, std::string(fn) + ": d_ws must be aligned to 16 bytes");
  return IGC_OK;
}

// Checks a window (null: none) and adds it to the device arguments.
int window_args(const char* fn, const Window* w, AttnArgs& a) {
  if (!w) return IGC_OK;
  const std::string f(fn);
  if (w->left < -1 || w->right < -1) return set_error(IGC_ERR_INVALID_ARG, f + ": left and right must be -1 (no limit) or more");
  if (w->sinks < 0) return set_error(IGC_ERR_INVALID_ARG, f + ": sinks is negative");
  a.windowed = w->left >= 0 || w->right >= 0;
  if (a.kl && !a.windowed)  // whose workspace would be cross attention's
    return set_error(IGC_ERR_INVALID_ARG, f + ": d_kv_lengths need a limit to one side (left 2^31-1 leaves nothing out)");
  a.win = *w;
  if (w->left < 0 || w->left >= a.nk) a.win.sinks = 0;  // all keys before a query are visible anyway
  return IGC_OK;
}

int attention_workspace(const char* fn, const igc_attention_t* p, const Window* w, int32_t backward, size_t* bytes) {
  AttnArgs a;
  int rc = attention_args(fn, p, a);
  if (!rc) rc = window_args(fn, w, a);
  if (rc) return rc;
  if (!bytes) return set_error(IGC_ERR_INVALID_ARG, std::string(fn) + ": bytes is null");
  if (backward) {
    *bytes = attn_bwd_plan(p->dtype, a).floats * sizeof(float);
  } else {
    a.splits = attn_fwd_splits(p->dtype, a);
    *bytes = forward_bytes(a);
  }
  return IGC_OK;
}

int attention_forward(const char* fn, const igc_attention_t* p, const Window* w, const int32_t* d_kv_lengths, const void* d_q, const void* d_k, const void* d_v,
                      void* d_out, float* d_lse, void* d_ws, size_t ws_bytes, hipStream_t stream) {
  const std::string f(fn);
  AttnArgs a;
  a.kl = d_kv_lengths;
  int rc = attention_args(fn, p, a);
  if (!rc) rc = window_args(fn, w, a);
  if (rc || a.nq == 0) return rc;
  if (!d_q || !d_out || !d_lse || (a.nk > 0 && (!d_k || !d_v)))
    return set_error(IGC_ERR_INVALID_ARG, f + ": d_q, d_k, d_v, d_out or d_lse is null");
  if (d_out == d_q || (d_out == d_k && a.nk > 0) || (d_out == d_v && a.nk > 0))
    return set_error(IGC_ERR_INVALID_ARG, f + ": d_out aliases an input");
  a.q = d_q, a.k = d_k, a.v = d_v, a.out = d_out, a.lse = d_lse;
  attention_alignment(p, a, d_out);
  a.splits = attn_fwd_splits(p->dtype, a);
  if (const int bad = check_workspace(fn, w, d_ws, ws_bytes, forward_bytes(a))) return bad;
  a.part_a = (float*)d_ws;
  a.part_b = a.part_a + forward_results(a);
  return launch_attn_fwd(a, p->dtype, stream);
}

int attention_backward(const char* fn, const igc_attention_t* p, const Window* w, const void* d_q, const void* d_k, const void* d_v,
                       const void* d_out, const float* d_lse, const void* d_dout, void* d_dq, void* d_dk, void* d_dv, void* d_ws,
                       size_t ws_bytes, hipStream_t stream) {
  const std::string f(fn);
  AttnArgs a;
  int rc = attention_args(fn, p, a);
  if (!rc) rc = window_args(fn, w, a);
  if (rc) return rc;
  if (!d_dk != !d_dv) return set_error(IGC_ERR_INVALID_ARG, f + ": d_dk and d_dv come together");
  if ((!d_dq || a.nq == 0) && (!d_dk || a.nk == 0)) return IGC_OK;
  if (a.nq > 0 && (!d_q || !d_out || !d_lse || !d_dout))
    return set_error(IGC_ERR_INVALID_ARG, f + ": d_q, d_out, d_lse or d_dout is null");
  if (a.nk > 0 && (!d_k || !d_v)) return set_error(IGC_ERR_INVALID_ARG, f + ": d_k or d_v is null");
  const void* in[] = {d_q, d_k, d_v, d_out, d_dout};
  for (const void* g : {(const void*)d_dq, (const void*)d_dk, (const void*)d_dv})
    for (const void* x : in)
      if (g && g == x) return set_error(IGC_ERR_INVALID_ARG, f + ": a gradient aliases an input");
  a.q = d_q, a.k = d_k, a.v = d_v, a.out_in = d_out, a.lse_in = d_lse, a.dout = d_dout;
  a.dq = d_dq, a.dk = d_dk, a.dv = d_dv;
  attention_alignment(p, a, (const void*)((uintptr_t)d_out | (uintptr_t)d_dout | (uintptr_t)d_dq | (uintptr_t)d_dk |
                                          (uintptr_t)d_dv));
  const AttnBwdPlan plan = attn_bwd_plan(p->dtype, a);
  if (d_dk && plan.dkv_threads > UINT32_MAX)
    return set_error(IGC_ERR_RANGE, f + ": too many keys, key heads and sinks for one launch");
  if (const int bad = check_workspace(fn, w, d_ws, ws_bytes, plan.floats * sizeof(float))) return bad;
  return launch_attn_bwd(a, p->dtype, plan, d_ws, stream);
}

// Checks the problem's description and fills the device arguments (fn names the call).
int qk_args(const char* fn, const igc_qk_t* p, QkArgs& a) {
  clear_error();
  const std::string f(fn);
  if (!p) return set_error(IGC_ERR_INVALID_ARG, f + ": the problem is null");
  if (p->dtype != IGC_F32 && p->dtype != IGC_BF16) return set_error(IGC_ERR_INVALID_ARG, f + ": bad dtype");
  if (p->n < 0) return set_error(IGC_ERR_INVALID_ARG, f + ": n is negative");
  if (p->heads < 1 || p->kv_heads < 0 || p->dim < 1)
    return set_error(IGC_ERR_INVALID_ARG, f + ": heads and dim must be positive, kv_heads not negative");
  if (p->dim > kAttnMaxDim)
    return set_error(IGC_ERR_UNSUPPORTED, f + ": at most " + std::to_string(kAttnMaxDim) + " channels a head");
  if (p->n > INT32_MAX) return set_error(IGC_ERR_RANGE, f + ": n exceeds 2^31-1");
  if ((int64_t)p->heads + p->kv_heads > 65535) return set_error(IGC_ERR_RANGE, f + ": at most 65535 heads in all");
  if (p->axes < 0 || p->axes > 3) return set_error(IGC_ERR_INVALID_ARG, f + ": axes must be 0 to 3");
  if (p->axes > 0 && (p->pairs < 1 || 2 * (int64_t)p->axes * p->pairs > p->dim))
    return set_error(IGC_ERR_INVALID_ARG, f + ": the pairs of all axes must fit the head");
  if (p->layout != 0 && p->layout != 1) return set_error(IGC_ERR_INVALID_ARG, f + ": layout must be 0 (halves) or 1 (interleaved)");
  if (p->norm && (!(p->eps >= 0.f) || std::isinf(p->eps)))
    return set_error(IGC_ERR_INVALID_ARG, f + ": eps must be finite and >= 0");
  if (!std::isfinite(p->amplitude)) return set_error(IGC_ERR_INVALID_ARG, f + ": amplitude must be finite");
  a.fn = fn, a.dtype = p->dtype, a.n = p->n, a.dim = p->dim, a.heads[0] = p->heads, a.heads[1] = p->kv_heads;
  for (int i = 0; i < 2; ++i) a.xs[0][i] = p->q_stride[i], a.xs[1][i] = p->k_stride[i];
  a.axes = p->axes, a.pairs = p->axes ? p->pairs : 0, a.interleaved = p->layout, a.norm = p->norm != 0;
  a.eps = p->eps, a.amplitude = p->amplitude, a.positions = p->d_positions, a.frequencies = p->d_frequencies;
  return IGC_OK;
}

// The rest of a call's checks: arrays for n rows, and the weights' type.
int qk_arrays(QkArgs& a, int32_t wdtype, bool inputs) {
  const std::string f(a.fn);
  if (wdtype != IGC_F32 && wdtype != a.dtype)
    return set_error(IGC_ERR_INVALID_ARG, f + ": weights must be fp32 or of the data's type");
  a.wf32 = wdtype == IGC_F32;
  for (int t = 0; t < 2; ++t)
    if (a.heads[t] > 0 && ((inputs && !a.x[t]) || !a.y[t]))
      return set_error(IGC_ERR_INVALID_ARG, f + ": an array of queries or keys is null");
  if (a.axes > 0 && (!a.positions || !a.frequencies))
    return set_error(IGC_ERR_INVALID_ARG, f + ": d_positions or d_frequencies is null");
  const void* in[] = {inputs ? a.x[0] : nullptr, inputs && a.heads[1] ? a.x[1] : nullptr, a.dy[0], a.heads[1] ? a.dy[1] : nullptr};
  for (int t = 0; t < 2; ++t)
    for (const void* x : in)
      if (a.heads[t] > 0 && x && x == a.y[t]) return set_error(IGC_ERR_INVALID_ARG, f + ": an output aliases an input");
  if (a.heads[1] > 0 && a.y[0] == a.y[1]) return set_error(IGC_ERR_INVALID_ARG, f + ": the outputs alias each other");
  return IGC_OK;
}

size_t qk_bytes(const QkArgs& a) {
  return a.n > 0 && a.norm ? (size_t)qk_parts(a.dtype, a.n, a.heads[0] + a.heads[1], a.dim) * 2 * a.dim * sizeof(float) : 0;
}

}  // namespace

extern "C" {

int igc_qk_norm_rotary_workspace(const igc_qk_t* p, size_t* bytes) {
  const char* fn = "igc_qk_norm_rotary_workspace";
  QkArgs a;
  const int rc = qk_args(fn, p, a);
  if (rc) return rc;
  if (!bytes) return set_error(IGC_ERR_INVALID_ARG, "igc_qk_norm_rotary_workspace: bytes is null");
  *bytes = qk_bytes(a);
  return IGC_OK;
}

int igc_qk_norm_rotary(const igc_qk_t* p, const void* d_q, const void* d_k, const void* d_qw, const void* d_kw,
                       int32_t wdtype, void* d_yq, void* d_yk, igc_stream stream) {
  QkArgs a;
  int rc = qk_args("igc_qk_norm_rotary", p, a);
  if (rc || a.n == 0) return rc;
  a.x[0] = d_q, a.x[1] = d_k, a.w[0] = d_qw, a.w[1] = d_kw, a.y[0] = d_yq, a.y[1] = d_yk;
  rc = qk_arrays(a, wdtype, true);
  return rc ? rc : launch_qk(a, false, (hipStream_t)stream);
}

int igc_qk_norm_rotary_backward(const igc_qk_t* p, const void* d_dyq, const void* d_dyk, const void* d_q, const void* d_k,
                                const void* d_qw, const void* d_kw, int32_t wdtype, void* d_dq, void* d_dk, float* d_dqw,
                                float* d_dkw, void* d_ws, size_t ws_bytes, igc_stream stream) {
  const std::string f = "igc_qk_norm_rotary_backward";
  QkArgs a;
  int rc = qk_args("igc_qk_norm_rotary_backward", p, a);
  if (rc) return rc;
  if (d_dqw && !a.norm) return set_error(IGC_ERR_INVALID_ARG, f + ": without the norm there are no weight gradients");
  if (d_dqw && a.heads[1] > 0 && !d_dkw) return set_error(IGC_ERR_INVALID_ARG, f + ": d_dqw and d_dkw come together");
  if (a.n == 0 && !d_dqw) return IGC_OK;
  a.x[0] = d_q, a.x[1] = d_k, a.w[0] = d_qw, a.w[1] = d_kw, a.dy[0] = d_dyq, a.dy[1] = d_dyk, a.y[0] = d_dq, a.y[1] = d_dk;
  if (a.n > 0) {
    if (!d_dyq || (a.heads[1] > 0 && !d_dyk)) return set_error(IGC_ERR_INVALID_ARG, f + ": d_dyq or d_dyk is null");
    rc = qk_arrays(a, wdtype, a.norm);
    if (rc) return rc;
  }
  if (d_dqw) {
    a.dw[0] = d_dqw, a.dw[1] = a.heads[1] > 0 ? d_dkw : nullptr;
    const size_t need = qk_bytes(a);
    if (need > 0 && (!d_ws || ws_bytes < need))
      return set_error(IGC_ERR_CAPACITY, f + ": needs " + std::to_string(need) + " bytes of workspace (igc_qk_norm_rotary_workspace)");
    a.part = (float*)d_ws;
    if (a.n == 0) return launch_pair_sum(a.fn, nullptr, 0, a.dim, a.dw[0], a.dw[1], (hipStream_t)stream);
  }
  return launch_qk(a, true, (hipStream_t)stream);
}

int igc_dropout(const void* d_x, const void* d_residual, int64_t count, int32_t dtype, double p, uint64_t seed,
                uint64_t offset, const uint64_t* d_offset, void* d_y, igc_stream stream) {
  clear_error();
  if (dtype != IGC_F32 && dtype != IGC_BF16) return set_error(IGC_ERR_INVALID_ARG, "igc_dropout: bad dtype");
  if (count < 0) return set_error(IGC_ERR_INVALID_ARG, "igc_dropout: count is negative");
  if (!(p >= 0.0 && p <= 1.0)) return set_error(IGC_ERR_INVALID_ARG, "igc_dropout: p must be 0 to 1");
  if (count == 0) return IGC_OK;
  if (!d_x || !d_y) return set_error(IGC_ERR_INVALID_ARG, "igc_dropout: d_x or d_y is null");
  DropoutArgs a;
  a.dtype = dtype, a.x = d_x, a.residual = d_residual, a.y = d_y, a.count = count;
  a.drop = (uint32_t)std::rint(65536.0 * p);
  a.scale = a.drop < 65536 ? 65536.f / (float)(65536 - a.drop) : 0.f;
  a.seed = seed, a.offset = offset, a.d_offset = d_offset;
  return launch_dropout(a, (hipStream_t)stream);
}

int igc_cross_attention_workspace(const igc_attention_t* p, int32_t backward, size_t* bytes) {
  return attention_workspace("igc_cross_attention_workspace", p, nullptr, backward, bytes);
}

int igc_cross_attention(const igc_attention_t* p, const void* d_q, const void* d_k, const void* d_v, void* d_out,
                        float* d_lse, void* d_ws, size_t ws_bytes, igc_stream stream) {
  return attention_forward("igc_cross_attention", p, nullptr, nullptr, d_q, d_k, d_v, d_out, d_lse, d_ws, ws_bytes, (hipStream_t)stream);
}

int igc_cross_attention_backward(const igc_attention_t* p, const void* d_q, const void* d_k, const void* d_v,
                                 const void* d_out, const float* d_lse, const void* d_dout, void* d_dq, void* d_dk,
                                 void* d_dv, void* d_ws, size_t ws_bytes, igc_stream stream) {
  return attention_backward("igc_cross_attention_backward", p, nullptr, d_q, d_k, d_v, d_out, d_lse, d_dout, d_dq, d_dk, d_dv, d_ws,
                            ws_bytes, (hipStream_t)stream);
}

int igc_window_attention_workspace(const igc_attention_t* p, int32_t left, int32_t right, int32_t sinks, int32_t backward,
                                   size_t* bytes) {
  const Window w = {left, right, sinks};
  return attention_workspace("igc_window_attention_workspace", p, &w, backward, bytes);
}

int igc_window_attention(const igc_attention_t* p, int32_t left, int32_t right, int32_t sinks, const int32_t* d_kv_lengths,
                         const void* d_q, const void* d_k, const void* d_v, void* d_out, float* d_lse, void* d_ws, size_t ws_bytes,
                         igc_stream stream) {
  const Window w = {left, right, sinks};
  return attention_forward("igc_window_attention", p, &w, d_kv_lengths, d_q, d_k, d_v, d_out, d_lse, d_ws, ws_bytes, (hipStream_t)stream);
}

int igc_window_attention_backward(const igc_attention_t* p, int32_t left, int32_t right, int32_t sinks, const void* d_q,
                                  const void* d_k, const void* d_v, const void* d_out, const float* d_lse, const void* d_dout,
                                  void* d_dq, void* d_dk, void* d_dv, void* d_ws, size_t ws_bytes, igc_stream stream) {
  const Window w = {left, right, sinks};
  return attention_backward("igc_window_attention_backward", p, &w, d_q, d_k, d_v, d_out, d_lse, d_dout, d_dq, d_dk, d_dv, d_ws,
                            ws_bytes, (hipStream_t)stream);
}

int igc_layer_norm(const void* d_x, int64_t n, int32_t c, int32_t dtype, const void* d_w, const void* d_b,
                   int32_t wdtype, float eps, void* d_y, float* d_mean, float* d_rstd, igc_stream stream) {
  NormArgs a;
  a.fn = "igc_layer_norm";
  a.dtype = dtype, a.c = c, a.n = n, a.x = d_x, a.w = d_w, a.b = d_b, a.wf32 = wdtype == IGC_F32, a.eps = eps;
  a.y = d_y, a.mean = d_mean, a.rstd = d_rstd;
  if (n > 0 && !d_mean) return set_error(IGC_ERR_INVALID_ARG, "igc_layer_norm: d_mean is null");
  return norm_forward(a, wdtype, (hipStream_t)stream);
}

int igc_layer_norm_q8(const void* d_x, int64_t n, int32_t c, int32_t dtype, const void* d_w, const void* d_b,
                      int32_t wdtype, float eps, void* d_y, int8_t* d_codes, float* d_scales, float* d_rstd,
                      igc_stream stream) {
  NormArgs a;
  a.fn = "igc_layer_norm_q8";
  a.dtype = dtype, a.c = c, a.n = n, a.x = d_x, a.w = d_w, a.b = d_b, a.wf32 = wdtype == IGC_F32, a.eps = eps;
  a.y = d_y, a.codes = d_codes, a.scales = d_scales, a.rstd = d_rstd;
  if (n > 0 && (!d_codes || !d_scales))
    return set_error(IGC_ERR_INVALID_ARG, "igc_layer_norm_q8: d_codes or d_scales is null");
  return norm_forward(a, wdtype, (hipStream_t)stream);
}

int igc_layer_norm_workspace(int64_t n, int32_t c, size_t* bytes) {
  clear_error();
  if (!bytes) return set_error(IGC_ERR_INVALID_ARG, "igc_layer_norm_workspace: bytes is null");
  *bytes = 0;
  const int rc = check_rows("igc_layer_norm_workspace", n, c, IGC_F32);
  if (rc) return rc;
  *bytes = n > 0 ? (size_t)norm_bwd_parts(n, c) * 2 * (size_t)c * sizeof(float) : 0;
  return IGC_OK;
}

int igc_layer_norm_backward(const void* d_dy, const void* d_x, const float* d_mean, const float* d_rstd, int64_t n,
                            int32_t c, int32_t dtype, const void* d_w, int32_t wdtype, void* d_dx, float* d_dw,
                            float* d_db, void* d_ws, size_t ws_bytes, igc_stream stream) {
  NormArgs a;
  a.fn = "igc_layer_norm_backward";
  a.dtype = dtype, a.c = c, a.n = n, a.x = d_x, a.dy = d_dy, a.w = d_w, a.wf32 = wdtype == IGC_F32, a.y = d_dx;
  a.mean = const_cast<float*>(d_mean), a.rstd = const_cast<float*>(d_rstd), a.dw = d_dw, a.db = d_db;
  if (n > 0 && (!d_x || !d_mean))
    return set_error(IGC_ERR_INVALID_ARG, "igc_layer_norm_backward: d_x or d_mean is null");
  return norm_backward(a, wdtype, d_ws, ws_bytes, (hipStream_t)stream);
}

int igc_layer_norm_q8_backward(const void* d_dy, const int8_t* d_codes, const float* d_scales, const float* d_rstd,
                               int64_t n, int32_t c, int32_t dtype, const void* d_w, int32_t wdtype, void* d_dx,
                               float* d_dw, float* d_db, void* d_ws, size_t ws_bytes, igc_stream stream) {
  NormArgs a;
  a.fn = "igc_layer_norm_q8_backward";
  a.dtype = dtype, a.c = c, a.n = n, a.dy = d_dy, a.w = d_w, a.wf32 = wdtype == IGC_F32, a.y = d_dx;
  a.codes = const_cast<int8_t*>(d_codes), a.scales = const_cast<float*>(d_scales);
  a.rstd = const_cast<float*>(d_rstd), a.dw = d_dw, a.db = d_db;
  if (n > 0 && (!d_codes || !d_scales))
    return set_error(IGC_ERR_INVALID_ARG, "igc_layer_norm_q8_backward: d_codes or d_scales is null");
  return norm_backward(a, wdtype, d_ws, ws_bytes, (hipStream_t)stream);
}

int igc_checkpoint_pack(const void* d_x, int64_t n, int32_t c, int32_t dtype, int8_t* d_codes, float* d_scales,
                        igc_stream stream) {
  clear_error();
  const int rc = check_rows("igc_checkpoint_pack", n, c, dtype);
  if (rc || n == 0) return rc;
  if (!d_x || !d_codes || !d_scales)
    return set_error(IGC_ERR_INVALID_ARG, "igc_checkpoint_pack: d_x, d_codes or d_scales is null");
  return launch_pack(d_x, dtype, n, c, d_codes, d_scales, (hipStream_t)stream);
}

int igc_checkpoint_unpack(const int8_t* d_codes, const float* d_scales, int64_t n, int32_t c, int32_t dtype,
                          void* d_x, igc_stream stream) {
  clear_error();
  const int rc = check_rows("igc_checkpoint_unpack", n, c, dtype);
  if (rc || n == 0) return rc;
  if (!d_x || !d_codes || !d_scales)
    return set_error(IGC_ERR_INVALID_ARG, "igc_checkpoint_unpack: d_x, d_codes or d_scales is null");
  return launch_unpack(d_codes, d_scales, n, c, dtype, d_x, (hipStream_t)stream);
}

}  // extern "C"
