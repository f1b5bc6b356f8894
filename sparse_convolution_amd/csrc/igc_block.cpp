// extern "C" entry points of the operators between convolutions: layer norm and 8-bit activation
// checkpoints. Every check runs on the host before any launch.
#include <hip/hip_runtime.h>

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

}  // namespace

extern "C" {

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
