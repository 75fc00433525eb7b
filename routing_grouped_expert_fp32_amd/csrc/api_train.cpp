// C ABI of the training operators: argument validation and dispatch. Declarations, argument meanings
// and error behaviour: include/beam_moe.h.
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "../../include/beam_moe.h"
#include "common.h"
#include "host_checks.h"

namespace {

using namespace beam::host;

constexpr int32_t kMaxGroupedExperts = 4096;
constexpr int32_t kMaxGroupedWidth = 1 << 20;
constexpr int32_t kMaxNsSide = 1 << 16;

beam_status_t check_grouped_shape(int64_t R, int32_t E, int32_t N, int32_t K, int32_t out_dtype) {
  if (R < 0 || E <= 0 || N <= 0 || K <= 0) return BEAM_ERR_SHAPE;
  if (out_dtype != BEAM_F32 && out_dtype != BEAM_BF16) return BEAM_ERR_DTYPE;
  if (N % 8 != 0 || K % 8 != 0 || N > kMaxGroupedWidth || K > kMaxGroupedWidth ||
      E > kMaxGroupedExperts || R >= (int64_t(1) << 31) || (int64_t)N * K >= (int64_t(1) << 31) ||
      !beam::grouped_grid_fits(R, E, N, K))
    return BEAM_ERR_UNSUPPORTED;
  return BEAM_OK;
}

beam_status_t check_grouped_buffers(const void* a, size_t a_bytes, const void* b, size_t b_bytes,
                                    const int32_t* offsets, int32_t E, const void* out,
                                    size_t out_bytes) {
  if (!a || !b || !offsets || !out) return BEAM_ERR_NULL;
  if (!aligned16(a) || !aligned16(b) || !aligned16(offsets) || !aligned16(out))
    return BEAM_ERR_ALIGN;
  if (any_alias({rng(a, a_bytes), rng(b, b_bytes), rng(offsets, sizeof(int32_t) * ((size_t)E + 1))},
                {rng(out, out_bytes)}))
    return BEAM_ERR_ALIAS;
  return check_device();
}

beam_status_t check_ns(int64_t n_mats, int32_t rows, int32_t cols) {
  if (n_mats < 0 || rows <= 0 || cols <= 0) return BEAM_ERR_SHAPE;
  if (rows > kMaxNsSide || cols > kMaxNsSide || !beam::ns_grid_fits(n_mats, rows, cols))
    return BEAM_ERR_UNSUPPORTED;
  return BEAM_OK;
}

}  // namespace

extern "C" {

beam_status_t beam_moe_grouped_mm(const void* x, const void* w, const int32_t* offsets, void* out,
                                  int64_t R, int32_t E, int32_t N, int32_t K, int32_t out_dtype,
                                  void* stream) {
  beam_status_t rc = check_grouped_shape(R, E, N, K, out_dtype);
  if (rc != BEAM_OK) return rc;
  if (R == 0) return BEAM_OK;
  const size_t r = (size_t)R, n = (size_t)N, k = (size_t)K;
  if ((rc = check_grouped_buffers(x, 2 * r * k, w, 2 * (size_t)E * n * k, offsets, E, out,
                                  dtype_bytes(out_dtype) * r * n)) != BEAM_OK)
    return rc;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return launched(beam::launch_grouped_rows(x, w, offsets, out, (int)R, E, N, K, false,
                                            out_dtype == BEAM_BF16, st),
                  st, "grouped_mm");
}

beam_status_t beam_moe_grouped_mm_dx(const void* dy, const void* w, const int32_t* offsets,
                                     void* dx, int64_t R, int32_t E, int32_t N, int32_t K,
                                     int32_t out_dtype, void* stream) {
  beam_status_t rc = check_grouped_shape(R, E, N, K, out_dtype);
  if (rc != BEAM_OK) return rc;
  if (R == 0) return BEAM_OK;
  const size_t r = (size_t)R, n = (size_t)N, k = (size_t)K;
  if ((rc = check_grouped_buffers(dy, 2 * r * n, w, 2 * (size_t)E * n * k, offsets, E, dx,
                                  dtype_bytes(out_dtype) * r * k)) != BEAM_OK)
    return rc;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return launched(beam::launch_grouped_rows(dy, w, offsets, dx, (int)R, E, K, N, true,
                                            out_dtype == BEAM_BF16, st),
                  st, "grouped_mm_dx");
}

beam_status_t beam_moe_grouped_mm_dw(const void* dy, const void* x, const int32_t* offsets,
                                     void* dw, int64_t R, int32_t E, int32_t N, int32_t K,
                                     int32_t out_dtype, void* stream) {
  beam_status_t rc = check_grouped_shape(R, E, N, K, out_dtype);
  if (rc != BEAM_OK) return rc;
  const size_t r = (size_t)R, n = (size_t)N, k = (size_t)K;
  // no rows at all: every gradient is zero, dy and x are not read
  if (R == 0 && offsets && dw && !dy && !x) dy = x = offsets;
  if ((rc = check_grouped_buffers(dy, 2 * r * n, x, 2 * r * k, offsets, E, dw,
                                  dtype_bytes(out_dtype) * (size_t)E * n * k)) != BEAM_OK)
    return rc;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return launched(beam::launch_grouped_dw(dy, x, offsets, dw, (int)R, E, N, K,
                                          out_dtype == BEAM_BF16, st),
                  st, "grouped_mm_dw");
}

size_t beam_residual_boundary_backward_workspace_bytes(int64_t T, int32_t hidden) {
  if (T <= 0 || hidden <= 0 || hidden > beam::boundary_max_hidden()) return 0;
  return sizeof(float) * 2 * (size_t)beam::boundary_bwd_parts(T, hidden) * (size_t)hidden;
}

beam_status_t beam_residual_boundary_backward(
    const void* y, int32_t y_dtype, const void* h_out, const float* gamma_post,
    const float* gamma_next, const void* d_h_out, const void* d_x_next, void* d_y, void* d_h,
    float* d_gamma_post, float* d_gamma_next, int64_t T, int32_t hidden, int32_t depth_n, float eps,
    void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || hidden <= 0 || depth_n < 1 || !(std::isfinite(eps) && eps >= 0.f))
    return BEAM_ERR_SHAPE;
  if (y_dtype != BEAM_F32 && y_dtype != BEAM_BF16) return BEAM_ERR_DTYPE;
  if (hidden % 256 != 0 || hidden > beam::boundary_max_hidden() || T >= (int64_t(1) << 31))
    return BEAM_ERR_UNSUPPORTED;
  if (!d_gamma_post || !d_gamma_next) return BEAM_ERR_NULL;
  // without tokens the weights' gradients are still written (zeros), and nothing else is touched
  if (T > 0 && (!y || !h_out || !gamma_post || !gamma_next || !d_x_next || !d_y || !d_h || !workspace))
    return BEAM_ERR_NULL;
  const void* ptrs[] = {y,   h_out, gamma_post,   gamma_next,   d_h_out,  d_x_next,
                        d_y, d_h,   d_gamma_post, d_gamma_next, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return BEAM_ERR_ALIGN;   // d_h_out may be NULL, which is aligned
  const size_t need = beam_residual_boundary_backward_workspace_bytes(T, hidden);
  if (workspace_bytes < need) return BEAM_ERR_WORKSPACE;
  const size_t TH = (size_t)T * hidden, yb = dtype_bytes(y_dtype), gb = sizeof(float) * hidden;
  std::vector<Range> ins = {rng(y, TH * yb), rng(h_out, TH * 2), rng(gamma_post, gb),
                            rng(gamma_next, gb), rng(d_x_next, TH * 2)};
  // d_h may be d_h_out itself (in place)
  if (d_h_out && d_h_out != d_h) ins.push_back(rng(d_h_out, TH * 2));
  if (any_alias(ins, {rng(d_y, TH * yb), rng(d_h, TH * 2), rng(d_gamma_post, gb),
                      rng(d_gamma_next, gb), rng(workspace, need)}))
    return BEAM_ERR_ALIAS;
  const beam_status_t rc = check_device();
  if (rc != BEAM_OK) return rc;
  const double n = depth_n;
  beam::BoundaryBwdArgs a;
  a.y = y;
  a.y_bf16 = y_dtype == BEAM_BF16;
  a.h = reinterpret_cast<const uint16_t*>(h_out);
  a.gamma_post = gamma_post;
  a.gamma_next = gamma_next;
  a.d_h_in = reinterpret_cast<const uint16_t*>(d_h_out);
  a.d_x = reinterpret_cast<const uint16_t*>(d_x_next);
  a.d_y = d_y;
  a.d_h = reinterpret_cast<uint16_t*>(d_h);
  a.d_gamma_post = d_gamma_post;
  a.d_gamma_next = d_gamma_next;
  a.parts = reinterpret_cast<float*>(workspace);
  a.alpha = (float)std::sqrt((n - 1.0) / n);
  a.beta = (float)(1.0 / std::sqrt(n));
  a.eps = eps;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return launched(beam::launch_boundary_bwd(a, T, hidden, st), st, "residual_boundary_backward");
}

size_t beam_moe_orthogonalise_workspace_bytes(int64_t n_mats, int32_t rows, int32_t cols) {
  if (n_mats <= 0 || check_ns(n_mats, rows, cols) != BEAM_OK) return 0;
  return beam::ns_layout(n_mats, rows, cols).total;
}

beam_status_t beam_moe_orthogonalise(const void* g, int32_t g_dtype, void* out, int64_t n_mats,
                                     int32_t rows, int32_t cols, int32_t steps, const float* coeffs,
                                     float eps, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  beam_status_t rc = check_ns(n_mats, rows, cols);
  if (rc != BEAM_OK) return rc;
  if (g_dtype != BEAM_F32 && g_dtype != BEAM_BF16) return BEAM_ERR_DTYPE;
  if (!coeffs) return BEAM_ERR_NULL;
  if (steps < 1 || !(std::isfinite(eps) && eps >= 0.f)) return BEAM_ERR_SHAPE;
  // at a norm of 1 the stored B + s I is inside fp16 (|b| + |c| + |s| <= 65 of 255); iterates that the
  // coefficients let grow may still leave it
  for (int i = 0; i < 3; ++i)
    if (!(std::fabs(coeffs[i]) <= 16.f)) return BEAM_ERR_SHAPE;
  if (steps > beam::kNsMaxSteps) return BEAM_ERR_UNSUPPORTED;
  if (n_mats == 0) return BEAM_OK;
  if (!g || !out || !workspace) return BEAM_ERR_NULL;
  if (!aligned16(g) || !aligned16(out) || !aligned16(workspace)) return BEAM_ERR_ALIGN;
  const size_t need = beam::ns_layout(n_mats, rows, cols).total;
  if (workspace_bytes < need) return BEAM_ERR_WORKSPACE;
  const size_t count = (size_t)n_mats * (size_t)rows * (size_t)cols;
  if (any_alias({rng(g, dtype_bytes(g_dtype) * count)}, {rng(out, 2 * count), rng(workspace, need)}))
    return BEAM_ERR_ALIAS;
  if ((rc = check_device()) != BEAM_OK) return rc;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return launched(beam::launch_orthogonalise(g, g_dtype == BEAM_BF16,
                                             reinterpret_cast<uint16_t*>(out), (int)n_mats, rows,
                                             cols, steps, coeffs, eps,
                                             reinterpret_cast<char*>(workspace), st),
                  st, "orthogonalise");
}

}  // extern "C"
