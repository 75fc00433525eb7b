// C ABI of the operators that close a training step (gated products, the head's loss, AdamW): argument
// validation and dispatch. Declarations, argument meanings and error behaviour: include/beam_moe.h.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/beam_moe.h"
#include "host_checks.h"
#include "step_rules.h"

namespace {

using namespace beam::host;

constexpr int32_t kMaxGroupedExperts = 4096;
constexpr int32_t kMaxWidth = 1 << 20;
constexpr int64_t kMaxVocab = int64_t(1) << 23;

// Rows, experts, hidden values and width of the gated products; `stored`: rows of an expert's weights.
beam_status_t check_gated_shape(int64_t R, int32_t E, int32_t F, int32_t K, int64_t stored) {
  if (R < 0 || E <= 0 || F <= 0 || K <= 0) return BEAM_ERR_SHAPE;
  if (F % 8 != 0 || K % 8 != 0 || F > kMaxWidth || K > kMaxWidth || E > kMaxGroupedExperts ||
      R >= (int64_t(1) << 31) || stored * K >= (int64_t(1) << 30))
    return BEAM_ERR_UNSUPPORTED;
  return BEAM_OK;
}

template <size_t N>
bool any_null(const void* const (&p)[N]) {
  return std::any_of(p, p + N, [](const void* q) { return !q; });
}
template <size_t N>
bool all_aligned(const void* const (&p)[N]) {
  return std::all_of(p, p + N, aligned16);
}

// Arrays of one number a row are read and written one by one: any address of theirs will do.
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
template <size_t N>
bool all_aligned4(const void* const (&p)[N]) {
  return std::all_of(p, p + N, aligned4);
}

// True where an output meets an input or another output (fixed lists: no allocation, nothing thrown).
template <size_t I, size_t O>
bool meets(const Range (&ins)[I], const Range (&outs)[O]) {
  auto cut = [](const Range& a, const Range& b) { return a.lo != a.hi && b.lo != b.hi && overlap(a, b); };
  for (size_t i = 0; i < O; ++i) {
    for (const Range& r : ins)
      if (cut(outs[i], r)) return true;
    for (size_t j = i + 1; j < O; ++j)
      if (cut(outs[i], outs[j])) return true;
  }
  return false;
}

beam_status_t check_head(int64_t T, int64_t V, int32_t H, float softcap) {
  if (T < 0 || V <= 0 || H <= 0 || !(std::isfinite(softcap) && softcap >= 0.f)) return BEAM_ERR_SHAPE;
  if (H % 8 != 0 || H > kMaxWidth || V > kMaxVocab || T >= (int64_t(1) << 31) ||
      (softcap != 0.f && !(softcap >= 0.0625f && softcap <= 1024.f)) || !beam::head_grid_fits(std::max<int64_t>(T, 1), V, H))
    return BEAM_ERR_UNSUPPORTED;
  return BEAM_OK;
}

beam_status_t check_adamw_types(int32_t n, int32_t p, int32_t g, int32_t state) {
  if (n < 0) return BEAM_ERR_SHAPE;
  if ((p != BEAM_F32 && p != BEAM_BF16) || (g != BEAM_F32 && g != BEAM_BF16) ||
      (state != BEAM_F32 && state != BEAM_FP8_E4M3))
    return BEAM_ERR_DTYPE;
  return BEAM_OK;
}

struct AdamwRanges {
  Range outs[6], grad;
};
AdamwRanges adamw_ranges(const beam_adamw_tensor& t, int32_t p, int32_t g, int32_t state) {
  const size_t n = (size_t)t.count, s = state == BEAM_F32 ? 0 : 4 * (size_t)beam::ceil_div(t.count, 256);
  return {{rng(t.param, n * dtype_bytes(p)), rng(t.m, n * dtype_bytes(state)), rng(t.v, n * dtype_bytes(state)),
           rng(t.m_scale, t.m_scale ? s : 0), rng(t.v_scale, t.v_scale ? s : 0), rng(t.copy, t.copy ? 2 * n : 0)},
          rng(t.grad, n * dtype_bytes(g))};
}

// The tensors one by one.
beam_status_t check_adamw_tensors(const beam_adamw_tensor* tensors, int32_t n, int32_t p, int32_t g,
                                  int32_t state) {
  if (n > 0 && !tensors) return BEAM_ERR_NULL;
  int64_t blocks = 0;
  bool copies = false, without = false;
  for (int32_t i = 0; i < n; ++i) {
    const beam_adamw_tensor& t = tensors[i];
    if (t.count < 0) return BEAM_ERR_SHAPE;
    if (t.count == 0) continue;
    if (t.count > beam::kAdamwMostValues) return BEAM_ERR_UNSUPPORTED;
    blocks += beam::ceil_div(t.count, 256);
    if (!t.param || !t.grad || !t.m || !t.v || (state == BEAM_FP8_E4M3 && (!t.m_scale || !t.v_scale)))
      return BEAM_ERR_NULL;
    const void* const wide[] = {t.param, t.grad, t.m, t.v, t.copy};
    if (!all_aligned(wide) || !aligned4(t.m_scale) || !aligned4(t.v_scale)) return BEAM_ERR_ALIGN;
    (t.copy ? copies : without) = true;
    const AdamwRanges r = adamw_ranges(t, p, g, state);
    const Range ins[] = {r.grad};
    if (meets(ins, r.outs)) return BEAM_ERR_ALIAS;
  }
  // copies are of FP32 weights, of all of the call's or of none
  if (copies && (p != BEAM_F32 || without)) return BEAM_ERR_UNSUPPORTED;
  if (blocks >= (int64_t(1) << 31)) return BEAM_ERR_UNSUPPORTED;
  return BEAM_OK;
}

}  // namespace

extern "C" {

beam_status_t beam_moe_gated_mm(const void* x, const void* w_gate_up, const int32_t* offsets, void* h, void* gu,
                                int64_t R, int32_t E, int32_t F, int32_t K, int32_t round_products, void* stream) {
  beam_status_t rc = check_gated_shape(R, E, F, K, 2 * (int64_t)F);
  if (rc != BEAM_OK) return rc;
  if (R == 0) return BEAM_OK;
  if (!beam::gated_grid_fits(R, E, F, K)) return BEAM_ERR_UNSUPPORTED;
  const void* const ptrs[] = {x, w_gate_up, offsets, h};
  if (any_null(ptrs)) return BEAM_ERR_NULL;
  if (!all_aligned(ptrs) || !aligned16(gu)) return BEAM_ERR_ALIGN;
  const size_t r = (size_t)R, f = (size_t)F, k = (size_t)K, e = (size_t)E;
  const Range ins[] = {rng(x, 2 * r * k), rng(w_gate_up, 4 * e * f * k), rng(offsets, 4 * (e + 1))};
  const Range outs[] = {rng(h, 2 * r * f), rng(gu, gu ? 4 * r * f : 0)};
  if (meets(ins, outs)) return BEAM_ERR_ALIAS;
  if ((rc = check_device()) != BEAM_OK) return rc;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return launched(beam::launch_gated(x, w_gate_up, offsets, h, gu, (int)R, E, F, K, round_products != 0, st), st, "gated_mm");
}

size_t beam_moe_gated_mm_backward_workspace_bytes(int64_t R, int32_t F) {
  if (R <= 0 || F <= 0 || R >= (int64_t(1) << 31) || F > kMaxWidth) return 0;
  return sizeof(float) * (size_t)R * (size_t)beam::gated_scale_parts(F);
}

beam_status_t beam_moe_gated_mm_backward(const void* dy, const void* w_down, const void* gu, const int32_t* offsets,
                                         const float* row_scale, void* d_gu, void* h, float* d_row_scale, int64_t R,
                                         int32_t E, int32_t F, int32_t H, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  beam_status_t rc = check_gated_shape(R, E, F, H, F);
  if (rc != BEAM_OK) return rc;
  if (R == 0) return BEAM_OK;
  if (!beam::gated_bwd_grid_fits(R, E, F, H)) return BEAM_ERR_UNSUPPORTED;
  const void* const ptrs[] = {dy, w_down, gu, offsets, d_gu, h};
  if (any_null(ptrs) || !row_scale != !d_row_scale || (row_scale && !workspace)) return BEAM_ERR_NULL;
  const void* const rows[] = {row_scale, d_row_scale};
  if (!all_aligned(ptrs) || !all_aligned4(rows) || !aligned16(workspace)) return BEAM_ERR_ALIGN;
  const size_t need = row_scale ? beam_moe_gated_mm_backward_workspace_bytes(R, F) : 0;
  if (workspace_bytes < need) return BEAM_ERR_WORKSPACE;
  const size_t r = (size_t)R, f = (size_t)F, n = (size_t)H, e = (size_t)E, s = row_scale ? 4 * r : 0;
  const Range ins[] = {rng(dy, 2 * r * n), rng(w_down, 2 * e * f * n), rng(gu, 4 * r * f), rng(offsets, 4 * (e + 1)),
                       rng(row_scale, s)};
  const Range outs[] = {rng(d_gu, 4 * r * f), rng(h, 2 * r * f), rng(d_row_scale, s), rng(workspace, need)};
  if (meets(ins, outs)) return BEAM_ERR_ALIAS;
  if ((rc = check_device()) != BEAM_OK) return rc;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return launched(beam::launch_gated_bwd(dy, w_down, gu, offsets, row_scale, d_gu, h, d_row_scale,
                                         reinterpret_cast<float*>(workspace), (int)R, E, F, H, st),
                  st, "gated_mm_backward");
}

size_t beam_head_loss_workspace_bytes(int64_t T, int64_t V, int32_t H) {
  if (T <= 0 || check_head(T, V, H, 0.f) != BEAM_OK) return 0;
  return beam::head_layout(T, V, H).total;
}

beam_status_t beam_head_loss(const void* x, const void* w, const int32_t* targets, float* loss, float* lse, int64_t T,
                             int64_t V, int32_t H, float softcap, void* workspace, size_t workspace_bytes,
                             void* stream) {
  beam_status_t rc = check_head(T, V, H, softcap);
  if (rc != BEAM_OK) return rc;
  if (T == 0) return BEAM_OK;
  const void* const ptrs[] = {x, w, workspace};
  const void* const rows[] = {targets, loss, lse};
  if (any_null(ptrs) || any_null(rows)) return BEAM_ERR_NULL;
  if (!all_aligned(ptrs) || !all_aligned4(rows)) return BEAM_ERR_ALIGN;
  const size_t need = beam::head_layout(T, V, H).total, t = (size_t)T, v = (size_t)V, n = (size_t)H;
  if (workspace_bytes < need) return BEAM_ERR_WORKSPACE;
  const Range ins[] = {rng(x, 2 * t * n), rng(w, 2 * v * n), rng(targets, 4 * t)};
  const Range outs[] = {rng(loss, 4 * t), rng(lse, 4 * t), rng(workspace, need)};
  if (meets(ins, outs)) return BEAM_ERR_ALIAS;
  if ((rc = check_device()) != BEAM_OK) return rc;
  const beam::HeadArgs a = {reinterpret_cast<const uint16_t*>(x), reinterpret_cast<const uint16_t*>(w), targets, T, V,
                            H, softcap};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return launched(beam::launch_head_loss(a, loss, lse, reinterpret_cast<char*>(workspace), st), st, "head_loss");
}

size_t beam_head_loss_backward_workspace_bytes(int64_t T, int64_t V, int32_t H) {
  if (T <= 0 || check_head(T, V, H, 0.f) != BEAM_OK) return 0;
  return beam::head_bwd_layout(T, V, H).total;
}

beam_status_t beam_head_loss_backward(const void* x, const void* w, const int32_t* targets, const float* lse,
                                      const float* d_loss, void* dx, void* dw, int32_t dw_dtype, int64_t T, int64_t V,
                                      int32_t H, float softcap, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  beam_status_t rc = check_head(T, V, H, softcap);
  if (rc != BEAM_OK) return rc;
  if (dw_dtype != BEAM_F32 && dw_dtype != BEAM_BF16) return BEAM_ERR_DTYPE;
  if (!dw) return BEAM_ERR_NULL;
  if (!aligned16(dw)) return BEAM_ERR_ALIGN;
  // without tokens dw is still written (zeros), and nothing else is touched
  const void* const ptrs[] = {x, w, dx, workspace};
  const void* const rows[] = {targets, lse, d_loss};
  if (T > 0 && (any_null(ptrs) || any_null(rows))) return BEAM_ERR_NULL;
  if (T > 0 && (!all_aligned(ptrs) || !all_aligned4(rows))) return BEAM_ERR_ALIGN;
  const size_t need = T > 0 ? beam::head_bwd_layout(T, V, H).total : 0;
  if (workspace_bytes < need) return BEAM_ERR_WORKSPACE;
  const size_t t = (size_t)T, v = (size_t)V, n = (size_t)H;
  const Range ins[] = {rng(x, 2 * t * n), rng(w, T > 0 ? 2 * v * n : 0), rng(targets, 4 * t), rng(lse, 4 * t),
                       rng(d_loss, 4 * t)};
  const Range outs[] = {rng(dx, 2 * t * n), rng(dw, dtype_bytes(dw_dtype) * v * n), rng(workspace, need)};
  if (meets(ins, outs)) return BEAM_ERR_ALIAS;
  if ((rc = check_device()) != BEAM_OK) return rc;
  const beam::HeadArgs a = {reinterpret_cast<const uint16_t*>(x), reinterpret_cast<const uint16_t*>(w), targets, T, V,
                            H, softcap};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return launched(beam::launch_head_loss_bwd(a, lse, d_loss, reinterpret_cast<uint16_t*>(dx), dw, dw_dtype == BEAM_BF16,
                                             reinterpret_cast<char*>(workspace), st),
                  st, "head_loss_backward");
}

size_t beam_moe_adamw_table_bytes(const beam_adamw_tensor* tensors, int32_t n) {
  size_t bytes = sizeof(beam::AdamwTableHead);
  for (int32_t i = 0; tensors && i < n; ++i)
    if (tensors[i].count > 0)
      bytes += sizeof(beam::AdamwEntry) + 4 * (size_t)beam::adamw_chunks(std::min(tensors[i].count, beam::kAdamwMostValues));
  return bytes;
}

beam_status_t beam_moe_adamw_table(const beam_adamw_tensor* tensors, int32_t n, int32_t param_dtype, int32_t grad_dtype,
                                   int32_t state_dtype, void* table, size_t table_bytes) {
  beam_status_t rc = check_adamw_types(n, param_dtype, grad_dtype, state_dtype);
  if (rc == BEAM_OK) rc = check_adamw_tensors(tensors, n, param_dtype, grad_dtype, state_dtype);
  if (rc != BEAM_OK || n == 0) return rc;
  if (!table) return BEAM_ERR_NULL;
  if (table_bytes < beam_moe_adamw_table_bytes(tensors, n)) return BEAM_ERR_WORKSPACE;
  struct Piece {
    Range r;
    bool out;
  };
  Piece* const all = new (std::nothrow) Piece[7 * (size_t)n];
  if (!all) return BEAM_ERR_UNSUPPORTED;
  size_t count = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (tensors[i].count == 0) continue;
    const AdamwRanges r = adamw_ranges(tensors[i], param_dtype, grad_dtype, state_dtype);
    for (const Range& o : r.outs)
      if (o.lo != o.hi) all[count++] = {o, true};
    all[count++] = {r.grad, false};
  }
  std::sort(all, all + count, [](const Piece& a, const Piece& b) { return a.r.lo < b.r.lo; });
  // in order of their starts: an output may reach no later piece, no piece an output (`end` of both kinds)
  uintptr_t out_end = 0, in_end = 0;
  for (size_t i = 0; i < count && rc == BEAM_OK; ++i) {
    if (all[i].r.lo < out_end || (all[i].out && all[i].r.lo < in_end)) rc = BEAM_ERR_ALIAS;
    uintptr_t& end = all[i].out ? out_end : in_end;
    end = std::max(end, all[i].r.hi);
  }
  delete[] all;
  if (rc != BEAM_OK) return rc;
  size_t used = 0;
  bool copies = false;   // of all or of none
  for (int32_t i = 0; i < n; ++i) {
    if (tensors[i].count == 0) continue;
    ++used;
    copies = tensors[i].copy != nullptr;
  }
  char* const entries = reinterpret_cast<char*>(table) + sizeof(beam::AdamwTableHead);
  char* const map = entries + used * sizeof(beam::AdamwEntry);
  int64_t chunks = 0, base = 0;
  int32_t k = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (tensors[i].count == 0) continue;
    beam::AdamwEntry e;
    std::memcpy(&e.t, &tensors[i], sizeof(e.t));
    e.first = (int32_t)chunks;
    e.base256 = (int32_t)base;
    std::memcpy(entries + k * sizeof(e), &e, sizeof(e));
    for (const int64_t end = chunks + beam::adamw_chunks(tensors[i].count); chunks < end; ++chunks)
      std::memcpy(map + 4 * chunks, &k, 4);
    base += beam::ceil_div(tensors[i].count, 256);
    ++k;
  }
  // a list of more chunks than a launch takes is launched without its table
  const beam::AdamwTableHead head = {
      k, (int32_t)std::min<int64_t>(chunks, beam::kAdamwMostChunks),
      beam::adamw_types(param_dtype == BEAM_BF16, grad_dtype == BEAM_BF16, state_dtype == BEAM_FP8_E4M3, copies), 0};
  std::memcpy(table, &head, sizeof(head));
  return BEAM_OK;
}

beam_status_t beam_moe_adamw(const beam_adamw_tensor* tensors, int32_t n, int32_t param_dtype, int32_t grad_dtype,
                             int32_t state_dtype, const beam_adamw_cfg* cfg, const void* device_table, void* stream) {
  beam_status_t rc = check_adamw_types(n, param_dtype, grad_dtype, state_dtype);
  if (rc != BEAM_OK) return rc;
  if (!cfg) return BEAM_ERR_NULL;
  const beam_adamw_cfg& c = *cfg;
  auto beta_ok = [](double b) { return b >= 0.0 && (float)b < 1.f; };
  if (!std::isfinite((float)c.lr) || !std::isfinite((float)c.weight_decay) || !beta_ok(c.beta1) || !beta_ok(c.beta2) ||
      !(c.eps >= 1e-30 && c.eps <= 1e30) || (!c.step_on_device && c.step < 1))
    return BEAM_ERR_SHAPE;
  if ((rc = check_adamw_tensors(tensors, n, param_dtype, grad_dtype, state_dtype)) != BEAM_OK) return rc;
  if (!aligned16(device_table)) return BEAM_ERR_ALIGN;
  if (!aligned4(c.step_on_device) || !aligned4(c.lr_on_device) || !aligned4(c.grad_scale)) return BEAM_ERR_ALIGN;
  bool some = false, copies = false;
  for (int32_t i = 0; i < n; ++i) {
    some = some || tensors[i].count > 0;
    copies = copies || (tensors[i].count > 0 && tensors[i].copy);
  }
  if (!some) return BEAM_OK;
  if ((rc = check_device()) != BEAM_OK) return rc;
  beam::AdamwScalars s = {};
  s.beta1 = (float)c.beta1;
  s.rest1 = (float)(1.0 - c.beta1);
  s.beta2 = (float)c.beta2;
  s.rest2 = (float)(1.0 - c.beta2);
  s.lr = (float)c.lr;
  s.weight_decay = (float)c.weight_decay;
  s.decay = (float)(1.0 - c.lr * c.weight_decay);
  s.eps = (float)c.eps;
  s.correction = (float)(1.0 / (1.0 - std::pow(c.beta1, (double)c.step)));
  s.root_scale = (float)(1.0 / std::sqrt(1.0 - std::pow(c.beta2, (double)c.step)));
  s.log_beta1 = (float)std::log(c.beta1);
  s.log_beta2 = (float)std::log(c.beta2);
  s.key = beam::mix32(c.seed);
  if (!c.step_on_device) s.key = beam::mix32(s.key + (uint32_t)c.step);
  s.step = c.step_on_device;
  s.lr_now = c.lr_on_device;
  s.grad_scale = c.grad_scale;
  static_assert(sizeof(beam::AdamwTensor) == sizeof(beam_adamw_tensor) &&
                    offsetof(beam::AdamwTensor, count) == offsetof(beam_adamw_tensor, count),
                "one layout");
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return launched(beam::launch_adamw(reinterpret_cast<const beam::AdamwTensor*>(tensors), n, device_table,
                                     param_dtype == BEAM_BF16, grad_dtype == BEAM_BF16, state_dtype == BEAM_FP8_E4M3, copies, c.stochastic != 0,
                                     s, st),
                  st, "adamw");
}

}  // extern "C"
