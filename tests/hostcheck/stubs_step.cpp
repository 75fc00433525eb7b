// Host-only stand-ins for the launchers of the operators that close a training step, beside stubs.cpp:
// every buffer and workspace region that a launch would touch is checked against the memory that the
// driver registered.
#include <cstdio>
#include <cstdlib>

#include "../../routing_grouped_expert_fp32_amd/csrc/step_rules.h"
#include "hostcheck_step.h"

namespace hostcheck {
void need(const char* launcher, const char* what, const void* p, size_t bytes);   // stubs.cpp
namespace {
long g_step_launches = 0;
}
long step_launches() { return g_step_launches; }
}  // namespace hostcheck

using hostcheck::need;

namespace beam {

hipError_t launch_gated(const void* x, const void* w, const int32_t* offsets, void* h, void* gu, int R, int E,
                        int F, int K, bool, hipStream_t) {
  const char* l = "gated";
  need(l, "x", x, 2 * (size_t)R * K);
  need(l, "w", w, 4 * (size_t)E * F * K);
  need(l, "offsets", offsets, 4 * ((size_t)E + 1));
  need(l, "h", h, 2 * (size_t)R * F);
  if (gu) need(l, "gu", gu, 4 * (size_t)R * F);
  ++hostcheck::g_step_launches;
  return hipSuccess;
}

hipError_t launch_gated_bwd(const void* dy, const void* w, const void* gu, const int32_t* offsets,
                            const float* scale, void* d_gu, void* h, float* d_scale, float* parts, int R, int E,
                            int F, int H, hipStream_t) {
  const char* l = "gated_bwd";
  need(l, "dy", dy, 2 * (size_t)R * H);
  need(l, "w", w, 2 * (size_t)E * F * H);
  need(l, "gu", gu, 4 * (size_t)R * F);
  need(l, "offsets", offsets, 4 * ((size_t)E + 1));
  need(l, "d_gu", d_gu, 4 * (size_t)R * F);
  need(l, "h", h, 2 * (size_t)R * F);
  if (scale) {
    need(l, "scale", scale, 4 * (size_t)R);
    need(l, "d_scale", d_scale, 4 * (size_t)R);
    size_t rows = 0;
    with_gated_bwd_tile(R, E, F, H, [&](auto s) { rows = ceil_div(F, kScaleCols<decltype(s)>); });
    need(l, "parts", parts, 4 * rows * R);
  }
  ++hostcheck::g_step_launches;
  return hipSuccess;
}

hipError_t launch_head_loss(const HeadArgs& a, float* loss, float* lse, char* ws, hipStream_t) {
  const char* l = "head_loss";
  const size_t t = a.T;
  const HeadLayout L = head_layout(a.T, a.V, a.H);
  need(l, "x", a.x, 2 * t * a.H);
  need(l, "w", a.w, 2 * (size_t)a.V * a.H);
  need(l, "targets", a.targets, 4 * t);
  need(l, "loss", loss, 4 * t);
  need(l, "lse", lse, 4 * t);
  need(l, "stats", ws, 8 * t * L.slots);
  need(l, "at_target", ws + L.at_target, 4 * t);
  if (8 * t * L.slots > L.at_target || L.at_target % 256) std::abort();
  ++hostcheck::g_step_launches;
  return hipSuccess;
}

hipError_t launch_head_loss_bwd(const HeadArgs& a, const float* lse, const float* d_loss, uint16_t* dx, void* dw,
                                bool dw_bf16, char* ws, hipStream_t) {
  const char* l = "head_loss_bwd";
  const size_t t = a.T, h = a.H;
  need(l, "dw", dw, (dw_bf16 ? 2 : 4) * (size_t)a.V * h);
  ++hostcheck::g_step_launches;
  if (t == 0) return hipSuccess;
  const HeadBwdLayout L = head_bwd_layout(a.T, a.V, a.H);
  need(l, "x", a.x, 2 * t * h);
  need(l, "w", a.w, 2 * (size_t)a.V * h);
  need(l, "targets", a.targets, 4 * t);
  need(l, "lse", lse, 4 * t);
  need(l, "d_loss", d_loss, 4 * t);
  need(l, "dx", dx, 2 * t * h);
  const size_t dz = 2 * t * L.pitch, sums = L.direct() ? 0 : 4 * (size_t)L.dx.parts * t * h;
  need(l, "dz", ws, dz);
  need(l, "c", ws + L.c, 8 * t);
  need(l, "xc", ws + L.xc, 2 * t * h);
  if (sums) need(l, "sums", ws + L.sums, sums);
  if (dz > L.c || L.c + 8 * t > L.xc || L.xc + 2 * t * h > L.sums || L.xc % 16 || L.sums % 16 || L.sums + sums > L.total)
    std::abort();
  return hipSuccess;
}

hipError_t launch_adamw(const AdamwTensor* t, int n, const void* table, bool p_bf16, bool g_bf16, bool q8, bool copy,
                        bool, const AdamwScalars&, hipStream_t) {
  const char* l = "adamw";
  size_t entries = 0, chunks = 0;
  for (int i = 0; i < n; ++i) entries += t[i].count > 0, chunks += adamw_chunks(t[i].count);
  if (table) need(l, "table", table, sizeof(AdamwTableHead) + entries * sizeof(AdamwEntry) + 4 * chunks);
  for (int i = 0; i < n; ++i) {
    const size_t c = (size_t)t[i].count, blocks = 4 * ((c + 255) / 256);
    if (c == 0) continue;
    need(l, "param", t[i].param, (p_bf16 ? 2 : 4) * c);
    need(l, "grad", t[i].grad, (g_bf16 ? 2 : 4) * c);
    need(l, "m", t[i].m, (q8 ? 1 : 4) * c);
    need(l, "v", t[i].v, (q8 ? 1 : 4) * c);
    if (q8) need(l, "m_scale", t[i].m_scale, blocks);
    if (q8) need(l, "v_scale", t[i].v_scale, blocks);
    if (copy) need(l, "copy", t[i].copy, 2 * c);
  }
  ++hostcheck::g_step_launches;
  return hipSuccess;
}

}  // namespace beam
