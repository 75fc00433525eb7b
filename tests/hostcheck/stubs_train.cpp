// Host-only stand-ins for the launchers of the training operators, beside stubs.cpp: every buffer that
// a launch would touch, the workspace's regions among them, is checked against the memory that the
// driver registered.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../routing_grouped_expert_fp32_amd/csrc/train_rules.h"
#include "hostcheck_train.h"

namespace hostcheck {
void need(const char* launcher, const char* what, const void* p, size_t bytes);   // stubs.cpp
namespace {
long g_train_launches = 0;
}
long train_launches() { return g_train_launches; }
}  // namespace hostcheck

using hostcheck::need;

namespace beam {

hipError_t launch_grouped_rows(const void* a, const void* w, const int32_t* offsets, void* out,
                               int R, int E, int No, int Kc, bool, bool out_bf16, hipStream_t) {
  const char* l = "grouped_rows";
  need(l, "a", a, 2 * (size_t)R * Kc);
  need(l, "w", w, 2 * (size_t)E * No * Kc);
  need(l, "offsets", offsets, 4 * ((size_t)E + 1));
  need(l, "out", out, (out_bf16 ? 2 : 4) * (size_t)R * No);
  ++hostcheck::g_train_launches;
  return hipSuccess;
}

hipError_t launch_grouped_dw(const void* dy, const void* x, const int32_t* offsets, void* dw, int R,
                             int E, int N, int K, bool out_bf16, hipStream_t) {
  const char* l = "grouped_dw";
  if (R > 0) {
    need(l, "dy", dy, 2 * (size_t)R * N);
    need(l, "x", x, 2 * (size_t)R * K);
  }
  need(l, "offsets", offsets, 4 * ((size_t)E + 1));
  need(l, "dw", dw, (out_bf16 ? 2 : 4) * (size_t)E * N * K);
  ++hostcheck::g_train_launches;
  return hipSuccess;
}

hipError_t launch_boundary_bwd(const BoundaryBwdArgs& a, int64_t T, int H, hipStream_t) {
  const char* l = "boundary_bwd";
  const size_t TH = (size_t)T * H, gb = 4 * (size_t)H;
  need(l, "d_gamma_post", a.d_gamma_post, gb);
  need(l, "d_gamma_next", a.d_gamma_next, gb);
  if (T > 0) {
    need(l, "y", a.y, TH * (a.y_bf16 ? 2 : 4));
    need(l, "h", a.h, 2 * TH);
    need(l, "gamma_post", a.gamma_post, gb);
    need(l, "gamma_next", a.gamma_next, gb);
    if (a.d_h_in) need(l, "d_h_in", a.d_h_in, 2 * TH);
    need(l, "d_x", a.d_x, 2 * TH);
    need(l, "d_y", a.d_y, TH * (a.y_bf16 ? 2 : 4));
    need(l, "d_h", a.d_h, 2 * TH);
    need(l, "parts", a.parts, 2 * gb * (size_t)boundary_bwd_parts(T, H));
  }
  ++hostcheck::g_train_launches;
  return hipSuccess;
}

hipError_t launch_orthogonalise(const void* g, bool g_bf16, uint16_t* out, int n_mats, int rows,
                                int cols, int steps, const float*, float, char* ws, hipStream_t) {
  const char* l = "orthogonalise";
  const size_t b = (size_t)n_mats, count = b * rows * cols;
  need(l, "g", g, (g_bf16 ? 2 : 4) * count);
  need(l, "out", out, 2 * count);
  const NsLayout L = ns_layout(n_mats, rows, cols);
  if (steps > kNsMaxSteps || L.m != std::min(rows, cols) || L.n != std::max(rows, cols) ||
      L.mp < L.m || L.ld < L.n || L.mp % 8 || L.ld % 8)
    return hipErrorInvalidValue;
  if (!ns_is_small(L.m, L.n)) {
    // what the launches read and write of each region
    const GramParts split = gram_parts(n_mats, L.m, L.n);
    struct Region {
      const char* name;
      size_t at, bytes;
    };
    std::vector<Region> r = {
        {"parts", L.parts, 8 * b * ns_norm_parts((int64_t)rows * cols)},
        {"units", L.units, 4 * (b * kNsMaxSteps)},
        {"hi 0", L.hi[0], 2 * b * L.m * L.ld},
        {"hi 1", L.hi[1], 2 * b * L.m * L.ld},
        {"lo", L.lo, 2 * b * L.m * L.ld},
        {"gram", L.gram, 2 * b * L.m * L.mp},
        {"poly", L.poly, 2 * b * L.m * L.mp}};
    if (split.parts > 1) {
      if (split.kp % kStageK || (int64_t)split.parts * split.kp < L.n ||
          (int64_t)(split.parts - 1) * split.kp >= L.n)
        return hipErrorInvalidValue;
      r.push_back({"sums", L.sums,
                   4 * b * (size_t)ns_triangle(ceil_div(L.m, 64)) * split.parts * 64 * 64});
    }
    std::sort(r.begin(), r.end(), [](const Region& x, const Region& y) { return x.at < y.at; });
    for (size_t i = 0; i < r.size(); ++i) {
      need(l, r[i].name, ws + r[i].at, r[i].bytes);
      const size_t next = i + 1 < r.size() ? r[i + 1].at : L.total;
      if (r[i].at % 256 || r[i].at + r[i].bytes > next) {
        std::fprintf(stderr, "%s: region %s of %d x %d x %d reaches into the next\n", l, r[i].name,
                     n_mats, rows, cols);
        std::abort();
      }
    }
  }
  ++hostcheck::g_train_launches;
  return hipSuccess;
}

}  // namespace beam
