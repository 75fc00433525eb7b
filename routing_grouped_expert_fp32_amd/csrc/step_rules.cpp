// Launch bounds and workspace sizes of the operators that close a training step (see step_rules.h).
#include "step_rules.h"

namespace beam {

bool gated_is_narrow(int64_t R, int64_t E, int64_t Fw, int64_t K) {
  const double full = (double)std::min(R, E), mean = (double)R / full;
  const double blocks = E == 1                                      ? std::ceil(mean / 32)
                        : mean + 2.5 * std::sqrt(mean) <= 32.0 ? 1.0
                                                                    : mean / 32 + 0.5;
  return K >= 1280 && full * blocks * ceil_div(Fw, kNarrowCols) <= 1.5 * kGroupedCus;
}

bool gated_grid_fits(int64_t R, int64_t E, int64_t Fw, int64_t K) {
  // the narrowest tiles' launch fits: so does any
  if (threads_fit<Tile256>(grouped_max_blocks(R, E, 32) * ceil_div(Fw, 32))) return true;
  bool ok = true;
  for (bool keep : {false, true})
    with_gated_tile(R, E, Fw, K, keep, [&](auto s) {
      using S = decltype(s);
      ok = ok && threads_fit<S>(grouped_max_blocks(R, E, S::BM) * ceil_div(Fw, kGatedCols<S>));
    });
  return ok;
}

bool gated_bwd_grid_fits(int64_t R, int64_t E, int64_t Fw, int64_t H) {
  if (threads_fit<Tile256>(grouped_max_blocks(R, E, 32) * ceil_div(Fw, 64))) return true;
  bool ok = true;
  with_gated_bwd_tile(R, E, Fw, H, [&](auto s) {
    using S = decltype(s);
    ok = threads_fit<S>(grouped_max_blocks(R, E, S::BM) * ceil_div(Fw, S::BN));
  });
  return ok;
}

HeadDxPlan head_dx_plan(int64_t T, int64_t H, int64_t cols) {
  struct Side {
    int side, bm, bn, per_cu;
    double ends, stage;
  };
  static constexpr Side kSides[] = {{256, 256, 256, 1, 9.0, 1.4},
                                    {128, 128, 128, 2, 4.0, 1.05},
                                    {64, 64, 64, 3, 3.0, 0.6},
                                    {32, 32, 128, 2, 2.5, 0.6}};
  const int64_t stages = ceil_div(cols, kStageK);
  HeadDxPlan best = {256, 1, stages * kStageK};
  double best_us = 1e300;
  for (const Side& s : kSides) {
    const int64_t tiles = ceil_div(T, s.bm) * ceil_div(H, s.bn), slots = kGroupedCus * s.per_cu;
    // one part, or what fills one to six rounds, of at least four stages each
    for (int rounds = 0; rounds <= 6; ++rounds) {
      const int64_t asked = std::min(std::max<int64_t>(1, rounds * slots / tiles), ceil_div(stages, 4));
      const int64_t each = ceil_div(stages, asked), p = ceil_div(stages, each);
      double us = (double)ceil_div(tiles * p, slots) * (s.ends + (double)each * s.stage);
      // weights read once, and once more for every further row of tiles
      us = std::max(us, (double)cols * H * 2e-6 * (0.2 + 0.1 * (double)(ceil_div(T, s.bm) - 1)));
      us += p > 1 ? 3.0 + (double)p * T * H * 8e-6 * 0.22 : 0.0;
      if (us < best_us) {
        best_us = us;
        best = {s.side, (int)p, each * kStageK};
      }
    }
  }
  return best;
}

HeadLayout head_layout(int64_t T, int64_t V, int64_t H) {
  HeadLayout L;
  if (head_is_narrow(T, V, H))
    L.slots = ceil_div(V, kNarrowLogits);
  else
    with_head_tile(T, V, H, false, [&](auto s) { L.slots = head_slots<decltype(s)>(V); });
  L.at_target = ((size_t)L.slots * (size_t)T * 8 + 255) & ~size_t(255);
  L.total = L.at_target + (((size_t)T * 4 + 255) & ~size_t(255));
  return L;
}

HeadBwdLayout head_bwd_layout(int64_t T, int64_t V, int64_t H) {
  HeadBwdLayout L;
  const int64_t column = 2 * std::max<int64_t>(T, 1);   // bytes of dz
  const int64_t most = std::max({kHeadLeastCols, kHeadPieceBytes / column / 256 * 256,
                                 std::min(kHeadPieceCols, kHeadMostBytes / column / 256 * 256)});
  L.pieces = ceil_div(V, most);
  L.cols = L.pieces == 1 ? V : ceil_div(ceil_div(V, L.pieces), 256) * 256;
  L.pieces = ceil_div(V, L.cols);
  L.pitch = ceil_div(L.cols, kStageK) * kStageK;
  L.dx = head_dx_plan(T, H, L.cols);
  auto whole = [](size_t bytes) { return (bytes + 255) & ~size_t(255); };
  L.c = whole((size_t)T * (size_t)L.pitch * 2);
  L.xc = L.c + whole((size_t)T * 8);
  L.sums = L.xc + whole((size_t)T * (size_t)H * 2);
  L.total = L.sums + (L.direct() ? 0 : (size_t)L.dx.parts * (size_t)T * (size_t)H * 4);
  return L;
}

bool head_grid_fits(int64_t T, int64_t V, int64_t H) {
  // 64 x 128 tiles of 256 threads are the weight gradient's smallest; six rounds of parts are added to x's
  // (and one workgroup of 256 threads a token takes its scale)
  if (T >= (int64_t(1) << 24) || !threads_fit<Tile256>((ceil_div(V, 64) + 7) * (ceil_div(H, 128) + 7)) ||
      ceil_div(T, 32) * ceil_div(H, 64) >= (int64_t(1) << 22))
    return false;
  if (threads_fit<Tile256>(ceil_div(T, 32) * ceil_div(V, 64))) return true;   // the narrowest tiles' launch
  bool ok = true;
  for (bool store : {false, true})
    with_head_tile(T, V, H, store, [&](auto s) {
      using S = decltype(s);
      ok = ok && threads_fit<S>(ceil_div(T, S::BM) * ceil_div(V, S::BN));
    });
  return ok;
}

}  // namespace beam
