// Launch bounds and workspace sizes of the training operators (see train_rules.h).
#include "train_rules.h"

namespace beam {

bool grouped_grid_fits(int64_t R, int64_t E, int64_t N, int64_t K) {
  // 64 x 128 tiles of 256 threads are the weight gradient's smallest
  bool ok = threads_fit<Tile256>(E * (ceil_div(N, 128) + 7) * (ceil_div(K, 128) + 7));
  for (int64_t width : {N, K}) {
    // the narrowest tiles' launch fits: so does any
    if (threads_fit<Tile256>(grouped_max_blocks(R, E, 32) * ceil_div(width, 64))) continue;
    for (bool out_bf16 : {false, true})
      with_rows_tile(R, E, width, N + K - width, out_bf16, [&](auto s) {
        using S = decltype(s);
        ok = ok && threads_fit<S>(grouped_max_blocks(R, E, S::BM) * ceil_div(width, S::BN));
      });
  }
  return ok;
}

int boundary_bwd_parts(int64_t T, int H) {
  return (int)std::min<int64_t>(T, boundary_bwd_threads(H) == 256 ? 512 : 256);
}

NsLayout ns_layout(int64_t n_mats, int rows, int cols) {
  NsLayout L;
  L.tall = rows > cols;
  L.m = std::min(rows, cols);
  L.n = std::max(rows, cols);
  L.mp = (L.m + 7) / 8 * 8;
  L.ld = (L.n + 7) / 8 * 8;
  if (ns_is_small(L.m, L.n)) {   // uses none
    L.total = 16;
    return L;
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) & ~size_t(255);
    return o;
  };
  const size_t x = 2 * (size_t)n_mats * L.m * L.ld, a = 2 * (size_t)n_mats * L.m * L.mp;
  L.parts = take(sizeof(double) * kNormParts * (size_t)n_mats);
  L.units = take(sizeof(float) * kNsMaxSteps * (size_t)n_mats);
  L.hi[0] = take(x);
  L.hi[1] = take(x);
  L.lo = take(x);
  L.gram = take(a);
  L.poly = take(a);
  const int np = gram_parts(n_mats, L.m, L.n).parts;
  if (np > 1)
    L.sums = take(sizeof(float) * 64 * 64 * (size_t)(np * n_mats * ns_triangle(ceil_div(L.m, 64))));
  L.total = off;
  return L;
}

bool ns_grid_fits(int64_t n_mats, int rows, int cols) {
  // 64 x 64 tiles of 128 threads; wider ones have fewer of both together. A launch counts its threads
  // in 32 bits.
  const int64_t mt = ceil_div(std::min(rows, cols), 64), ct = ceil_div(std::max(rows, cols), 64);
  return n_mats <= 65535 &&
         (n_mats * mt * std::max(ct, (mt + 1) / 2) + 8 * kXcdCus) * 512 < (int64_t(1) << 32);
}

}  // namespace beam
