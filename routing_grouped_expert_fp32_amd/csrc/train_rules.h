// Host-side rules of the training operators (gfx950): tile shapes and their choice, the deal of tiles to
// workgroups and XCDs, launch and workspace sizes. Plain C++, as host_rules.cpp, so that they also
// build without the GPU compiler (sanitizer checks); the kernels share the constants and, being
// constexpr, the deals.
#pragma once

#include <algorithm>
#include <cmath>

#include "common.h"

namespace beam {

// Workgroup tile of BM x BN, WM x WN waves; LDS rings of AST stages of the A operand and BST of B
// (AST <= BST: B is the one that streams from HBM, A's rows are shared by neighbouring tiles), of kStageK
// values of k each.
// Row sub-tiles (16 rows) are dealt to the wave rows in turn, so that a partly filled tile loads them
// alike.
constexpr int kStageK = 64;
template <int BM_, int BN_, int WM_, int WN_, int AST_, int BST_>
struct TileShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, AST = AST_, BST = BST_;
  static_assert(2 <= AST && AST <= BST, "ring depths");
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int FM = BM / 16 / WM, FN = BN / 16 / WN;   // 16 x 16 sub-tiles of a wave
  static constexpr int kABytes = BM * 2 * kStageK, kBBytes = BN * 2 * kStageK;
  static constexpr int kLdsBytes = AST * kABytes + BST * kBBytes;
  static_assert(kLdsBytes <= 160 * 1024, "LDS budget");
  static_assert(FM * 16 * WM == BM && FN * 16 * WN == BN, "whole sub-tiles");
  // sub-tile i of wave row wm
  static constexpr int row_tile(int wm, int i) { return wm + WM * i; }
};

// Tile v of `total` for workgroup `wg` of a grid of 8 ceil(total / 8), one run of tiles per XCD.
constexpr int xcd_tile(int wg, int total) {
  const int per = (total + 7) >> 3, local = wg >> 3;
  const int v = (wg & 7) * per + local;
  return local < per && v < total ? v : -1;
}
inline int64_t xcd_workgroups(int64_t tiles) { return 8 * ceil_div(tiles, 8); }

// The same where tiles 256 columns wide have a CU each: a last round of at most half an XCD's CUs would
// leave the others idle, so its tiles are split into two column halves (`half` 0 or 1, else -1),
// which take about 0.6 of a tile's time. Two and a half rounds of 320 x 256 tiles: 467 us as three,
// 447 with halves.
constexpr int kXcdCus = 32;
template <class S>
using HalfTile = TileShape<S::BM, S::BN / 2, S::WM, S::WN, S::AST, S::BST>;
template <class S>
constexpr bool kHalves = S::BN == 256 && S::kLdsBytes > 80 * 1024;
template <class S>
constexpr int xcd_tile_halves(int wg, int total, int& half) {
  const int per = (total + 7) >> 3, first = (wg & 7) * per;
  const int mine = std::min(per, total - first);   // tiles of this XCD
  int local = wg >> 3;
  half = -1;
  if constexpr (kHalves<S>) {
    const int tail = mine % kXcdCus, whole = mine - tail;
    if (mine > 0 && tail <= kXcdCus / 2 && local >= whole) {
      half = (local - whole) & 1;
      local = whole + ((local - whole) >> 1);
    }
  }
  return local < mine ? first + local : -1;
}
// The same where tiles are of unequal height in runs (an expert's blocks are alike, another's are not):
// an XCD takes every eighth run of 32 tiles instead of one eighth of them all, so that none has the tall ones
// alone; the tiles behind the last 256 are cut into eight runs as above.
template <class S>
constexpr int xcd_tile_dealt(int wg, int total, int& half) {
  const int rounds = total / (8 * kXcdCus), whole = rounds * kXcdCus;
  const int xcd = wg & 7, local = wg >> 3;
  half = -1;
  if (local < whole) return (local / kXcdCus * 8 + xcd) * kXcdCus + local % kXcdCus;
  // the rest of an XCD's tiles begins where its CUs get free: fewer than 32, as a tail above
  const int t = xcd_tile_halves<S>((local - whole) << 3 | xcd, total - 8 * whole, half);
  return t < 0 ? -1 : 8 * whole + t;
}
template <class S>
int64_t xcd_workgroups_halves(int64_t tiles) {
  return 8 * (ceil_div(tiles, 8) + (kHalves<S> ? kXcdCus / 2 : 0));
}

// ---- products grouped by expert ----
// Blocks of BM rows that n rows make (unsigned: n + BM may pass 2^31).
template <int BM>
constexpr int blocks_of(int n) {
  return (int)(((unsigned)n + (BM - 1)) / BM);
}

// An expert's n rows in blocks_of(n) blocks of about the same height, counted in units of 64 rows (what
// a tile's bodies tell apart): 655 rows as 256 + 256 + 143 cost less than as 320 + 320 + 15, whose
// last block would read all the weights for one body's work.
template <int BM>
constexpr void block_rows(int n, int n_blocks, int i, int& first, int& rows) {
  constexpr int kUnit = BM % 64 == 0 ? 64 : BM;
  const int units = blocks_of<kUnit>(n), each = units / n_blocks, more = units % n_blocks;
  first = kUnit * (i * each + std::min(i, more));
  rows = std::min(kUnit * (each + (i < more ? 1 : 0)), n - first);
}

// Tile v = b n_ctiles + .. of a deal of all blocks' column tiles, where block b is block in_expert of an
// expert's n_blocks, falls on block `block` of that expert and column tile `ctile`: an expert's blocks
// go in groups of kTileGroup, column-tile major inside a group, so that the blocks that read one weight
// tile run side by side.
constexpr int kTileGroup = 4;
constexpr void group_tile(int v, int b, int in_expert, int n_blocks, int n_ctiles, int& block,
                          int& ctile) {
  const int g0 = in_expert - in_expert % kTileGroup;
  const int sz = std::min(kTileGroup, n_blocks - g0);
  const int at = v - (b - (in_expert - g0)) * n_ctiles;   // tile within the group
  block = g0 + at % sz;
  ctile = at / sz;
}

// Tile t of one matrix, in bands of kTileGroup tile rows, column by column.
constexpr void band_tile(int t, int n_mtiles, int n_ctiles, int& mtile, int& ctile) {
  const int m0 = t / (kTileGroup * n_ctiles) * kTileGroup;
  const int sz = std::min(kTileGroup, n_mtiles - m0), at = t - m0 * n_ctiles;
  mtile = m0 + at % sz;
  ctile = at / sz;
}

// Weight gradient: tile t of workgroup `wg` among the `per` of one matrix, and `pos`, the matrix's position
// among the E (false: no tile), for a grid of dw_workgroups(per, E): each matrix's tiles in 8 runs, one
// an XCD.
constexpr bool dw_tile(unsigned wg, int per, int E, int& pos, int& t) {
  const int run = (per + 7) >> 3, local = (int)(wg >> 3);
  t = (int)(wg & 7) * run + local % run;
  pos = local / run;
  return pos < E && t < per;
}
inline int64_t dw_workgroups(int64_t per, int64_t E) { return 8 * E * ceil_div(per, 8); }

// The tile of a call is the one that a model of its time puts first; the experts' own row counts are on
// the device, so it goes by their mean. Per tile shape, in us, fitted together for the order of the tiles
// of some 400 calls (between one row and 65536, one expert and 256, widths of 128 to 8192, each measured
// with every tile). They give the time of calls that memory or latency bounds; where operations do, only
// the order of the tiles: a 320 x 256 tile's stage takes 1.94 us on this card, not 1.0, and 65536 rows
// of one expert, 5120 x 5120, 2.6 ms, not the model's 1.5.
struct TileCost {
  double mb;      // a megabyte from or to HBM (small tiles keep more loads in flight)
  double l2_mb;   // a megabyte of operands that other tiles read too
  double ends;    // a tile's start and end
  double stage;   // 64 values of its contraction, as far as other tiles' memory time does not hide them
  double alone;   // the same on a CU that runs no other tile
};
// Workgroups of a shape that the GPU holds at once (the LDS rings decide).
constexpr int kGroupedCus = 256;
template <class S>
constexpr int kSlots = kGroupedCus * (160 * 1024 / S::kLdsBytes);

// Calls f with the candidate for which us(candidate) is least.
template <class Us, class F, class... S>
void with_least(Us&& us, F&& f, S... tiles) {
  const double t[] = {us(tiles)...};
  const int pick = (int)(std::min_element(t, t + sizeof...(S)) - t);
  int i = 0;
  ((i++ == pick ? f(tiles) : void()), ...);
}

// Forward and input gradient. Measured (us, forward, bf16; the last columns with few columns and
// many rows, 40 experts of 632 x 1824 and 27 of 616 x 592):
//                        32 experts of 5120 x 5120, rows each          467    322
//                        64    110    156    219    256    375    656   rows   rows
//    32 x 128  (4, 4)   449    572    882   1084   1283   1779   3067    106    24
//    64 x 64   (3, 3)   420    516    652    788    969   1379   2286     91    21
//   128 x 128  (2, 2)   338    360    462    526    631    771   1339     60    15
//   128 x 256  (2, 3)   300    318    438    478    570    741   1263     67    16
//   192 x 256  (2, 3)   307    312    339    494    551    687   1119     69    21
//   256 x 256  (2, 3)   324    324    350    403    505    651   1050     57    17
//   320 x 256  (2, 2)   374    362    380    408    451    676    995     55    19
// Few rows: narrow tiles, many workgroups streaming weights. More: one block an expert if it can be, as
// every further block reads the weights again (rows spread by about the square root of their mean:
// 2.5 of it are allowed for); the B operand's third stage covers their latency while LDS lasts. Fewer
// tiles than CUs and a long contraction: 32 x 64 tiles with twelve stages (3 experts of 2 rows, 2232 x
// 4464: 24 us, 64 x 64 29, 32 x 128 39).
// Taken by this rule, the calls it was fitted to take 7% more than each one's best tile.
using TileStream = TileShape<32, 128, 1, 4, 4, 4>;
using TileLone = TileShape<32, 64, 1, 4, 12, 12>;
using Tile64 = TileShape<64, 64, 1, 2, 3, 3>;
using TilePair = TileShape<128, 128, 2, 2, 2, 2>;
using Tile128 = TileShape<128, 256, 2, 4, 2, 3>;
using Tile192 = TileShape<192, 256, 2, 4, 2, 3>;
using Tile256Deep = TileShape<256, 256, 2, 4, 2, 3>;
using Tile320 = TileShape<320, 256, 2, 4, 2, 2>;
constexpr TileCost rows_cost(TileStream) { return {.172, .1, 1.8, .41, 0.}; }
constexpr TileCost rows_cost(TileLone) { return {.21, .1, 1.7, .25, 0.}; }
constexpr TileCost rows_cost(Tile64) { return {.228, .1, 2.3, .34, 0.}; }
constexpr TileCost rows_cost(TilePair) { return {.240, .1, 1.7, .82, 0.}; }
constexpr TileCost rows_cost(Tile128) { return {.215, .1, 3.2, .50, 0.}; }
constexpr TileCost rows_cost(Tile192) { return {.235, .1, 3.2, .59, 0.}; }
constexpr TileCost rows_cost(Tile256Deep) { return {.25, .1, 2.4, .83, 0.}; }
constexpr TileCost rows_cost(Tile320) { return {.28, .1, 2.3, 1.0, 0.}; }

// A call of R rows, E experts, contraction Kc, whose tiles cover No columns of weights and move `mb`
// megabytes, of them w_mb of weights, with tile shape S.
struct RowsCall {
  double full, mean, w_mb, mb, stages;
  int64_t E, No;
  RowsCall(int64_t R, int64_t E_, int64_t No_, int64_t Kc, double out_mb)
      : full((double)std::min(R, E_)), mean((double)R / full), w_mb(full * No_ * Kc * 2e-6),
        mb(w_mb + R * Kc * 2e-6 + out_mb), stages((double)ceil_div(Kc, 64)), E(E_), No(No_) {}
  template <class S>
  double us(S s) const {
    const TileCost c = rows_cost(s);
    double blocks = std::ceil(mean / S::BM);   // of an expert
    if (E > 1)
      blocks = mean + 2.5 * std::sqrt(mean) <= S::BM ? 1.0 : std::max(1.0, mean / S::BM + 0.5);
    const double rounds = std::ceil(full * blocks * ceil_div(No, S::BN) / kSlots<S> - 1e-9);
    return std::max(4.3 + rounds * (c.ends + stages * c.stage),
                    mb * c.mb + w_mb * (blocks - 1.0) * c.l2_mb);
  }
};

template <class F>
void with_rows_tile(int64_t R, int64_t E, int64_t No, int64_t Kc, bool out_bf16, F&& f) {
  const RowsCall call(R, E, No, Kc, R * (No * (out_bf16 ? 2e-6 : 4e-6)));
  with_least([&](auto s) { return call.us(s); }, f, TileStream{}, TileLone{}, Tile64{}, TilePair{}, Tile128{},
             Tile192{}, Tile256Deep{}, Tile320{});
}

// Weight gradient. Measured (us) with 256 x 256, 128 x 128 and 64 x 128 tiles: 32 experts of 1024 rows,
// two with 40% of them, 5120 x 5120 fp32, 1783, 2127, 2783; 22 of 42 rows, 2536 x 4432 bf16, 132, 151,
// 169; 24 of 33 rows, 1656 x 344 fp32, 21, 15, 15. A launch is no shorter than the tiles of its longest
// expert, which is taken to have four times the mean's rows: 24 experts, one with 7500 of 18850 rows,
// 1016 x 392, 166, 98, 86. Taken by this rule, the calls it was fitted to take 3% more than each
// one's best tile.
using Tile256 = TileShape<256, 256, 2, 4, 2, 2>;
using TileHalfPair = TileShape<64, 128, 1, 4, 2, 2>;
constexpr TileCost dw_cost(Tile256) { return {.205, .10, 3.9, 2.2, 1.4}; }
constexpr TileCost dw_cost(TilePair) { return {.20, .06, 2.2, 1.1, .8}; }
constexpr TileCost dw_cost(TileHalfPair) { return {.20, .05, 1.8, 1.0, .7}; }

template <class F>
void with_dw_tile(int64_t R, int64_t E, int64_t N, int64_t K, bool out_bf16, F&& f) {
  const double mean = (double)R / E;
  const double stages = E == 1 ? (double)std::max<int64_t>(1, ceil_div(R, 64))
                               : std::max(1.0, mean > 32.0 ? mean / 64 + 0.5 : 1.0);
  const double longest = E == 1 ? stages : 4.0 * stages;
  const double mb = (double)E * N * K * (out_bf16 ? 2e-6 : 4e-6) + R * (N + K) * 2e-6;
  auto us = [&](auto s) {
    using S = decltype(s);
    const TileCost c = dw_cost(s);
    const double tiles = (double)ceil_div(N, S::BM) * ceil_div(K, S::BN);
    const double rounds = std::ceil(E * tiles / kSlots<S> - 1e-9);
    return std::max({5.3 + rounds * (c.ends + stages * c.stage), 5.3 + c.ends + longest * c.alone,
                     mb * c.mb + tiles * R * (S::BM + S::BN) * 2e-6 * c.l2_mb});
  };
  with_least(us, f, Tile256{}, TilePair{}, TileHalfPair{});
}

// Blocks that R rows of E experts can make.
inline int64_t grouped_max_blocks(int64_t R, int64_t E, int64_t bm) { return R / bm + std::min(R, E) + 1; }

// A launch counts its threads in 32 bits.
template <class S>
bool threads_fit(int64_t tiles) {
  return (tiles + 8 * kXcdCus) * S::kThreads < (int64_t(1) << 32);
}

// ---- gradient of the boundary ----
// Threads of a workgroup and workgroups of the first launch (two a CU at 256 threads) for rows of H.
inline int boundary_bwd_threads(int H) { return H <= 5 * 1024 ? 256 : H <= 5 * 2048 ? 512 : 1024; }

// ---- orthogonalised update ----
constexpr int kNormParts = 512;         // most partial sums of squares of a matrix
inline bool ns_is_small(int m, int n) { return m <= 64 ? n <= 1024 : m <= 128 && n <= 384; }
using NsTile256 = TileShape<256, 256, 2, 4, 2, 2>;
using NsTile128 = TileShape<128, 128, 2, 2, 2, 2>;
using NsTile64 = TileShape<64, 64, 1, 2, 3, 3>;
constexpr int kNsCus = 256;

inline int64_t ns_triangle(int64_t n) { return n * (n + 1) / 2; }

// Time in us of a launch of `count` tiles of a side, `stages` of 64 values of the contraction each: full
// rounds of the workgroups that the GPU holds (3, 2, 1 a CU), then the rest. A tile's ends and its
// stage were measured on one to eight matrices of 130 to 5120 rows; against the tile it puts first, us a
// launch: A of 4 matrices 2000 x 2500 256 wide, 128 +19, 64 +40; of 3 1000 x 3000 64 wide, 128 +11, 256
// +44; of 2560 x 5120 128 wide, 256 +65, of 8 of them 256 wide, 128 +33; the update of 3 632 x 1656
// 128 wide, 64 +5, 256 +5, of 2 603 x 1532 64 wide, 128 +3, 256 +10.
inline double ns_launch_us(int side, int64_t count, double stages, bool update) {
  const double ends = side == 64 ? 2.5 : side == 128 ? 3.0 : update ? 5.0 : 9.0;
  const int64_t slots = kNsCus * (side == 64 ? 3 : side == 128 ? 2 : 1);
  auto round = [&](int64_t wgs) {
    const int64_t each = ceil_div(wgs, kNsCus);   // workgroups a CU
    const double stage = side == 64    ? each == 1 ? .36 : each == 2 ? .46 : .6
                         : side == 128 ? each == 1 ? .65 : 1.05
                         : update      ? .9 + .8 * (double)wgs / kNsCus
                                       : 1.4;
    return ends + stages * stage;
  };
  const int64_t rest = count % slots;
  double us = (double)(count / slots) * round(slots);
  if (rest > 0)   // an update's last wide tiles are split where they leave half the CUs idle
    us += (update && side == 256 && rest <= kNsCus / 2 ? 0.7 : 1.0) * round(rest);
  return us;
}

// Calls f with the tile that is fastest; `count` is the tiles' number for a side.
template <class Count, class F>
void with_ns_tile(bool update, int contraction, Count&& count, F&& f) {
  const double stages = (double)ceil_div(contraction, 64);
  auto us = [&](int side) { return ns_launch_us(side, count(side), stages, update); };
  const double t64 = us(64), t128 = us(128), t256 = us(256);
  if (t256 < t128 && t256 < t64)
    f(NsTile256{});
  else if (t128 < t64)
    f(NsTile128{});
  else
    f(NsTile64{});
}

// Parts of the contraction of A's products: more than one, of at least four stages each and at most two
// workgroups of 64 x 64 tiles a CU, where that saves more than the launch that adds them takes
// (3.5 us and 1 a megabyte of sums). 256 x 5120 update: 125 us, in one part 205; 3 of 632 x 1656: one
// part saves 22 us of 222 over three.
struct GramParts {
  int parts, kp;   // kp: values of k of a part, whole stages
};
inline GramParts gram_parts(int64_t n_mats, int m, int k) {
  const int64_t tiles = n_mats * ns_triangle(ceil_div(m, 64)), stages = ceil_div(k, 64);
  const int64_t most = std::min(2 * kNsCus / tiles, ceil_div(k, 256));
  double best = 1e300;
  for (int side : {64, 128, 256})
    best = std::min(best, ns_launch_us(side, n_mats * ns_triangle(ceil_div(m, side)), (double)stages, false));
  int parts = 1;
  for (int64_t p = 2; p <= most; ++p) {
    const double us = ns_launch_us(64, tiles * p, (double)ceil_div(stages, p), false) + 3.5 +
                      (double)(tiles * p) * (64 * 64 * 4 * 1e-6);
    if (us < best) {
      best = us;
      parts = (int)p;
    }
  }
  const int kp = (int)ceil_div(ceil_div(k, parts), 64) * 64;
  return {(int)ceil_div(k, kp), kp};   // rounding to stages can leave fewer parts
}

// Workgroups of a matrix's partial sums of squares.
inline int ns_norm_parts(int64_t count) { return (int)std::min<int64_t>(kNormParts, ceil_div(count, 8192)); }

}  // namespace beam
