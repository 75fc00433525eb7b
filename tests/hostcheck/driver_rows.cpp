// The blocks of rows and tiles that the products grouped by expert find on the device (row_blocks.h), run on the
// CPU: 64 lanes in turn, their exchanges handed on when all have reached them. For lists of offsets of every kind
// each workgroup of a launch is asked for its tile. Every row of every expert and every column has one tile
// (or the two halves of one), none is outside, and what the tile's loads, stores and partial sums reach lies inside
// the arrays.
#include <ucontext.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <numeric>
#include <random>
#include <type_traits>
#include <vector>

// ---- 64 lanes ----
namespace lanes {
constexpr int kLanes = 64;
ucontext_t g_main, g_ctx[kLanes];
std::vector<char> g_stack(kLanes * 65536);
uint64_t g_slot[2][kLanes];
int g_now, g_turn[kLanes];
bool g_done[kLanes];
void (*g_body)(int);

// Hands `v` in and returns when every lane has: the slots of one exchange are read before those of the next but
// one are written.
const uint64_t* exchange(uint64_t v) {
  const int me = g_now, side = g_turn[me]++ & 1;
  g_slot[side][me] = v;
  swapcontext(&g_ctx[me], &g_main);
  return g_slot[side];
}
void enter(int lane) {
  g_body(lane);
  g_done[lane] = true;
  swapcontext(&g_ctx[lane], &g_main);
}
void run(void (*body)(int)) {
  g_body = body;
  for (int l = 0; l < kLanes; ++l) {
    getcontext(&g_ctx[l]);
    g_ctx[l].uc_stack.ss_sp = &g_stack[l * 65536];
    g_ctx[l].uc_stack.ss_size = 65536;
    g_ctx[l].uc_link = nullptr;
    g_turn[l] = 0;
    g_done[l] = false;
    makecontext(&g_ctx[l], (void (*)())enter, 1, l);
  }
  for (int left = kLanes; left > 0;) {
    int ended = 0;
    for (g_now = 0; g_now < kLanes; ++g_now) {
      if (g_done[g_now]) {
        std::fprintf(stderr, "a lane waits for one that has returned\n");
        std::abort();
      }
      swapcontext(&g_main, &g_ctx[g_now]);
      ended += g_done[g_now];
    }
    if (ended != 0 && ended != kLanes) {
      std::fprintf(stderr, "lanes part at an exchange\n");
      std::abort();
    }
    left -= ended;
  }
}
}  // namespace lanes

#define __device__
#define __forceinline__ inline
struct {
  int x;
} blockIdx;
using std::max;
using std::min;
static int lane_now() { return lanes::g_now; }
static int __shfl_up(int v, int d) {
  const int l = lane_now();
  const uint64_t* s = lanes::exchange((uint32_t)v);
  return (int)(uint32_t)s[l >= d ? l - d : l];
}
static int __shfl(int v, int src) { return (int)(uint32_t)lanes::exchange((uint32_t)v)[src & 63]; }
static uint64_t __ballot(bool b) {
  const uint64_t* s = lanes::exchange(b);
  uint64_t m = 0;
  for (int l = 0; l < 64; ++l) m |= s[l] << l;
  return m;
}
static int __ffsll(unsigned long long v) { return __builtin_ffsll((long long)v); }
static int first_lane(int v) { return (int)(uint32_t)lanes::exchange((uint32_t)v)[0]; }
#define __builtin_amdgcn_readfirstlane first_lane

#include "../../routing_grouped_expert_fp32_amd/csrc/row_blocks.h"
#include "../../routing_grouped_expert_fp32_amd/csrc/step_rules.h"

namespace {

using namespace beam;

long g_checks = 0;
int g_fail = 0;
void expect(bool ok, const char* what, long a = 0, long b = 0, long c = 0, long d = 0) {
  ++g_checks;
  if (!ok && ++g_fail <= 20) std::fprintf(stderr, "FAIL: %s (%ld, %ld, %ld, %ld)\n", what, a, b, c, d);
}

std::mt19937 g_rng(3);
int pick(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(g_rng); }

// ---- one workgroup's tile, by all lanes ----
struct Ask {
  const int32_t* offsets;
  int R, E, n_ctiles, max_blocks;
  bool found[64];
  RowBlock blk[64];
  int ctile[64], half[64];
} g_ask;
template <class S, bool DEALT>
void ask(int lane) {
  g_ask.found[lane] = row_block_tile<S, DEALT>(g_ask.offsets, g_ask.R, g_ask.E, g_ask.n_ctiles, g_ask.max_blocks, lane,
                                              g_ask.blk[lane], g_ask.ctile[lane], g_ask.half[lane]);
}

// The operands and results of a tile of the gated gradient or product: rows row0 .. +rows, columns col0 .. of F.
template <class S>
void reaches(const RowBlock& b, int col0, int R, int E, int64_t F, int64_t K, int part_cols) {
  const int64_t ld = 2 * K, h_ld = 2 * F, gu_ld = 4 * F, rows = b.rows;
  const int64_t cols = std::min<int64_t>(F - col0, S::BN);
  expect(cols > 0 && rows <= S::BM, "columns of a tile", col0, F, rows);
  // what a descriptor spans, from the tile's first value on, and its end in the array
  expect((b.row0 + rows) * ld <= R * ld && rows * ld < (int64_t(1) << 31), "rows of x and dy", b.row0, rows, R);
  expect(b.row0 * gu_ld + col0 * 2 + (rows - 1) * gu_ld + h_ld + cols * 2 <= R * gu_ld, "gate and up", b.row0, rows, col0);
  expect((rows - 1) * gu_ld + h_ld + cols * 2 < (int64_t(1) << 31), "a tile's gate and up in 31 bits", rows, F);
  expect(b.row0 * h_ld + col0 * 2 + (rows - 1) * h_ld + cols * 2 <= R * h_ld, "activation", b.row0, rows, col0);
  // the gradient's weights, stage by stage: 64 stored rows from k0 on, the last one to its own end
  for (int64_t k0 = 0; k0 < K; k0 += kStageK) {
    const int64_t n = std::min<int64_t>(K - k0, kStageK);
    expect(b.e * K * h_ld + col0 * 2 + k0 * h_ld + (n - 1) * h_ld + (F - col0) * 2 <= E * K * h_ld, "weights of a stage", b.e, k0);
  }
  // the products' weights: rows from col0 on to the end of the expert's up rows
  expect((b.e * 2 * F + col0) * ld + (2 * F - col0) * ld <= E * 2 * F * ld, "gate and up rows", b.e, col0);
  // partial sums of the scales' gradient: of each wave's columns, in the place of their first part, zeros in the others
  std::vector<int> written((size_t)gated_scale_parts(F), 0);
  for (int wn = 0; wn < S::WN; ++wn) {
    const int own = (col0 + wn * S::FN * 16) / part_cols, n_own = S::FN * 16 / part_cols;
    expect(n_own >= 1 && n_own <= 2 * S::FN && (col0 + wn * S::FN * 16) % part_cols == 0, "parts of a wave", own, n_own);
    for (int k = 0; k < n_own; ++k)
      if ((int64_t)(own + k) * part_cols < F) {
        const int64_t at = (int64_t)(own + k) * R + b.row0 + rows - 1;
        expect(at < gated_scale_parts(F) * R, "a part", own + k, at);
        if (own + k < (int)written.size()) ++written[own + k];
      }
  }
  for (int p = 0; p < (int)written.size(); ++p) {   // each part of the tile's columns once
    const int64_t first = (int64_t)p * part_cols;
    expect(written[p] == (first < F && first >= col0 && first < col0 + S::BN), "a part written once", p, written[p]);
  }
}

template <class S, bool DEALT>
void launch(const std::vector<int32_t>& off, int R, int64_t F, int64_t K, bool in_order) {
  const int E = (int)off.size() - 1;
  const int64_t blocks = grouped_max_blocks(R, E, S::BM);
  g_ask.offsets = off.data();
  g_ask.R = R;
  g_ask.E = E;
  g_ask.n_ctiles = (int)ceil_div(F, S::BN);
  g_ask.max_blocks = (int)blocks;
  // rows x half columns of each tile
  std::vector<int> seen((size_t)R * g_ask.n_ctiles * 2, 0);
  const int64_t wgs = xcd_workgroups_halves<S>(blocks * g_ask.n_ctiles);
  for (int64_t wg = 0; wg < wgs; ++wg) {
    blockIdx.x = (int)wg;
    lanes::run(ask<S, DEALT>);
    const bool found = g_ask.found[0];
    const RowBlock b = g_ask.blk[0];
    const int ctile = g_ask.ctile[0], half = g_ask.half[0];
    for (int l = 1; l < 64; ++l) {
      expect(g_ask.found[l] == found, "lanes agree", wg, l);
      if (found) {
        const RowBlock& o = g_ask.blk[l];
        expect(o.e == b.e && o.row0 == b.row0 && o.rows == b.rows && g_ask.ctile[l] == ctile && g_ask.half[l] == half,
               "lanes agree on a tile", wg, l);
      }
    }
    if (!found) continue;
    expect(b.e >= 0 && b.e < E && b.row0 >= 0 && b.rows > 0 && b.rows <= S::BM && (int64_t)b.row0 + b.rows <= R, "a block of rows",
           b.e, b.row0, b.rows, R);
    expect(ctile >= 0 && ctile < g_ask.n_ctiles && half >= -1 && half <= 1 && (kHalves<S> || half < 0), "a tile's columns", ctile,
           half);
    if (g_fail > 0) continue;
    if (in_order) expect(b.row0 >= off[b.e] && b.row0 + b.rows <= off[b.e + 1], "rows of the expert", b.e, b.row0, b.rows);
    const int col0 = ctile * S::BN;
    if constexpr (kHalves<S>) {
      if (half >= 0) {
        const int c = col0 + half * (S::BN / 2);
        if (c < F) reaches<HalfTile<S>>(b, c, R, E, F, K, kScaleCols<S>);
      } else {
        reaches<S>(b, col0, R, E, F, K, kScaleCols<S>);
      }
    } else {
      reaches<S>(b, col0, R, E, F, K, kScaleCols<S>);
    }
    for (int r = b.row0; r < b.row0 + b.rows; ++r)
      for (int h = 0; h < 2; ++h)
        if (half < 0 || half == h) ++seen[((size_t)r * g_ask.n_ctiles + ctile) * 2 + h];
  }
  if (!in_order || g_fail > 0) return;
  for (int r = 0; r < R; ++r)
    for (int t = 0; t < g_ask.n_ctiles * 2; ++t)
      expect(seen[(size_t)r * g_ask.n_ctiles * 2 + t] == (r >= off[0] && r < off[E]), "a row's columns once", r, t, R, E);
}

// Both deals in turn, so that each shape sees either in about half of the lists.
int g_list = 0;
template <class... S>
void launches(const std::vector<int32_t>& off, int R, int64_t F, int64_t K, bool in_order) {
  ((++g_list & 1 ? launch<S, true>(off, R, F, K, in_order) : launch<S, false>(off, R, F, K, in_order)), ...);
  ++g_list;
}
void every_tile(const std::vector<int32_t>& off, int R, int64_t F, int64_t K, bool in_order = true) {
  launches<TileStream, TileLone, Tile64, TilePair, Tile128, Tile192, Tile256Deep, Tile320>(off, R, F, K, in_order);
}

std::vector<int32_t> offsets_of(const std::vector<int>& counts, int first) {
  std::vector<int32_t> off{first};
  for (int n : counts) off.push_back(off.back() + n);
  return off;
}

}  // namespace

int main() {
  // ordinary, empty, odd and skewed lists; rows before the first expert and behind the last
  const std::vector<std::vector<int>> lists = {
      {1}, {0}, {0, 0, 5}, {17, 33, 0, 15}, {257, 0, 300, 12}, {700}, {320, 321, 319, 64, 65, 63}, {0, 0, 0, 1000, 0},
  };
  for (const auto& l : lists)
    for (int first : {0, 3}) {
      const auto off = offsets_of(l, first);
      every_tile(off, std::max(1, off.back() + (first ? 4 : 0)), first ? 776 : 264, 136);
    }
  // many experts: several a lane, most of them empty
  std::vector<int> many(130, 0);
  many[0] = 2, many[64] = 70, many[65] = 1, many[129] = 333;
  every_tile(offsets_of(many, 0), offsets_of(many, 0).back(), 520, 72);
  // a skewed training batch at the model's sizes: two of 32 experts with 40% of the rows (the wide tiles, whole rounds
  // of them and halves behind)
  {
    const int R = 32768;
    std::vector<int> c(32, (int)(R * 0.6 / 30));
    c[5] = c[20] = (int)(R * 0.2);
    c[31] += R - std::accumulate(c.begin(), c.end(), 0);
    const auto off = offsets_of(c, 0);
    launch<Tile320, true>(off, R, 2560, 5120, true);
    launch<Tile256Deep, true>(off, R, 2560, 5120, true);
  }
  for (int i = 0; i < 5; ++i) {
    std::vector<int> c((size_t)pick(1, 80));
    for (int& n : c) n = pick(0, 3) == 0 ? 0 : pick(0, 9) == 0 ? pick(1, 900) : pick(1, 40);
    const int first = pick(0, 1) * pick(0, 9);
    const auto off = offsets_of(c, first);
    every_tile(off, std::max(1, off.back() + pick(0, 5)), 8 * pick(1, 50), 8 * pick(1, 40));
  }
  // offsets out of order: nothing outside the arrays, whatever they hold
  for (const auto& off : std::vector<std::vector<int32_t>>{
           {0, 60, -5, 50}, {50, 20, 30, 0}, {-9, -3, 2147483647, 7}, {2147483647, -2147483647 - 1, 0, 50}, {40, 40, 0, 90, 3, 50}})
    every_tile(off, 50, 392, 64, false);
  for (int i = 0; i < 4; ++i) {
    std::vector<int32_t> off((size_t)pick(2, 70));
    for (int32_t& o : off) o = pick(-50, 900);
    every_tile(off, 700, 8 * pick(1, 40), 64, false);
  }
  std::printf("hostcheck: %ld checks, %d failed\n", g_checks, g_fail);
  return g_fail ? 1 : 0;
}
