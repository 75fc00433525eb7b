// Matrix products grouped by expert with ragged row counts (gfx950), forward and both gradients, the
// training side of the expert GEMMs ([S] §Reinforcement learning in Miles: the routes are recorded
// once and the trainer recomputes the experts on them).
//
//   forward          Y[r]  = X[r] W[e]^T      rows x N,  contraction over K
//   input gradient   dX[r] = dY[r] W[e]       rows x K,  contraction over N
//   weight gradient  dW[e] = dY_e^T X_e       N x K,     contraction over the expert's rows
// offsets[e] .. offsets[e + 1] are expert e's rows. Every sum is one FP32 accumulation in k order,
// rounded once if the output is bf16.
//
// Forward and input gradient: a workgroup owns one block of an expert's rows and one column tile;
// each wave finds the block itself from the offsets by a scan over the experts (no table, no second
// launch, no host readback). Weight gradient: a workgroup owns a tile of one expert's matrix.
// Workgroup L runs on XCD L % 8, so the tiles are cut into 8 contiguous runs, one per XCD, whose
// neighbours share operands in that XCD's L2.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gemm_tile.h"

namespace beam {

// A block of rows of one expert, as found from the offsets.
struct RowBlock {
  int e;          // expert
  int row0;       // first row of the block (from find(): of the expert)
  int rows;       // rows in the block (from find(): of the expert)
  int in_expert;  // the block's index among the expert's blocks
  int n_blocks;   // the expert's blocks
};

__device__ __forceinline__ int clamped(int v, int lo, int hi) { return min(max(v, lo), hi); }

// Rows [begin, end) of expert e, clamped into [0, R) whatever the offsets hold.
__device__ __forceinline__ void expert_rows(const int32_t* __restrict__ off, int e, int R,
                                            int& begin, int& end) {
  begin = clamped(off[e], 0, R);
  end = clamped(off[e + 1], begin, R);
}

// Blocks of BM rows that n rows make (unsigned: n + BM may pass 2^31).
template <int BM>
__device__ __forceinline__ int blocks_of(int n) {
  return (int)(((unsigned)n + (BM - 1)) / BM);
}

// An expert's n rows in blocks_of(n) blocks of about the same height, counted in units of 64 rows (what
// a tile's bodies tell apart): 655 rows as 256 + 256 + 143 cost less than as 320 + 320 + 15, whose
// last block would read all the weights for one body's work.
template <int BM>
__device__ __forceinline__ void block_rows(int n, int n_blocks, int i, int& first, int& rows) {
  constexpr int kUnit = BM % 64 == 0 ? 64 : BM;
  const int units = blocks_of<kUnit>(n), each = units / n_blocks, more = units % n_blocks;
  first = kUnit * (i * each + min(i, more));
  rows = min(kUnit * (each + (i < more ? 1 : 0)), n - first);
}

// Blocks of at most BM rows of all experts in expert order: `total` of them; find(b) gives block b. Lane l
// counts the blocks of experts [l * per, (l + 1) * per); a wave scan orders the lanes.
template <int BM>
struct BlockScan {
  const int32_t* off;
  int E, R, per, lane, first, count, total;

  __device__ __forceinline__ void init(const int32_t* offsets, int n_experts, int n_rows, int ln) {
    off = offsets;
    E = n_experts;
    R = n_rows;
    lane = ln;
    per = (E + 63) >> 6;
    int c = 0;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < E) {
        int a, z;
        expert_rows(off, e, R, a, z);
        c += blocks_of<BM>(z - a);
      }
    }
    int incl = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
    first = incl - c;
    count = c;
    total = __builtin_amdgcn_readfirstlane(__shfl(incl, 63));
  }
  __device__ __forceinline__ RowBlock find(int b) const {   // b < total
    const uint64_t has = __ballot(b >= first && b < first + count);
    if (!has) return RowBlock{0, 0, 0, 0, 0};   // only offsets that are not in order
    const int src = __ffsll((unsigned long long)has) - 1;
    int left = b - __shfl(first, src);
    RowBlock r{0, 0, 0, 0, 0};
    for (int i = 0; i < per; ++i) {
      const int e = src * per + i;   // < E: the lane that holds block b has it
      if (e >= E) break;
      int a, z;
      expert_rows(off, e, R, a, z);
      const int n = blocks_of<BM>(z - a);
      if (left < n) {
        r = RowBlock{e, a, z - a, left, n};
        break;
      }
      left -= n;
    }
    r.e = __builtin_amdgcn_readfirstlane(r.e);
    r.row0 = __builtin_amdgcn_readfirstlane(r.row0);
    r.rows = __builtin_amdgcn_readfirstlane(r.rows);
    r.in_expert = __builtin_amdgcn_readfirstlane(r.in_expert);
    r.n_blocks = __builtin_amdgcn_readfirstlane(r.n_blocks);
    return r;
  }
};

constexpr int kTileGroup = 4;   // blocks of one expert walked together, column tile by column tile

// One tile: rows of `blk`, columns from col0 on.
template <class S, bool WCOL, bool OUT_BF16>
__device__ __forceinline__ void grouped_rows_tile(const unsigned char* __restrict__ a,
                                                  const unsigned char* __restrict__ w,
                                                  unsigned char* __restrict__ out,
                                                  const RowBlock& blk, int col0, int No, int Kc,
                                                  unsigned char* smem, int wave, int lane) {
  const int64_t wbytes = (int64_t)No * Kc * 2;
  const int64_t a_ld = (int64_t)Kc * 2;
  OperandLoader<S::BM, S::kWaves, false> la;
  OperandLoader<S::BN, S::kWaves, WCOL> lb;
  lb.stream = blk.n_blocks == 1;   // weights that no other block reads need not stay in L2
  la.init({a + (int64_t)blk.row0 * a_ld, a_ld, blk.rows, 0}, wave, lane);
  if constexpr (WCOL)
    lb.init({w + blk.e * wbytes + (int64_t)col0 * 2, (int64_t)No * 2, 0, (No - col0) * 2}, wave,
            lane);
  else
    lb.init({w + blk.e * wbytes + (int64_t)col0 * a_ld, a_ld, min(S::BN, No - col0), 0}, wave, lane);

  floatx4 acc[S::FM][S::FN];
  tile_zero<S>(acc);

  // sub-tiles of 16 rows are dealt to the wave rows in turn; a wave runs the body for the number it
  // has, in steps of two, so a partly filled block costs about its rows
  const int nsub = (blk.rows + 15) >> 4, wm = wave / S::WN;
  const int nv = (nsub - wm + S::WM - 1) / S::WM;   // wave-uniform; 0 where nsub <= wm
  auto body = [&](auto nv_tag) {
    constexpr int NV = decltype(nv_tag)::value;
    tile_kloop<S, false, WCOL, false, NV>(la, lb, Kc, smem, wave, lane, acc);
    constexpr int kSize = OUT_BF16 ? 2 : 4;
    tile_store<S, NV, OUT_BF16>(acc, out + ((int64_t)blk.row0 * No + col0) * kSize,
                                (int64_t)No * kSize, blk.rows, No - col0, smem, wave, lane);
  };
  if (S::FM > 8 && nv > 8)
    body(std::integral_constant<int, S::FM>{});
  else if (S::FM > 6 && nv > 6)
    body(std::integral_constant<int, S::FM < 8 ? S::FM : 8>{});
  else if (S::FM > 4 && nv > 4)
    body(std::integral_constant<int, S::FM < 6 ? S::FM : 6>{});
  else if (S::FM > 2 && nv > 2)
    body(std::integral_constant<int, S::FM < 4 ? S::FM : 4>{});
  else
    body(std::integral_constant<int, 2>{});
}

// out[row][0 .. No) = a[row][0 .. Kc) . w[e], w stored [No][Kc] (forward) or, WCOL, [Kc][No] (input
// gradient: the weight's rows run across the contraction).
template <class S, bool WCOL, bool OUT_BF16>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void grouped_rows_kernel(
    const unsigned char* __restrict__ a, const unsigned char* __restrict__ w,
    const int32_t* __restrict__ offsets, unsigned char* __restrict__ out, int R, int E, int No, int Kc,
    int n_ctiles, int max_blocks) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  BlockScan<S::BM> scan;
  scan.init(offsets, E, R, lane);
  // more blocks than the grid has come only from offsets that are not in order
  const int total = min(scan.total, max_blocks) * n_ctiles;
  int half;
  const int v = xcd_tile_halves<S>(blockIdx.x, total, half);
  if (v < 0) return;
  // an expert's blocks in groups of kTileGroup, column-tile major inside a group: the blocks that
  // read one weight tile run side by side
  RowBlock blk = scan.find(v / n_ctiles);
  if (blk.rows <= 0) return;
  int ctile;
  {
    const int g0 = blk.in_expert - blk.in_expert % kTileGroup;
    const int sz = min(kTileGroup, blk.n_blocks - g0);
    const int at = v - (v / n_ctiles - (blk.in_expert - g0)) * n_ctiles;   // tile within the group
    ctile = at / sz;
    int first, rows;
    block_rows<S::BM>(blk.rows, blk.n_blocks, g0 + at % sz, first, rows);
    blk.row0 += first;
    blk.rows = rows;
  }
  const int col0 = ctile * S::BN;
  if constexpr (kHalves<S>) {
    if (half >= 0) {
      if (col0 + half * (S::BN / 2) < No)
        grouped_rows_tile<HalfTile<S>, WCOL, OUT_BF16>(a, w, out, blk, col0 + half * (S::BN / 2), No,
                                                       Kc, smem, wave, lane);
      return;
    }
  }
  grouped_rows_tile<S, WCOL, OUT_BF16>(a, w, out, blk, col0, No, Kc, smem, wave, lane);
}

// Expert at position `pos` < E of the order in which those with more than 1.5 times the mean's rows come
// first, and its rows [begin, end).
__device__ __forceinline__ int heavy_first(const int32_t* __restrict__ off, int E, int R, int pos,
                                           int lane, int& begin, int& end) {
  const int heavy_rows = R / E + R / E / 2;
  int a0 = 0, z0 = 0;   // the first 64 experts' rows
  if (lane < E) expert_rows(off, lane, R, a0, z0);
#pragma unroll
  for (int light = 0; light < 2; ++light)
    for (int base = 0; base < E; base += 64) {
      const bool in = base + lane < E;
      int a = a0, z = z0;
      if (base > 0 && in) expert_rows(off, base + lane, R, a, z);
      const uint64_t mask = __ballot(in && (z - a > heavy_rows) != (bool)light);
      const int n = __popcll(mask);
      if (pos < n) {
        const bool mine = mask >> lane & 1 && __popcll(mask & ((uint64_t(1) << lane) - 1)) == pos;
        const int at = __ffsll((unsigned long long)__ballot(mine)) - 1;
        begin = uniform(__shfl(a, at));
        end = uniform(__shfl(z, at));
        return uniform(base + at);
      }
      pos -= n;
    }
  begin = end = 0;
  return -1;
}

// dw[e] (N x K) = dy_e^T x_e: both operands lie across the contraction (the expert's rows).
//
// Each expert's tiles are cut into 8 runs, one per XCD, so an expert with many rows loads all XCDs
// alike (experts dealt to XCDs whole: 4.36 ms instead of 2.07 at 32768 rows, two of 32 experts with
// 40% of them, 5120 x 5120 gradients in fp32).
template <class S, bool OUT_BF16>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void grouped_dw_kernel(
    const unsigned char* __restrict__ dy, const unsigned char* __restrict__ x,
    const int32_t* __restrict__ offsets, unsigned char* __restrict__ dw, int R, int E, int N, int K,
    int n_mtiles, int n_ctiles) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = n_mtiles * n_ctiles, run = (per + 7) >> 3;
  const int local = blockIdx.x >> 3;
  const int t = (blockIdx.x & 7) * run + local % run;
  if (local / run >= E || t >= per) return;
  int begin, end;
  const int e = heavy_first(offsets, E, R, local / run, lane, begin, end);
  if (e < 0) return;   // not reached: every expert has a position
  // tiles of one matrix in bands of kTileGroup tile rows, column by column
  const int m0 = t / (kTileGroup * n_ctiles) * kTileGroup;
  const int sz = min(kTileGroup, n_mtiles - m0), at = t - m0 * n_ctiles;
  const int row0 = (m0 + at % sz) * S::BM, col0 = at / sz * S::BN;
  const int64_t a_ld = (int64_t)N * 2, b_ld = (int64_t)K * 2;
  OperandLoader<S::BM, S::kWaves, true> la;
  OperandLoader<S::BN, S::kWaves, true> lb;
  la.init({dy + begin * a_ld + (int64_t)row0 * 2, a_ld, 0, (N - row0) * 2}, wave, lane);
  lb.init({x + begin * b_ld + (int64_t)col0 * 2, b_ld, 0, (K - col0) * 2}, wave, lane);
  floatx4 acc[S::FM][S::FN];
  tile_zero<S>(acc);
  tile_kloop<S, true, true, false, S::FM>(la, lb, end - begin, smem, wave, lane, acc);
  constexpr int kSize = OUT_BF16 ? 2 : 4;
  tile_store<S, S::FM, OUT_BF16>(acc, dw + (((int64_t)e * N + row0) * K + col0) * kSize,
                                 (int64_t)K * kSize, N - row0, K - col0, smem, wave, lane);
}

// The tile of a call is the one that a model of its time puts first; the experts' own row counts are on
// the device, so it goes by their mean. Per tile shape, in us (fitted to some 400 calls between one
// row and 65536, one expert and 256, widths of 128 to 8192, each measured with every tile):
struct TileCost {
  double mb;      // a megabyte from or to HBM (small tiles keep more loads in flight)
  double l2_mb;   // a megabyte of operands that other tiles read too
  double ends;    // a tile's start and end
  double stage;   // 64 values of its contraction
  double alone;   // the same on a CU that runs no other tile
};
// Workgroups of a shape that the GPU holds at once (the LDS rings decide).
constexpr int kGroupedCus = 256;
template <class S>
constexpr int kSlots = kGroupedCus * (160 * 1024 / S::kLdsBytes);

// Calls f with the candidate for which us(candidate) is least.
template <class Us, class F, class... S>
static void with_least(Us&& us, F&& f, S... tiles) {
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
static constexpr TileCost rows_cost(TileStream) { return {.172, .1, 1.8, .41, 0.}; }
static constexpr TileCost rows_cost(TileLone) { return {.21, .1, 1.7, .25, 0.}; }
static constexpr TileCost rows_cost(Tile64) { return {.228, .1, 2.3, .34, 0.}; }
static constexpr TileCost rows_cost(TilePair) { return {.240, .1, 1.7, .82, 0.}; }
static constexpr TileCost rows_cost(Tile128) { return {.215, .1, 3.2, .50, 0.}; }
static constexpr TileCost rows_cost(Tile192) { return {.235, .1, 3.2, .59, 0.}; }
static constexpr TileCost rows_cost(Tile256Deep) { return {.25, .1, 2.4, .83, 0.}; }
static constexpr TileCost rows_cost(Tile320) { return {.28, .1, 2.3, 1.0, 0.}; }

template <class F>
static void with_rows_tile(int64_t R, int64_t E, int64_t No, int64_t Kc, bool out_bf16, F&& f) {
  const double full = (double)std::min(R, E), mean = (double)R / full;
  const double w_mb = full * No * Kc * 2e-6;
  const double mb = w_mb + R * (Kc * 2e-6 + No * (out_bf16 ? 2e-6 : 4e-6));
  const double stages = (double)ceil_div(Kc, 64);
  auto us = [&](auto s) {
    using S = decltype(s);
    const TileCost c = rows_cost(s);
    double blocks = std::ceil(mean / S::BM);   // of an expert
    if (E > 1)
      blocks = mean + 2.5 * std::sqrt(mean) <= S::BM ? 1.0 : std::max(1.0, mean / S::BM + 0.5);
    const double rounds = std::ceil(full * blocks * ceil_div(No, S::BN) / kSlots<S> - 1e-9);
    return std::max(4.3 + rounds * (c.ends + stages * c.stage),
                    mb * c.mb + w_mb * (blocks - 1.0) * c.l2_mb);
  };
  with_least(us, f, TileStream{}, TileLone{}, Tile64{}, TilePair{}, Tile128{}, Tile192{}, Tile256Deep{},
             Tile320{});
}

// Weight gradient. Measured (us) with 256 x 256, 128 x 128 and 64 x 128 tiles: 32 experts of 1024 rows,
// two with 40% of them, 5120 x 5120 fp32, 1783, 2127, 2783; 22 of 42 rows, 2536 x 4432 bf16, 132, 151,
// 169; 24 of 33 rows, 1656 x 344 fp32, 21, 15, 15. A launch is no shorter than the tiles of its longest
// expert, which is taken to have four times the mean's rows: 24 experts, one with 7500 of 18850 rows,
// 1016 x 392, 166, 98, 86. Taken by this rule, the calls it was fitted to take 3% more than each
// one's best tile.
using Tile256 = TileShape<256, 256, 2, 4, 2, 2>;
using TileHalfPair = TileShape<64, 128, 1, 4, 2, 2>;
static constexpr TileCost dw_cost(Tile256) { return {.205, .10, 3.9, 2.2, 1.4}; }
static constexpr TileCost dw_cost(TilePair) { return {.20, .06, 2.2, 1.1, .8}; }
static constexpr TileCost dw_cost(TileHalfPair) { return {.20, .05, 1.8, 1.0, .7}; }

template <class F>
static void with_dw_tile(int64_t R, int64_t E, int64_t N, int64_t K, bool out_bf16, F&& f) {
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
static int64_t max_blocks(int64_t R, int64_t E, int64_t bm) { return R / bm + std::min(R, E) + 1; }

// A launch counts its threads in 32 bits.
template <class S>
static bool threads_fit(int64_t tiles) {
  return (tiles + 8 * kXcdCus) * S::kThreads < (int64_t(1) << 32);
}

bool grouped_grid_fits(int64_t R, int64_t E, int64_t N, int64_t K) {
  // 64 x 128 tiles of 256 threads are the weight gradient's smallest
  bool ok = threads_fit<Tile256>(E * (ceil_div(N, 128) + 7) * (ceil_div(K, 128) + 7));
  for (int64_t width : {N, K}) {
    // the narrowest tiles' launch fits: so does any
    if (threads_fit<Tile256>(max_blocks(R, E, 32) * ceil_div(width, 64))) continue;
    for (bool out_bf16 : {false, true})
      with_rows_tile(R, E, width, N + K - width, out_bf16, [&](auto s) {
        using S = decltype(s);
        ok = ok && threads_fit<S>(max_blocks(R, E, S::BM) * ceil_div(width, S::BN));
      });
  }
  return ok;
}

hipError_t launch_grouped_rows(const void* a, const void* w, const int32_t* offsets, void* out,
                               int R, int E, int No, int Kc, bool w_across, bool out_bf16,
                               hipStream_t st) {
  with_rows_tile(R, E, No, Kc, out_bf16, [&](auto s) {
    using S = decltype(s);
    const int64_t blocks = max_blocks(R, E, S::BM);
    const int n_ctiles = (int)ceil_div(No, S::BN);
    const dim3 grid = xcd_grid_halves<S>(blocks * n_ctiles);
    auto go = [&](auto across, auto bf16) {
      hipLaunchKernelGGL((grouped_rows_kernel<S, decltype(across)::value, decltype(bf16)::value>),
                         grid, dim3(S::kThreads), 0, st, reinterpret_cast<const unsigned char*>(a),
                         reinterpret_cast<const unsigned char*>(w), offsets,
                         reinterpret_cast<unsigned char*>(out), R, E, No, Kc, n_ctiles, (int)blocks);
    };
    using Y = std::true_type;
    using N = std::false_type;
    if (w_across)
      out_bf16 ? go(Y{}, Y{}) : go(Y{}, N{});
    else
      out_bf16 ? go(N{}, Y{}) : go(N{}, N{});
  });
  return hipGetLastError();
}

template <class S>
static void launch_dw(const void* dy, const void* x, const int32_t* offsets, void* dw, int R, int E,
                      int N, int K, bool out_bf16, hipStream_t st) {
  const int n_mtiles = (int)ceil_div(N, S::BM), n_ctiles = (int)ceil_div(K, S::BN);
  const dim3 grid((unsigned)(8 * E * ceil_div((int64_t)n_mtiles * n_ctiles, 8)));
  const auto* pd = reinterpret_cast<const unsigned char*>(dy);
  const auto* px = reinterpret_cast<const unsigned char*>(x);
  auto* po = reinterpret_cast<unsigned char*>(dw);
  if (out_bf16)
    hipLaunchKernelGGL((grouped_dw_kernel<S, true>), grid, dim3(S::kThreads), 0, st, pd, px,
                       offsets, po, R, E, N, K, n_mtiles, n_ctiles);
  else
    hipLaunchKernelGGL((grouped_dw_kernel<S, false>), grid, dim3(S::kThreads), 0, st, pd, px,
                       offsets, po, R, E, N, K, n_mtiles, n_ctiles);
}

hipError_t launch_grouped_dw(const void* dy, const void* x, const int32_t* offsets, void* dw, int R,
                             int E, int N, int K, bool out_bf16, hipStream_t st) {
  with_dw_tile(R, E, N, K, out_bf16, [&](auto s) {
    launch_dw<decltype(s)>(dy, x, offsets, dw, R, E, N, K, out_bf16, st);
  });
  return hipGetLastError();
}

}  // namespace beam
