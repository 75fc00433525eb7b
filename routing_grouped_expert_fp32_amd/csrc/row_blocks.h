// Blocks of rows of the products grouped by expert, found on the device from the offsets (gfx950): shared
// by the grouped products and the gated ones. Device code, but for the wave's exchanges plain C++: included behind the
// header that declares those (gemm_tile.h; a check on the CPU hands in its own and runs the lanes in turn).
#pragma once

#include <type_traits>

#include "train_rules.h"

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

// Tile of a workgroup: the block's rows, its column tile and, for the last tiles of a launch, which
// column half (else -1). False: none. DEALT: tiles dealt to the XCDs by xcd_tile_dealt.
template <class S, bool DEALT = false>
__device__ __forceinline__ bool row_block_tile(const int32_t* __restrict__ offsets, int R, int E,
                                               int n_ctiles, int max_blocks, int lane, RowBlock& blk,
                                               int& ctile, int& half) {
  BlockScan<S::BM> scan;
  scan.init(offsets, E, R, lane);
  // more blocks than the grid has come only from offsets that are not in order
  const int total = min(scan.total, max_blocks) * n_ctiles;
  const int v = DEALT ? xcd_tile_dealt<S>(blockIdx.x, total, half) : xcd_tile_halves<S>(blockIdx.x, total, half);
  if (v < 0) return false;
  blk = scan.find(v / n_ctiles);
  if (blk.rows <= 0) return false;
  int i, first, rows;
  group_tile(v, v / n_ctiles, blk.in_expert, blk.n_blocks, n_ctiles, i, ctile);
  block_rows<S::BM>(blk.rows, blk.n_blocks, i, first, rows);
  blk.row0 += first;
  blk.rows = rows;
  return true;
}

// Calls body(NV) with the number of a wave's row sub-tiles that `rows` rows of a tile fill, rounded up to
// two: sub-tiles of 16 rows are dealt to the wave rows in turn, so a partly filled block costs about its
// rows.
template <class S, class F>
__device__ __forceinline__ void with_row_subtiles(int rows, int wave, F&& body) {
  const int nsub = (rows + 15) >> 4, wm = wave / S::WN;
  const int nv = (nsub - wm + S::WM - 1) / S::WM;   // wave-uniform; 0 where nsub <= wm
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

}  // namespace beam
