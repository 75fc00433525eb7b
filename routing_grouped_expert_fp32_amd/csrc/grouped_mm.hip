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

#include "gemm_tile.h"

namespace beam {

// A block of rows of one expert, as found from the offsets.
struct RowBlock {
  int e;          // expert
  int row0;       // first row of the block
  int rows;       // rows in the block
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

// Blocks of BM rows of all experts in expert order: `total` of them; find(b) gives block b. Lane l
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
        c += (z - a + BM - 1) / BM;
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
      const int n = (z - a + BM - 1) / BM;
      if (left < n) {
        r = RowBlock{e, a + left * BM, min(BM, z - a - left * BM), left, n};
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

// Tile v of `total` for workgroup `wg` of a grid of 8 ceil(total / 8), one run of tiles per XCD.
__device__ __forceinline__ int xcd_tile(int wg, int total) {
  const int per = (total + 7) >> 3, local = wg >> 3;
  const int v = (wg & 7) * per + local;
  return local < per && v < total ? v : -1;
}

constexpr int kTileGroup = 4;   // blocks of one expert walked together, column tile by column tile

// out[row][0 .. No) = a[row][0 .. Kc) . w[e], w stored [No][Kc] (forward) or, WCOL, [Kc][No] (input
// gradient: the weight's rows run across the contraction).
template <class S, bool WCOL, bool OUT_BF16>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void grouped_rows_kernel(
    const unsigned char* __restrict__ a, const unsigned char* __restrict__ w,
    const int32_t* __restrict__ offsets, void* __restrict__ out, int R, int E, int No, int Kc,
    int n_ctiles, int max_blocks) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  BlockScan<S::BM> scan;
  scan.init(offsets, E, R, lane);
  // more blocks than the grid has come only from offsets that are not in order
  const int v = xcd_tile(blockIdx.x, min(scan.total, max_blocks) * n_ctiles);
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
    int lo, hi;
    expert_rows(offsets, blk.e, R, lo, hi);
    blk.row0 = lo + (g0 + at % sz) * S::BM;
    blk.rows = min(S::BM, hi - blk.row0);
  }
  const int col0 = ctile * S::BN;
  const int64_t wbytes = (int64_t)No * Kc * 2;
  const int64_t a_ld = (int64_t)Kc * 2;
  OperandLoader<S::BM, S::kWaves, false> la;
  OperandLoader<S::BN, S::kWaves, WCOL> lb;
  la.init({a + (int64_t)blk.row0 * a_ld, a_ld, blk.rows, 0}, wave, lane);
  if constexpr (WCOL)
    lb.init({w + blk.e * wbytes + (int64_t)col0 * 2, (int64_t)No * 2, 0, (No - col0) * 2}, wave,
            lane);
  else
    lb.init({w + blk.e * wbytes + (int64_t)col0 * a_ld, a_ld, min(S::BN, No - col0), 0}, wave, lane);

  floatx4 acc[S::FM][S::FN];
#pragma unroll
  for (int i = 0; i < S::FM; ++i)
#pragma unroll
    for (int j = 0; j < S::FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  auto store = [&](int m, int n, floatx4 d) {
    if (m < blk.rows && col0 + n < No)   // No % 8 == 0: four columns are all in or all out
      store4<OUT_BF16>(out, (int64_t)(blk.row0 + m) * No + col0 + n, d);
  };
  tile_kloop<S, false, WCOL, false, S::FM>(la, lb, Kc, smem, wave, lane, acc);
  tile_for_each<S, S::FM>(acc, wave, lane, store);
}

// dw[e] (N x K) = dy_e^T x_e: both operands lie across the contraction (the expert's rows).
template <class S, bool OUT_BF16>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void grouped_dw_kernel(
    const unsigned char* __restrict__ dy, const unsigned char* __restrict__ x,
    const int32_t* __restrict__ offsets, void* __restrict__ dw, int R, int E, int N, int K,
    int n_mtiles, int n_ctiles) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int v = xcd_tile(blockIdx.x, E * n_mtiles * n_ctiles);
  if (v < 0) return;
  const int per = n_mtiles * n_ctiles, e = v / per, t = v % per;
  // tiles of one matrix in bands of kTileGroup tile rows, column by column
  const int band = t / (kTileGroup * n_ctiles), m0 = band * kTileGroup;
  const int sz = min(kTileGroup, n_mtiles - m0), at = t - m0 * n_ctiles;
  const int row0 = (m0 + at % sz) * S::BM, col0 = at / sz * S::BN;
  int begin, end;
  expert_rows(offsets, e, R, begin, end);
  OperandLoader<S::BM, S::kWaves, true> la;
  OperandLoader<S::BN, S::kWaves, true> lb;
  la.init({dy + (int64_t)begin * N * 2 + (int64_t)row0 * 2, (int64_t)N * 2, 0, (N - row0) * 2},
          wave, lane);
  lb.init({x + (int64_t)begin * K * 2 + (int64_t)col0 * 2, (int64_t)K * 2, 0, (K - col0) * 2},
          wave, lane);
  floatx4 acc[S::FM][S::FN];
#pragma unroll
  for (int i = 0; i < S::FM; ++i)
#pragma unroll
    for (int j = 0; j < S::FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  tile_kloop<S, true, true, false, S::FM>(la, lb, end - begin, smem, wave, lane, acc);
  tile_for_each<S, S::FM>(acc, wave, lane, [&](int m, int n, floatx4 d) {
    if (row0 + m < N && col0 + n < K)
      store4<OUT_BF16>(dw, ((int64_t)e * N + row0 + m) * K + col0 + n, d);
  });
}

using TileLarge = TileShape<256, 256, 2, 4, 2>;
using TileSmall = TileShape<128, 128, 2, 2, 2>;

bool grouped_grid_fits(int64_t R, int64_t E, int64_t N, int64_t K) {
  const int64_t blocks = R / 128 + std::min(R, E) + 1;
  const int64_t nt = ceil_div(N, 128), kt = ceil_div(K, 128), lim = (int64_t(1) << 31) - 8;
  return blocks * std::max(nt, kt) < lim && E * nt * kt < lim;
}

template <class S, bool WCOL>
static void launch_rows(const void* a, const void* w, const int32_t* offsets, void* out, int R,
                        int E, int No, int Kc, bool out_bf16, hipStream_t st) {
  const int64_t blocks = R / S::BM + std::min(R, E) + 1;
  const int n_ctiles = (int)ceil_div(No, S::BN);
  const dim3 grid((unsigned)(8 * ceil_div(blocks * n_ctiles, 8)));
  const auto* pa = reinterpret_cast<const unsigned char*>(a);
  const auto* pw = reinterpret_cast<const unsigned char*>(w);
  if (out_bf16)
    hipLaunchKernelGGL((grouped_rows_kernel<S, WCOL, true>), grid, dim3(S::kThreads), 0, st, pa, pw,
                       offsets, out, R, E, No, Kc, n_ctiles, (int)blocks);
  else
    hipLaunchKernelGGL((grouped_rows_kernel<S, WCOL, false>), grid, dim3(S::kThreads), 0, st, pa,
                       pw, offsets, out, R, E, No, Kc, n_ctiles, (int)blocks);
}

hipError_t launch_grouped_rows(const void* a, const void* w, const int32_t* offsets, void* out,
                               int R, int E, int No, int Kc, bool w_across, bool out_bf16,
                               hipStream_t st) {
  if (w_across)
    launch_rows<TileSmall, true>(a, w, offsets, out, R, E, No, Kc, out_bf16, st);
  else
    launch_rows<TileSmall, false>(a, w, offsets, out, R, E, No, Kc, out_bf16, st);
  return hipGetLastError();
}

hipError_t launch_grouped_dw(const void* dy, const void* x, const int32_t* offsets, void* dw, int R,
                             int E, int N, int K, bool out_bf16, hipStream_t st) {
  using S = TileSmall;
  const int n_mtiles = (int)ceil_div(N, S::BM), n_ctiles = (int)ceil_div(K, S::BN);
  const dim3 grid((unsigned)(8 * ceil_div((int64_t)E * n_mtiles * n_ctiles, 8)));
  const auto* pd = reinterpret_cast<const unsigned char*>(dy);
  const auto* px = reinterpret_cast<const unsigned char*>(x);
  if (out_bf16)
    hipLaunchKernelGGL((grouped_dw_kernel<S, true>), grid, dim3(S::kThreads), 0, st, pd, px,
                       offsets, dw, R, E, N, K, n_mtiles, n_ctiles);
  else
    hipLaunchKernelGGL((grouped_dw_kernel<S, false>), grid, dim3(S::kThreads), 0, st, pd, px,
                       offsets, dw, R, E, N, K, n_mtiles, n_ctiles);
  return hipGetLastError();
}

}  // namespace beam
