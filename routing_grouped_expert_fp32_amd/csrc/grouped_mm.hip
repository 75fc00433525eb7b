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
#include "row_blocks.h"

namespace beam {

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

  with_row_subtiles<S>(blk.rows, wave, [&](auto nv_tag) {
    constexpr int NV = decltype(nv_tag)::value;
    tile_kloop<S, false, WCOL, false, NV>(la, lb, Kc, smem, wave, lane, acc);
    constexpr int kSize = OUT_BF16 ? 2 : 4;
    tile_store<S, NV, OUT_BF16>(acc, out + ((int64_t)blk.row0 * No + col0) * kSize,
                                (int64_t)No * kSize, blk.rows, No - col0, smem, wave, lane);
  });
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
  RowBlock blk;
  int ctile, half;
  if (!row_block_tile<S>(offsets, R, E, n_ctiles, max_blocks, lane, blk, ctile, half)) return;
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
  const int per = n_mtiles * n_ctiles;
  int pos, t;
  if (!dw_tile(blockIdx.x, per, E, pos, t)) return;
  int begin, end;
  const int e = heavy_first(offsets, E, R, pos, lane, begin, end);
  if (e < 0) return;   // not reached: every expert has a position
  int mtile, ctile;
  band_tile(t, n_mtiles, n_ctiles, mtile, ctile);
  const int row0 = mtile * S::BM, col0 = ctile * S::BN;
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

hipError_t launch_grouped_rows(const void* a, const void* w, const int32_t* offsets, void* out,
                               int R, int E, int No, int Kc, bool w_across, bool out_bf16,
                               hipStream_t st) {
  with_rows_tile(R, E, No, Kc, out_bf16, [&](auto s) {
    using S = decltype(s);
    const int64_t blocks = grouped_max_blocks(R, E, S::BM);
    const int n_ctiles = (int)ceil_div(No, S::BN);
    const dim3 grid((unsigned)xcd_workgroups_halves<S>(blocks * n_ctiles));
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
  const dim3 grid((unsigned)dw_workgroups((int64_t)n_mtiles * n_ctiles, E));
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
