// Gated feed-forward products grouped by expert (gfx950): both projections, the activation and the product
// in one launch, and the gradient through them behind the down projection.
//
//   forward    (g | u) = X[r] W_gu[e]^T,  h[r] = bf16(silu(g) u), bf16(g | u) kept          contraction over K
//   gradient   dh = dY[r] W_dn[e] (FP32),  sig = 1 / (1 + e^-g)                           contraction over H
//              d_g = s dh u sig (1 + g (1 - sig)),  d_u = s dh silu(g),  h = s silu(g) u,
//              d_s[r] = sum_f dh silu(g) u                                   (s: the row's scale, or 1)
// h comes from the FP32 products (one rounding, 2^-9 of it), or, where asked, from g and u rounded to bf16 as in
// the block's own forward ([S] §BF16 MoE Kernel Optimization), so that a step recomputed on recorded routes sees
// the values that served them (three roundings). The gradient starts from the kept g and u, whose roundings it
// passes through as the identity.
//
// The products are those of the grouped ones (grouped_mm.hip): a workgroup owns a block of an expert's
// rows and a tile of columns. Forward: a tile of BN weight rows takes BN / 2 gate rows and the same BN / 2
// up rows, in turns of 16, so that a wave holds g and u of the same values. Gradient: the products dh
// never leave the registers; g and u are read, and d_g, d_u and h written, by its epilogue.
//
// Bound by reading the weights for few rows (32 rows, 21 of 32 experts, 5120 -> 2560: 171 us, 6.4 TB/s), by the matrix
// cores for many (4096 rows of one expert, 5120 -> 20480: 1.38 to 1.44 ms, 1190 to 1240 TFLOP/s), in between by the
// weights' latency (8192 rows of 32 experts: 0.46 to 0.48 ms, 4.0 TB/s). The gradient's epilogue moves 10 bytes a
// value, which little of another tile's arithmetic hides: 32768 skewed rows, 5120 -> 2560, 0.86 to 0.88 ms (matrix
// cores busy 49%). Fetching its g and u ahead of the products, or two to five sub-tiles ahead, gained nothing.
#include <type_traits>

#include "narrow.h"
#include "row_blocks.h"
#include "step_rules.h"

namespace beam {

// 1 / (1 + e^-g) with the hardware's exponential and reciprocal: off by (2 + |g|) 2^-23 of it, which the bf16
// results do not show; its limits where e^-g is 0 or infinite. (Full-precision ones, some 40 instructions a
// value, made the gradient of 32768 skewed rows 3% slower.)
__device__ __forceinline__ float sigmoid_fast(float g) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g * -1.442695041f));
}

// silu(g) u of four values, from the FP32 products or from their bf16 roundings gb, ub.
__device__ __forceinline__ floatx4 gated_values(const floatx4 g, const floatx4 u, u32x2 gb, u32x2 ub, bool rounded) {
  const floatx4 gv = rounded ? floatx4{bf16_lo(gb.x), bf16_hi(gb.x), bf16_lo(gb.y), bf16_hi(gb.y)} : g;
  const floatx4 uv = rounded ? floatx4{bf16_lo(ub.x), bf16_hi(ub.x), bf16_lo(ub.y), bf16_hi(ub.y)} : u;
  floatx4 h;
#pragma unroll
  for (int c = 0; c < 4; ++c) h[c] = gv[c] * sigmoid_fast(gv[c]) * uv[c];
  return h;
}

// One tile: rows of `blk`, hidden values from col0 on.
template <class S, bool KEEP>
__device__ __forceinline__ void gated_tile(const unsigned char* __restrict__ x,
                                           const unsigned char* __restrict__ w,
                                           unsigned char* __restrict__ h, unsigned char* __restrict__ gu,
                                           const RowBlock& blk, int col0, int F, int K, bool rounded,
                                           unsigned char* smem, int wave, int lane) {
  static_assert(S::FN % 2 == 0, "gate and up sub-tiles in pairs");
  constexpr int COLS = kGatedCols<S>;
  const int64_t ld = (int64_t)K * 2;
  OperandLoader<S::BM, S::kWaves, false> la;
  OperandLoader<S::BN, S::kWaves, false> lb;
  lb.stream = blk.n_blocks == 1;
  la.init({x + (int64_t)blk.row0 * ld, ld, blk.rows, 0}, wave, lane);
  // weight rows past the gate's last are up rows, whose products are dropped; past those nothing is read
  lb.init({w + (blk.e * 2 * (int64_t)F + col0) * ld, ld, 2 * F - col0, 0}, wave, lane,
          [&](int r) { return (r >> 4 & 1) * F + (r >> 5) * 16 + (r & 15); });
  floatx4 acc[S::FM][S::FN];
  tile_zero<S>(acc);
  with_row_subtiles<S>(blk.rows, wave, [&](auto nv_tag) {
    constexpr int NV = decltype(nv_tag)::value;
    tile_kloop<S, false, false, false, NV>(la, lb, K, smem, wave, lane, acc);
    // a wave's 16 rows of a sub-tile in LDS, a row h | g | u of its 8 FN values each
    constexpr int kPart = S::FN * 16, kRow = (KEEP ? 3 : 1) * kPart, kPitch = kRow + 16;
    static_assert(S::kWaves * 2 * 16 * kPitch <= S::kLdsBytes, "staging fits the ring");
    constexpr int kChunks = kRow / 16, kItems = 16 * kChunks;
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int rows = min(blk.rows, S::BM), cols = min(F - col0, COLS);
    const int64_t h_ld = (int64_t)F * 2, gu_ld = 2 * h_ld;
    const auto h_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        uniform(h + blk.row0 * h_ld + col0 * 2), (short)0, uniform((int)((rows - 1) * h_ld + cols * 2)),
        0x00020000);
    const auto gu_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        uniform(KEEP ? gu + blk.row0 * gu_ld + col0 * 2 : h), (short)0,
        uniform(KEEP ? (int)((rows - 1) * gu_ld + h_ld + cols * 2) : 0), 0x00020000);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unsigned char* const buf = smem + (wave * 2 + (i & 1)) * 16 * kPitch;
#pragma unroll
      for (int j = 0; j < S::FN / 2; ++j) {
        unsigned char* const p = buf + (lane & 15) * kPitch + (16 * j + 4 * (lane >> 4)) * 2;
        const floatx4 g = acc[i][2 * j], u = acc[i][2 * j + 1];
        const u32x2 gb = {pack_bf16(g.x, g.y), pack_bf16(g.z, g.w)};
        const u32x2 ub = {pack_bf16(u.x, u.y), pack_bf16(u.z, u.w)};
        const floatx4 hv = gated_values(g, u, gb, ub, rounded);
        *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16(hv.x, hv.y), pack_bf16(hv.z, hv.w)};
        if constexpr (KEEP) {
          *reinterpret_cast<u32x2*>(p + kPart) = gb;
          *reinterpret_cast<u32x2*>(p + 2 * kPart) = ub;
        }
      }
      // the lanes read each other's values: the compiler keeps the order (no instruction)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int q = 0; q < (kItems + 63) / 64; ++q) {
        const int item = q * 64 + lane;
        if (kItems % 64 != 0 && item >= kItems) continue;
        const int r = item / kChunks, c = item % kChunks, part = c / S::FN;
        const int m = 16 * S::row_tile(wm, i) + r, n = wn * S::FN * 8 + c % S::FN * 8;
        const u32x4 v = *reinterpret_cast<const u32x4*>(buf + r * kPitch + c * 16);
        const bool in = m < rows && n < cols;
        if (part == 0)
          __builtin_amdgcn_raw_buffer_store_b128(v, h_rsrc, in ? (uint32_t)(m * h_ld + n * 2) : 0x80000000u, 0, 0);
        else
          __builtin_amdgcn_raw_buffer_store_b128(
              v, gu_rsrc, in ? (uint32_t)(m * gu_ld + (part - 1) * h_ld + n * 2) : 0x80000000u, 0, 0);
      }
    }
  });
}

template <class S, bool KEEP>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void gated_kernel(
    const unsigned char* __restrict__ x, const unsigned char* __restrict__ w,
    const int32_t* __restrict__ offsets, unsigned char* __restrict__ h, unsigned char* __restrict__ gu, int R,
    int E, int F, int K, bool rounded, int n_ctiles, int max_blocks) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowBlock blk;
  int ctile, half;
  if (!row_block_tile<S, true>(offsets, R, E, n_ctiles, max_blocks, lane, blk, ctile, half)) return;
  const int col0 = ctile * kGatedCols<S>;
  if constexpr (kHalves<S>) {
    if (half >= 0) {
      const int c = col0 + half * kGatedCols<HalfTile<S>>;
      if (c < F) gated_tile<HalfTile<S>, KEEP>(x, w, h, gu, blk, c, F, K, rounded, smem, wave, lane);
      return;
    }
  }
  gated_tile<S, KEEP>(x, w, h, gu, blk, col0, F, K, rounded, smem, wave, lane);
}

// Few rows of few experts: a block's 32 rows (NV sub-tiles of 16) by 16 hidden values a workgroup (narrow.h).
template <bool KEEP, int NV>
__device__ __forceinline__ void gated_narrow_block(const unsigned char* __restrict__ x,
                                                   const unsigned char* __restrict__ w,
                                                   unsigned char* __restrict__ h, unsigned char* __restrict__ gu,
                                                   const RowBlock& blk, int col0, int F, int K, bool rounded,
                                                   floatx4* red, int wave, int lane) {
  const int64_t ld = (int64_t)K * 2;
  floatx4 v[2];
  // weight rows past the up ones read as zero; gate rows past the last are up rows, whose sums are dropped
  if (!narrow_products<NV>(x + (int64_t)blk.row0 * ld, (uint32_t)(blk.rows * ld),
                           w + (blk.e * 2 * (int64_t)F + col0) * ld, (uint32_t)((2 * F - col0) * ld),
                           (uint32_t)(F * ld), K, red, wave, lane, v))
    return;
  const int m = 16 * wave + (lane & 15), n = col0 + 4 * (lane >> 4);
  if (m >= blk.rows || n >= F) return;
  const u32x2 gb = {pack_bf16(v[0].x, v[0].y), pack_bf16(v[0].z, v[0].w)};
  const u32x2 ub = {pack_bf16(v[1].x, v[1].y), pack_bf16(v[1].z, v[1].w)};
  const floatx4 hv = gated_values(v[0], v[1], gb, ub, rounded);
  const int64_t row = blk.row0 + m;
  *reinterpret_cast<u32x2*>(h + (row * F + n) * 2) = u32x2{pack_bf16(hv.x, hv.y), pack_bf16(hv.z, hv.w)};
  if constexpr (KEEP) {
    *reinterpret_cast<u32x2*>(gu + (row * 2 * F + n) * 2) = gb;
    *reinterpret_cast<u32x2*>(gu + (row * 2 * F + F + n) * 2) = ub;
  }
}

template <bool KEEP>
__global__ __launch_bounds__(64 * kNarrowWaves, 2) void gated_narrow_kernel(
    const unsigned char* __restrict__ x, const unsigned char* __restrict__ w,
    const int32_t* __restrict__ offsets, unsigned char* __restrict__ h, unsigned char* __restrict__ gu, int R,
    int E, int F, int K, bool rounded, int n_ctiles, int max_blocks) {
  __shared__ floatx4 red[kNarrowSums];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowBlock blk;
  int ctile, half;
  if (!row_block_tile<TileStream, true>(offsets, R, E, n_ctiles, max_blocks, lane, blk, ctile, half)) return;
  if (blk.rows > 16)
    gated_narrow_block<KEEP, 2>(x, w, h, gu, blk, ctile * kNarrowCols, F, K, rounded, red, wave, lane);
  else
    gated_narrow_block<KEEP, 1>(x, w, h, gu, blk, ctile * kNarrowCols, F, K, rounded, red, wave, lane);
}

struct GatedBwdArgs {
  const unsigned char *dy, *w, *gu;   // [R][H], [E][H][F], [R][2 F], bf16
  const int32_t* offsets;
  const float* scale;                 // [R], or null: 1
  unsigned char *d_gu, *h;            // [R][2 F], [R][F]
  float* parts;                       // [gated_scale_parts(F)][R], with a scale
  int R, E, F, H;
};

template <class S, bool SCALED>
__device__ __forceinline__ void gated_bwd_tile(const GatedBwdArgs& a, const RowBlock& blk, int col0,
                                               int part_cols, unsigned char* smem, int wave, int lane) {
  OperandLoader<S::BM, S::kWaves, false> la;
  OperandLoader<S::BN, S::kWaves, true> lb;
  lb.stream = blk.n_blocks == 1;
  const int64_t dy_ld = (int64_t)a.H * 2, h_ld = (int64_t)a.F * 2, gu_ld = 2 * h_ld;
  la.init({a.dy + blk.row0 * dy_ld, dy_ld, blk.rows, 0}, wave, lane);
  lb.init({a.w + blk.e * (a.H * h_ld) + (int64_t)col0 * 2, h_ld, 0, (a.F - col0) * 2}, wave, lane);
  floatx4 acc[S::FM][S::FN];
  tile_zero<S>(acc);
  with_row_subtiles<S>(blk.rows, wave, [&](auto nv_tag) {
    constexpr int NV = decltype(nv_tag)::value;
    tile_kloop<S, false, true, false, NV>(la, lb, a.H, smem, wave, lane, acc);
    // a wave's 16 rows of a sub-tile in LDS, FP32; eight values a lane, kLanes lanes a row
    constexpr int kPitch = S::FN * 64 + 16, kLanes = 2 * S::FN, kItems = 16 * kLanes;
    static_assert(S::kWaves * 2 * 16 * kPitch <= S::kLdsBytes, "staging fits the ring");
    constexpr int kTurns = (kItems + 63) / 64;
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int rows = min(blk.rows, S::BM), cols = min(a.F - col0, S::BN);
    const int gu_bytes = (int)((rows - 1) * gu_ld + h_ld + cols * 2);
    const unsigned char* const gu0 = uniform(a.gu + blk.row0 * gu_ld + col0 * 2);
    const auto dgu_rsrc = __builtin_amdgcn_make_buffer_rsrc(uniform(a.d_gu + blk.row0 * gu_ld + col0 * 2),
                                                            (short)0, uniform(gu_bytes), 0x00020000);
    const auto h_rsrc = __builtin_amdgcn_make_buffer_rsrc(uniform(a.h + blk.row0 * h_ld + col0 * 2), (short)0,
                                                          uniform((int)((rows - 1) * h_ld + cols * 2)),
                                                          0x00020000);
    struct Item {
      u32x4 g, u;
      float s;
      int m, n;
      bool in;
    };
    auto fetch = [&](int i, int q) {
      Item t;
      const int item = q * 64 + lane;
      t.m = 16 * S::row_tile(wm, i) + item / kLanes;
      t.n = wn * S::FN * 16 + item % kLanes * 8;
      t.in = (kItems % 64 == 0 || item < kItems) && t.m < rows && t.n < cols;
      const uint32_t off = t.in ? (uint32_t)(t.m * gu_ld + t.n * 2) : 0x80000000u;
      t.g = buffer_load16<0>(gu0, (uint32_t)gu_bytes, off, 0);
      t.u = buffer_load16<0>(gu0, (uint32_t)gu_bytes, off, (uint32_t)h_ld);
      t.s = SCALED && t.in ? a.scale[blk.row0 + t.m] : 1.f;
      return t;
    };
    Item next[kTurns];
#pragma unroll
    for (int q = 0; q < kTurns; ++q) next[q] = fetch(0, q);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unsigned char* const buf = smem + (wave * 2 + (i & 1)) * 16 * kPitch;
#pragma unroll
      for (int j = 0; j < S::FN; ++j)
        *reinterpret_cast<floatx4*>(buf + (lane & 15) * kPitch + (16 * j + 4 * (lane >> 4)) * 4) = acc[i][j];
      // the lanes read each other's values: the compiler keeps the order (no instruction)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int q = 0; q < kTurns; ++q) {
        const Item t = next[q];
        if (i + 1 < NV) next[q] = fetch(i + 1, q);
        const int item = q * 64 + lane;
        const floatx4* const p =
            reinterpret_cast<const floatx4*>(buf + (item / kLanes & 15) * kPitch + item % kLanes * 32);
        float dh[8];
        *reinterpret_cast<floatx4*>(dh) = p[0];
        *reinterpret_cast<floatx4*>(dh + 4) = p[1];
        float dg[8], du[8], hv[8], sum = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float g = c & 1 ? bf16_hi(t.g[c / 2]) : bf16_lo(t.g[c / 2]);
          const float u = c & 1 ? bf16_hi(t.u[c / 2]) : bf16_lo(t.u[c / 2]);
          const float sig = sigmoid_fast(g), act = g * sig, hc = act * u;
          if constexpr (SCALED) sum += dh[c] * hc;
          const float d = SCALED ? t.s * dh[c] : dh[c];
          dg[c] = d * u * (sig * (1.f + g * (1.f - sig)));
          du[c] = d * act;
          hv[c] = SCALED ? t.s * hc : hc;
        }
        const uint32_t off = t.in ? (uint32_t)(t.m * gu_ld + t.n * 2) : 0x80000000u;
        auto packed = [](const float(&v)[8]) {
          return u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        };
        // both offsets in the lane's register: behind a wide store with a scalar offset the compiler lets the next
        // instruction write its data registers, and some values in a million came out wrong
        __builtin_amdgcn_raw_buffer_store_b128(packed(dg), dgu_rsrc, off, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(packed(du), dgu_rsrc, off + (uint32_t)h_ld, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(packed(hv), h_rsrc,
                                               t.in ? (uint32_t)(t.m * h_ld + t.n * 2) : 0x80000000u, 0, 0);
        if constexpr (SCALED) {
          // the row's columns of this wave, in the place of their first part; further parts are zero
          sum = t.in ? sum : 0.f;
#pragma unroll
          for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor(sum, d);
          const int own = (col0 + wn * S::FN * 16) / part_cols, n_own = S::FN * 16 / part_cols, k = item % kLanes;
          if (k < n_own && t.m < rows && item < kItems && (own + k) * part_cols < a.F)
            a.parts[(int64_t)(own + k) * a.R + blk.row0 + t.m] = k == 0 ? sum : 0.f;
        }
      }
    }
  });
}

template <class S, bool SCALED>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void gated_bwd_kernel(
    GatedBwdArgs a, int n_ctiles, int max_blocks) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowBlock blk;
  int ctile, half;
  if (!row_block_tile<S, true>(a.offsets, a.R, a.E, n_ctiles, max_blocks, lane, blk, ctile, half)) return;
  const int col0 = ctile * S::BN;
  if constexpr (kHalves<S>) {
    if (half >= 0) {
      const int c = col0 + half * (S::BN / 2);
      if (c < a.F) gated_bwd_tile<HalfTile<S>, SCALED>(a, blk, c, kScaleCols<S>, smem, wave, lane);
      return;
    }
  }
  gated_bwd_tile<S, SCALED>(a, blk, col0, kScaleCols<S>, smem, wave, lane);
}

// d_scale[r] = the sum of row r's parts, in order, for the rows of any expert.
__global__ __launch_bounds__(256) void gated_scale_kernel(const float* __restrict__ parts,
                                                          const int32_t* __restrict__ offsets,
                                                          float* __restrict__ d_scale, int n_parts, int R,
                                                          int E) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r < clamped(offsets[0], 0, R) || r >= clamped(offsets[E], 0, R)) return;
  float s = 0.f;
#pragma unroll 8
  for (int p = 0; p < n_parts; ++p) s += parts[(int64_t)p * R + r];
  d_scale[r] = s;
}

hipError_t launch_gated(const void* x, const void* w, const int32_t* offsets, void* h, void* gu, int R, int E,
                        int F, int K, bool rounded, hipStream_t st) {
  if (gated_is_narrow(R, E, F, K)) {
    const int64_t blocks = grouped_max_blocks(R, E, TileStream::BM);
    const int n_ctiles = (int)ceil_div(F, kNarrowCols);
    const dim3 grid((unsigned)xcd_workgroups_halves<TileStream>(blocks * n_ctiles));
    auto go = [&](auto keep) {
      hipLaunchKernelGGL((gated_narrow_kernel<decltype(keep)::value>), grid, dim3(64 * kNarrowWaves), 0, st,
                         reinterpret_cast<const unsigned char*>(x), reinterpret_cast<const unsigned char*>(w),
                         offsets, reinterpret_cast<unsigned char*>(h), reinterpret_cast<unsigned char*>(gu), R,
                         E, F, K, rounded, n_ctiles, (int)blocks);
    };
    gu ? go(std::true_type{}) : go(std::false_type{});
    return hipGetLastError();
  }
  with_gated_tile(R, E, F, K, gu != nullptr, [&](auto s) {
    using S = decltype(s);
    const int64_t blocks = grouped_max_blocks(R, E, S::BM);
    const int n_ctiles = (int)ceil_div(F, kGatedCols<S>);
    const dim3 grid((unsigned)xcd_workgroups_halves<S>(blocks * n_ctiles));
    auto go = [&](auto keep) {
      hipLaunchKernelGGL((gated_kernel<S, decltype(keep)::value>), grid, dim3(S::kThreads), 0, st,
                         reinterpret_cast<const unsigned char*>(x), reinterpret_cast<const unsigned char*>(w),
                         offsets, reinterpret_cast<unsigned char*>(h), reinterpret_cast<unsigned char*>(gu), R,
                         E, F, K, rounded, n_ctiles, (int)blocks);
    };
    gu ? go(std::true_type{}) : go(std::false_type{});
  });
  return hipGetLastError();
}

hipError_t launch_gated_bwd(const void* dy, const void* w, const void* gu, const int32_t* offsets,
                            const float* scale, void* d_gu, void* h, float* d_scale, float* parts, int R, int E,
                            int F, int H, hipStream_t st) {
  const GatedBwdArgs a = {reinterpret_cast<const unsigned char*>(dy),
                          reinterpret_cast<const unsigned char*>(w),
                          reinterpret_cast<const unsigned char*>(gu),
                          offsets,
                          scale,
                          reinterpret_cast<unsigned char*>(d_gu),
                          reinterpret_cast<unsigned char*>(h),
                          parts,
                          R,
                          E,
                          F,
                          H};
  int part_cols = 0;
  with_gated_bwd_tile(R, E, F, H, [&](auto s) {
    using S = decltype(s);
    part_cols = kScaleCols<S>;
    const int64_t blocks = grouped_max_blocks(R, E, S::BM);
    const int n_ctiles = (int)ceil_div(F, S::BN);
    const dim3 grid((unsigned)xcd_workgroups_halves<S>(blocks * n_ctiles));
    if (scale)
      hipLaunchKernelGGL((gated_bwd_kernel<S, true>), grid, dim3(S::kThreads), 0, st, a, n_ctiles, (int)blocks);
    else
      hipLaunchKernelGGL((gated_bwd_kernel<S, false>), grid, dim3(S::kThreads), 0, st, a, n_ctiles, (int)blocks);
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || !scale) return err;
  hipLaunchKernelGGL(gated_scale_kernel, dim3((unsigned)ceil_div(R, 256)), dim3(256), 0, st, parts, offsets,
                     d_scale, (int)ceil_div(F, part_cols), R, E);
  return hipGetLastError();
}

}  // namespace beam
