// Loss of the output head without its logits, and the gradient (gfx950): softmax cross entropy over the
// vocabulary, the step behind the last boundary.
//
//   z = x w^T  (cap > 0: cap tanh(z / cap)),  lse[t] = log sum_v e^z[t][v],  loss[t] = lse[t] - z[t][y_t]
//   dz[t][v] = d_loss[t] (e^(z - lse) - [v = y_t]) (1 - (z / cap)^2),  dx = dz w,  dw = dz^T x
// The loss: a tile of logits leaves its rows' maxima and sums of exponentials, 8 bytes a row and tile, and
// a second launch joins a row's in order. The gradient: in pieces of the vocabulary, of which the logits
// are computed once more, dz rounded to bf16 (the type that the two products take; FP32 sums in both) and
// kept until dx and dw of that piece are added. dw is whole with its piece; dx is summed over the pieces
// in FP32, and over parts of a piece's contraction where its tiles are fewer than the GPU holds.
//
// Most of a row of dz is its target's value, whose rounding would be that of the whole row of dx and dw. So
// dz is held as c[t] q[t][v], c = d_loss max((1 - p) slope, 2^-20) of the target in FP32, from a product of its own,
// ahead. q at the target is then -1, up to what the two products' logits differ by over 1 - p, and at most 1 beside it
// without a cap; a target near the cap has a smaller slope than the others, whose q are up to 2^20; and where 1 - p
// is under the floor, q is what it leaves of dz. Any of these is rounded by 2^-9 of itself, as dz itself would be. dx
// takes c behind its sums; dw takes it in bf16(c x), whose roundings are independent from value to value. (Against 64
// bits, T = 1: dx 3.9e-3 at worst without, 1.7e-3 with it, which is the last rounding's.)
//
// Bound by the matrix cores, three products of T x V x H with the loss's as a fourth (4096 tokens, 131072 x 5120: loss
// 4.4 to 4.75 ms, 1160 to 1245 TFLOP/s with the machine's clock, gradient 13.1 to 13.85, 1190 to 1260); for few tokens
// by reading w (32 tokens: loss 200 us, 6.7 TB/s), twice for the gradient, and writing dw.
#include <cmath>
#include <type_traits>

#include "narrow.h"
#include "row_blocks.h"
#include "step_rules.h"

namespace beam {

namespace {

// Capped logits cap tanh(r), r = z / cap, within 4 2^-23 of themselves, and with SLOPE their slopes 1 - tanh(r)^2. To
// |r| = 1 tanh(r) / r is the continued fraction's (945 + 105 y + y^2) / (945 + 420 y + 15 y^2), y = r^2, off by 2^-24 there
// and less below; past it tanh = 1 - 2 s and the slope is 4 s (1 - s), s = 1 / (1 + e^2|r|), which would cancel near zero
// (all of 1e-4 for a logit of 1 under a cap of 1024), as 1 - tanh^2 does near the cap. Few logits of a model are past
// its cap: a wave whose row has none (`past`) leaves that out.
template <bool SLOPE>
__device__ __forceinline__ void soft_cap(floatx4& z, floatx4& slope, float cap, float inv_cap, bool past) {
  floatx4 r;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    r[c] = z[c] * inv_cap;
    const float y = r[c] * r[c];
    const float t = __builtin_fmaf(y, y + 105.f, 945.f) *
                    __builtin_amdgcn_rcpf(__builtin_fmaf(y, __builtin_fmaf(y, 15.f, 420.f), 945.f));
    z[c] *= t;
    if constexpr (SLOPE) slope[c] = 1.f - (r[c] * t) * (r[c] * t);
  }
  if (!past) return;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(fabsf(r[c]) * 2.885390082f));
    const bool within = r[c] * r[c] <= 1.f;
    z[c] = within ? z[c] : copysignf(cap * (1.f - 2.f * s), r[c]);
    if constexpr (SLOPE) slope[c] = within ? slope[c] : 4.f * s * (1.f - s);
  }
}
// Whether the wave has a logit past the cap (r^2 > 1 implies it; a NaN stays one through the fraction).
template <int N>
__device__ __forceinline__ bool any_past(const floatx4 (&z4)[N], float cap) {
  float most = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) most = fmaxf(most, fabsf(z4[j][c]));
  return __any(most > 0.999999f * cap);
}
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.442695041f); }

// The logits of T rows and V columns, those of a piece of the vocabulary from column v0 on.
struct LogitArgs {
  const unsigned char *x, *w;      // w: of the piece
  const int32_t* targets;
  int T, V, H, v0, vocab;
  float cap;
  float2* stats;                   // loss: [slots][T] maxima and sums
  float* at_target;                // loss: [T]
  const float *lse, *inv_c;        // gradient: [T]; 1 / (c / d_loss), 0 for a row without a loss
  unsigned char* q;                // gradient: [T][pitch] bf16
  int pitch;
};

// What a launch makes of 4 N FP32 logits z of a row that a lane has, columns n0 + 16 j + 0..3 of a tile of `cols`: with
// GRAD q, zero past the columns, else the row's maximum and sum of exponentials over the lanes that share it (16 and
// 32 apart). `in`: the row m of the block exists.
template <bool GRAD, bool CAP, int N>
__device__ __forceinline__ float2 logit_row(const LogitArgs& a, floatx4 (&z4)[N], int row0, int m, bool in, int col0,
                                            int n0, int cols) {
  const float inv_cap = CAP ? 1.f / a.cap : 0.f;
  const bool past = CAP && any_past(z4, a.cap);
  const int t = row0 + (in ? m : 0);
  const int y = a.targets[t] - a.v0 - col0;   // the target's column of this tile, if it has one
  if constexpr (GRAD) {
    const float lse = a.lse[t], inv = a.inv_c[t];
    const bool counts = in && inv != 0.f;   // a row without a loss may hold anything
#pragma unroll
    for (int j = 0; j < N; ++j) {
      floatx4 slope = {1.f, 1.f, 1.f, 1.f};
      if constexpr (CAP) soft_cap<true>(z4[j], slope, a.cap, inv_cap, past);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n = n0 + 16 * j + c;
        const float p = exp_fast(z4[j][c] - lse) - (n == y ? 1.f : 0.f);
        z4[j][c] = n < cols && counts ? p * slope[c] * inv : 0.f;
      }
      // computed here: left to the stores, behind the next caps' branches, it would take the slopes' registers along
      if constexpr (CAP) asm volatile("" : "+v"(z4[j]));
    }
    return make_float2(0.f, 0.f);
  } else {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      floatx4 unused;
      if constexpr (CAP) soft_cap<false>(z4[j], unused, a.cap, inv_cap, past);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n = n0 + 16 * j + c;
        const float z = n < cols ? z4[j][c] : -INFINITY;
        z4[j][c] = z;
        top = fmaxf(top, z);
        if (in && n == y && n < cols) a.at_target[t] = z;
      }
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float from = top == -INFINITY ? 0.f : top;   // no column: every term is e^-inf
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) sum += exp_fast(z4[j][c] - from);
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    return make_float2(top, sum);
  }
}

// The logits of a tile and what the launch makes of them: q from its columns to the pitch, or the rows' maxima and
// sums in column slot `slot`.
template <class S, bool GRAD, bool CAP>
__device__ __forceinline__ void logit_tile(const LogitArgs& a, const RowBlock& blk, int col0, int slot,
                                           unsigned char* smem, int wave, int lane) {
  const int64_t ld = (int64_t)a.H * 2;
  OperandLoader<S::BM, S::kWaves, false> la;
  OperandLoader<S::BN, S::kWaves, false> lb;
  lb.stream = blk.n_blocks == 1 && !GRAD;   // the gradient reads these rows of w again for dx
  const int cols = a.V - col0;   // of the piece; the pitch may reach further
  la.init({a.x + blk.row0 * ld, ld, blk.rows, 0}, wave, lane);
  lb.init({a.w + (cols > 0 ? col0 * ld : 0), ld, clamped(cols, 0, S::BN), 0}, wave, lane);
  floatx4 acc[S::FM][S::FN];
  tile_zero<S>(acc);
  const int wm = wave / S::WN, wn = wave % S::WN;
  float2* const row_sums = reinterpret_cast<float2*>(smem);   // [WN][BM], in the ring that nobody reads any more
  static_assert(S::WN * S::BM * 8 <= S::kLdsBytes, "row sums fit the ring");
  with_row_subtiles<S>(blk.rows, wave, [&](auto nv_tag) {
    constexpr int NV = decltype(nv_tag)::value;
    tile_kloop<S, false, false, false, NV>(la, lb, a.H, smem, wave, lane, acc);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int m = 16 * S::row_tile(wm, i) + (lane & 15);
      const float2 r = logit_row<GRAD, CAP>(a, acc[i], blk.row0, m, m < blk.rows, col0, wn * S::FN * 16 + 4 * (lane >> 4),
                                            cols);
      if (!GRAD && lane < 16) row_sums[wn * S::BM + m] = r;
    }
    if constexpr (GRAD)
      tile_store<S, NV, true>(acc, a.q + ((int64_t)blk.row0 * a.pitch + col0) * 2, (int64_t)a.pitch * 2, blk.rows,
                              a.pitch - col0, smem, wave, lane);
  });
  if constexpr (!GRAD) {
    __syncthreads();
    for (int m = threadIdx.x; m < blk.rows; m += S::kThreads) {
      float2 r = row_sums[m];
#pragma unroll
      for (int k = 1; k < S::WN; ++k) {
        const float2 o = row_sums[k * S::BM + m];
        const float top = fmaxf(r.x, o.x), from = top == -INFINITY ? 0.f : top;
        r = make_float2(top, r.y * exp_fast(r.x - from) + o.y * exp_fast(o.x - from));
      }
      a.stats[(int64_t)slot * a.T + blk.row0 + m] = r;
    }
  }
}

// The same for few rows and columns: a block of 32 rows by kNarrowLogits columns a workgroup (narrow.h), a slot each.
template <bool GRAD, bool CAP, int NV>
__device__ __forceinline__ void logit_narrow_block(const LogitArgs& a, const RowBlock& blk, int ctile, floatx4* red,
                                                   int wave, int lane) {
  const int64_t ld = (int64_t)a.H * 2;
  const int col0 = ctile * kNarrowLogits, cols = a.V - col0;   // none left between V and the pitch
  floatx4 v[2];
  if (!narrow_products<NV>(a.x + blk.row0 * ld, (uint32_t)(blk.rows * ld), a.w + (cols > 0 ? col0 * ld : 0),
                           (uint32_t)(clamped(cols, 0, kNarrowLogits) * ld), (uint32_t)(16 * ld), a.H, red, wave, lane, v))
    return;
  const int m = 16 * wave + (lane & 15), n0 = 4 * (lane >> 4);
  const bool in = m < blk.rows;
  const float2 r = logit_row<GRAD, CAP>(a, v, blk.row0, m, in, col0, n0, cols);
  if (!in) return;
  if constexpr (GRAD) {
#pragma unroll
    for (int j = 0; j < 2; ++j)   // the pitch is a multiple of 64
      *reinterpret_cast<u32x2*>(a.q + ((int64_t)(blk.row0 + m) * a.pitch + col0 + n0 + 16 * j) * 2) =
          u32x2{pack_bf16(v[j].x, v[j].y), pack_bf16(v[j].z, v[j].w)};
  } else {
    if (lane < 16) a.stats[(int64_t)ctile * a.T + blk.row0 + m] = r;
  }
}

template <bool GRAD, bool CAP>
__global__ __launch_bounds__(64 * kNarrowWaves, 2) void logit_narrow_kernel(LogitArgs a, int n_ctiles) {
  __shared__ floatx4 red[kNarrowSums];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowBlock blk{0, (int)blockIdx.x / n_ctiles * 32, 0, 0, 0};
  blk.rows = min(32, a.T - blk.row0);
  if (blk.rows > 16)
    logit_narrow_block<GRAD, CAP, 2>(a, blk, blockIdx.x % n_ctiles, red, wave, lane);
  else
    logit_narrow_block<GRAD, CAP, 1>(a, blk, blockIdx.x % n_ctiles, red, wave, lane);
}

// Nothing in column slot `slot`.
__device__ __forceinline__ void empty_slot(const LogitArgs& a, const RowBlock& blk, int slot) {
  for (int m = threadIdx.x; m < blk.rows; m += blockDim.x)
    a.stats[(int64_t)slot * a.T + blk.row0 + m] = make_float2(-INFINITY, 0.f);
}

template <class S, bool GRAD, bool CAP>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void logit_kernel(LogitArgs a,
                                                                                              int n_ctiles) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n_blocks = blocks_of<S::BM>(a.T);
  int half, ctile, i;
  const int v = xcd_tile_halves<S>(blockIdx.x, n_blocks * n_ctiles, half);
  if (v < 0) return;
  RowBlock blk{0, 0, 0, 0, n_blocks};
  group_tile(v, v / n_ctiles, v / n_ctiles, n_blocks, n_ctiles, i, ctile);
  block_rows<S::BM>(a.T, n_blocks, i, blk.row0, blk.rows);
  const int col0 = ctile * S::BN;
  if constexpr (kHalves<S>) {
    if (half >= 0) {
      const int c = col0 + half * (S::BN / 2), end = GRAD ? a.pitch : a.V;
      if (c < end)
        logit_tile<HalfTile<S>, GRAD, CAP>(a, blk, c, 2 * ctile + half, smem, wave, lane);
      else if (!GRAD)
        empty_slot(a, blk, 2 * ctile + half);
      return;
    }
    if (!GRAD) empty_slot(a, blk, 2 * ctile + 1);
    logit_tile<S, GRAD, CAP>(a, blk, col0, 2 * ctile, smem, wave, lane);
  } else {
    logit_tile<S, GRAD, CAP>(a, blk, col0, ctile, smem, wave, lane);
  }
}

// lse and loss of kJoinRows rows a workgroup: kJoinWays threads a row join every kJoinWays-th slot, then their
// results pair by pair. Few tokens: four rows and 128 threads each (32 tokens, 1024 slots: 4.2 us, 16 rows of 64
// 11); more: 16 rows of 32, a line of 128 bytes a slot (4096 tokens, 1024 slots: 9 us, four rows 25).
template <int kJoinRows, int kJoinWays>
__global__ __launch_bounds__(kJoinRows * kJoinWays) void head_join_kernel(
    const float2* __restrict__ stats, const float* __restrict__ at_target, const int32_t* __restrict__ targets,
    float* __restrict__ loss, float* __restrict__ lse_out, int slots, int T, int vocab) {
  __shared__ float2 part[kJoinWays][kJoinRows];
  const int r = threadIdx.x % kJoinRows, k = threadIdx.x / kJoinRows;
  const int t = blockIdx.x * kJoinRows + r;
  float top = -INFINITY, sum = 0.f;
  auto join = [&](float2 o) {
    const float m = fmaxf(top, o.x), from = m == -INFINITY ? 0.f : m;
    sum = sum * exp_fast(top - from) + o.y * exp_fast(o.x - from);
    top = m;
  };
  if (t < T) {
#pragma unroll 8
    for (int s = k; s < slots; s += kJoinWays) join(stats[(int64_t)s * T + t]);
  }
#pragma unroll
  for (int n = kJoinWays / 2; n > 0; n >>= 1) {
    if (k >= n && k < 2 * n) part[k][r] = make_float2(top, sum);
    __syncthreads();
    if (k < n) join(part[k + n][r]);
  }
  if (k > 0 || t >= T) return;
  const float lse = top + logf(sum);
  const int y = targets[t];
  lse_out[t] = lse;
  loss[t] = y >= 0 && y < vocab ? lse - at_target[t] : 0.f;
}

// c of each token, a workgroup a token: c = d_loss max((1 - p) slope, 2^-20) at its target (0 without one),
// inv_c = 1 / (c / d_loss), and xc = bf16(c x).
struct ScaleArgs {
  const uint16_t *x, *w;   // w: the whole vocabulary's
  const int32_t* targets;
  const float *lse, *d_loss;
  float *c, *inv_c;
  uint16_t* xc;
  int vocab, H;
  float cap;
};
constexpr int kScaleThreads = 256;
__global__ __launch_bounds__(kScaleThreads) void head_scale_kernel(ScaleArgs a) {
  __shared__ float waves[kScaleThreads / 64];
  const int64_t t = blockIdx.x;
  const int y = a.targets[t];
  const bool counts = y >= 0 && y < a.vocab;   // uniform
  const uint16_t* const x = a.x + t * a.H;
  const uint16_t* const w = a.w + (counts ? y : 0) * (int64_t)a.H;
  float c = 0.f;
  if (counts) {
    float sum = 0.f;
    for (int i = 8 * threadIdx.x; i < a.H; i += 8 * kScaleThreads) {
      const u32x4 u = *reinterpret_cast<const u32x4*>(x + i), v = *reinterpret_cast<const u32x4*>(w + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) sum += bf16_lo(u[k]) * bf16_lo(v[k]) + bf16_hi(u[k]) * bf16_hi(v[k]);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = sum;
    __syncthreads();
    float z = waves[0];
#pragma unroll
    for (int k = 1; k < kScaleThreads / 64; ++k) z += waves[k];
    float slope = 1.f;
    if (a.cap > 0.f) {
      floatx4 z4[1] = {{z, 0.f, 0.f, 0.f}}, slopes;
      soft_cap<true>(z4[0], slopes, a.cap, 1.f / a.cap, any_past(z4, a.cap));
      z = z4[0].x;
      slope = slopes.x;
    }
    const float share = fmaxf((1.f - exp_fast(z - a.lse[t])) * slope, 0x1p-20f);   // NaN: the floor
    c = a.d_loss[t] * share;
    if (threadIdx.x == 0) a.inv_c[t] = 1.f / share;
  } else if (threadIdx.x == 0) {
    a.inv_c[t] = 0.f;
  }
  if (threadIdx.x == 0) a.c[t] = c;
  for (int i = 8 * threadIdx.x; i < a.H; i += 8 * kScaleThreads) {
    u32x4 u = {0, 0, 0, 0};
    if (counts) {
      u = *reinterpret_cast<const u32x4*>(x + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = pack_bf16(c * bf16_lo(u[k]), c * bf16_hi(u[k]));
    }
    *reinterpret_cast<u32x4*>(a.xc + t * a.H + i) = u;
  }
}

// Sums of dx: D = q w over a run of kp columns of the piece, a part a run. OUT: 0 bf16(c D) to `out`, 1 FP32 to
// the part's sums, 2 added to them.
struct DxArgs {
  const unsigned char *q, *w;   // [T][pitch], [V][H] of the piece
  const float* c;               // [T]
  unsigned char* out;
  int T, V, H, pitch, parts, kp;
};
template <class S, int OUT>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void head_dx_kernel(DxArgs a, int n_mtiles,
                                                                                                int n_ctiles) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = n_mtiles * n_ctiles;
  const int v = xcd_tile(blockIdx.x, tiles * a.parts);
  if (v < 0) return;
  const int part = v / tiles, k0 = part * a.kp;
  int mtile, ctile;
  band_tile(v % tiles, n_mtiles, n_ctiles, mtile, ctile);
  const int row0 = mtile * S::BM, col0 = ctile * S::BN, rows = min(S::BM, a.T - row0);
  const int k = clamped(a.V - k0, 0, a.kp);   // none left: the last piece is the shortest
  const int64_t z_ld = (int64_t)a.pitch * 2, w_ld = (int64_t)a.H * 2;
  OperandLoader<S::BM, S::kWaves, false> la;
  OperandLoader<S::BN, S::kWaves, true> lb;
  la.init({a.q + row0 * z_ld + (k > 0 ? (int64_t)k0 * 2 : 0), z_ld, rows, 0}, wave, lane);
  lb.init({a.w + (k > 0 ? k0 * w_ld : 0) + (int64_t)col0 * 2, w_ld, 0, (a.H - col0) * 2}, wave, lane);
  floatx4 acc[S::FM][S::FN];
  tile_zero<S>(acc);
  with_row_subtiles<S>(rows, wave, [&](auto nv_tag) {
    constexpr int NV = decltype(nv_tag)::value;
    tile_kloop<S, false, true, false, NV>(la, lb, k, smem, wave, lane, acc);
    if constexpr (OUT == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int m = 16 * S::row_tile(wave / S::WN, i) + (lane & 15);
        const float c = m < rows ? a.c[row0 + m] : 0.f;
#pragma unroll
        for (int j = 0; j < S::FN; ++j) acc[i][j] *= c;
      }
      tile_store<S, NV, true>(acc, a.out + ((int64_t)row0 * a.H + col0) * 2, w_ld, rows, a.H - col0, smem, wave, lane);
    } else {
      unsigned char* const out = a.out + (((int64_t)part * a.T + row0) * a.H + col0) * 4;
      if constexpr (OUT == 1) {
        tile_store<S, NV, false>(acc, out, 2 * w_ld, rows, a.H - col0, smem, wave, lane);
      } else {
        const int64_t ld = 2 * w_ld;
        const int cols = min(a.H - col0, S::BN);
        const uint32_t bytes = (uint32_t)((rows - 1) * ld + cols * 4);
        const unsigned char* const base = uniform(out);
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(uniform(out), (short)0, uniform((int)bytes), 0x00020000);
        tile_rows<S, NV, 4>(
            smem, wave, lane,
            [&](int i, int j, unsigned char* p) { *reinterpret_cast<floatx4*>(p) = acc[i][j]; },
            [&](int m, int n, const unsigned char* p) {
              const uint32_t off = m < rows && n < cols ? (uint32_t)(m * ld + n * 4) : 0x80000000u;
              const floatx4 sum = *reinterpret_cast<const floatx4*>(p) +
                                  __builtin_bit_cast(floatx4, buffer_load16<0>(base, bytes, off, 0));
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sum), rsrc, off, 0, 0);
            });
      }
    }
  });
}

// dx = c times the sum of the parts, in order; eight values of a row a thread.
__global__ __launch_bounds__(256) void head_dx_sum_kernel(const float* __restrict__ sums, const float* __restrict__ c,
                                                          uint16_t* __restrict__ dx, int64_t count, int H, int parts) {
  const int64_t i = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (i >= count) return;
  floatx4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    a += *reinterpret_cast<const floatx4*>(sums + p * count + i);
    b += *reinterpret_cast<const floatx4*>(sums + p * count + i + 4);
  }
  const float scale = c[i / H];
  a *= scale;
  b *= scale;
  *reinterpret_cast<u32x4*>(dx + i) = u32x4{pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w)};
}

// dw (V x H of a piece) = q^T xc: both operands lie across the contraction (the tokens).
template <class S, bool OUT_BF16>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void head_dw_kernel(
    const unsigned char* __restrict__ q, const unsigned char* __restrict__ xc, unsigned char* __restrict__ dw, int T,
    int V, int H, int pitch, int n_mtiles, int n_ctiles) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int v = xcd_tile(blockIdx.x, n_mtiles * n_ctiles);
  if (v < 0) return;
  int mtile, ctile;
  band_tile(v, n_mtiles, n_ctiles, mtile, ctile);
  const int row0 = mtile * S::BM, col0 = ctile * S::BN;
  OperandLoader<S::BM, S::kWaves, true> la;
  OperandLoader<S::BN, S::kWaves, true> lb;
  la.init({q + (int64_t)row0 * 2, (int64_t)pitch * 2, 0, (pitch - row0) * 2}, wave, lane);
  lb.init({xc + (int64_t)col0 * 2, (int64_t)H * 2, 0, (H - col0) * 2}, wave, lane);
  floatx4 acc[S::FM][S::FN];
  tile_zero<S>(acc);
  tile_kloop<S, true, true, false, S::FM>(la, lb, T, smem, wave, lane, acc);
  constexpr int kSize = OUT_BF16 ? 2 : 4;
  tile_store<S, S::FM, OUT_BF16>(acc, dw + ((int64_t)row0 * H + col0) * kSize, (int64_t)H * kSize, V - row0, H - col0,
                                 smem, wave, lane);
}

template <bool GRAD>
void launch_logits(const LogitArgs& a, int64_t end, hipStream_t st) {
  if (head_is_narrow(a.T, end, a.H)) {
    const int n_ctiles = (int)ceil_div(end, kNarrowLogits);
    const dim3 grid((unsigned)(ceil_div(a.T, 32) * n_ctiles));
    if (a.cap > 0.f)
      hipLaunchKernelGGL((logit_narrow_kernel<GRAD, true>), grid, dim3(64 * kNarrowWaves), 0, st, a, n_ctiles);
    else
      hipLaunchKernelGGL((logit_narrow_kernel<GRAD, false>), grid, dim3(64 * kNarrowWaves), 0, st, a, n_ctiles);
    return;
  }
  with_head_tile(a.T, a.V, a.H, GRAD, [&](auto s) {
    using S = decltype(s);
    const int n_ctiles = (int)ceil_div(end, S::BN);
    const dim3 grid((unsigned)xcd_workgroups_halves<S>(blocks_of<S::BM>(a.T) * (int64_t)n_ctiles));
    if (a.cap > 0.f)
      hipLaunchKernelGGL((logit_kernel<S, GRAD, true>), grid, dim3(S::kThreads), 0, st, a, n_ctiles);
    else
      hipLaunchKernelGGL((logit_kernel<S, GRAD, false>), grid, dim3(S::kThreads), 0, st, a, n_ctiles);
  });
}

template <class S>
void launch_dx(const DxArgs& a, int out, hipStream_t st) {
  const int mt = (int)ceil_div(a.T, S::BM), ct = (int)ceil_div(a.H, S::BN);
  const dim3 grid((unsigned)xcd_workgroups((int64_t)mt * ct * a.parts));
  if (out == 0)
    hipLaunchKernelGGL((head_dx_kernel<S, 0>), grid, dim3(S::kThreads), 0, st, a, mt, ct);
  else if (out == 1)
    hipLaunchKernelGGL((head_dx_kernel<S, 1>), grid, dim3(S::kThreads), 0, st, a, mt, ct);
  else
    hipLaunchKernelGGL((head_dx_kernel<S, 2>), grid, dim3(S::kThreads), 0, st, a, mt, ct);
}

void launch_dw(const unsigned char* q, const unsigned char* xc, unsigned char* dw, bool bf16, int T, int V, int H,
               int pitch, hipStream_t st) {
  with_dw_tile(T, 1, V, H, bf16, [&](auto s) {
    using S = decltype(s);
    const int mt = (int)ceil_div(V, S::BM), ct = (int)ceil_div(H, S::BN);
    const dim3 grid((unsigned)xcd_workgroups((int64_t)mt * ct));
    if (bf16)
      hipLaunchKernelGGL((head_dw_kernel<S, true>), grid, dim3(S::kThreads), 0, st, q, xc, dw, T, V, H, pitch, mt, ct);
    else
      hipLaunchKernelGGL((head_dw_kernel<S, false>), grid, dim3(S::kThreads), 0, st, q, xc, dw, T, V, H, pitch, mt, ct);
  });
}

}  // namespace

hipError_t launch_head_loss(const HeadArgs& h, float* loss, float* lse, char* ws, hipStream_t st) {
  const HeadLayout L = head_layout(h.T, h.V, h.H);
  LogitArgs a = {};
  a.x = reinterpret_cast<const unsigned char*>(h.x);
  a.w = reinterpret_cast<const unsigned char*>(h.w);
  a.targets = h.targets;
  a.T = (int)h.T;
  a.V = a.vocab = (int)h.V;
  a.H = h.H;
  a.cap = h.cap;
  a.stats = reinterpret_cast<float2*>(ws);
  a.at_target = reinterpret_cast<float*>(ws + L.at_target);
  launch_logits<false>(a, a.V, st);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  auto join = [&](auto rows, auto ways) {
    constexpr int kRows = decltype(rows)::value, kWays = decltype(ways)::value;
    hipLaunchKernelGGL((head_join_kernel<kRows, kWays>), dim3((unsigned)ceil_div(h.T, kRows)), dim3(kRows * kWays), 0, st,
                       a.stats, a.at_target, a.targets, loss, lse, (int)L.slots, a.T, a.vocab);
  };
  if (h.T < 1024)
    join(std::integral_constant<int, 4>{}, std::integral_constant<int, 128>{});
  else
    join(std::integral_constant<int, 16>{}, std::integral_constant<int, 32>{});
  return hipGetLastError();
}

hipError_t launch_head_loss_bwd(const HeadArgs& h, const float* lse, const float* d_loss, uint16_t* dx, void* dw,
                                bool dw_bf16, char* ws, hipStream_t st) {
  if (h.T == 0) {   // a sum over no tokens
    launch_dw(nullptr, nullptr, reinterpret_cast<unsigned char*>(dw), dw_bf16, 0, (int)h.V, h.H, (int)h.V, st);
    return hipGetLastError();
  }
  const HeadBwdLayout L = head_bwd_layout(h.T, h.V, h.H);
  float* const sums = reinterpret_cast<float*>(ws + L.sums);
  float* const c = reinterpret_cast<float*>(ws + L.c);
  unsigned char* const xc = reinterpret_cast<unsigned char*>(ws + L.xc);
  const ScaleArgs scales = {h.x, h.w, h.targets, lse, d_loss, c, c + h.T, reinterpret_cast<uint16_t*>(xc), (int)h.V, h.H,
                            h.cap};
  hipLaunchKernelGGL(head_scale_kernel, dim3((unsigned)h.T), dim3(kScaleThreads), 0, st, scales);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  for (int64_t p = 0; p < L.pieces; ++p) {
    const int64_t v0 = p * L.cols, cols = std::min(L.cols, h.V - v0);
    LogitArgs a = {};
    a.x = reinterpret_cast<const unsigned char*>(h.x);
    a.w = reinterpret_cast<const unsigned char*>(h.w + v0 * h.H);
    a.targets = h.targets;
    a.T = (int)h.T;
    a.V = (int)cols;
    a.H = h.H;
    a.v0 = (int)v0;
    a.vocab = (int)h.V;
    a.cap = h.cap;
    a.lse = lse;
    a.inv_c = c + h.T;
    a.q = reinterpret_cast<unsigned char*>(ws);
    a.pitch = (int)(ceil_div(cols, kStageK) * kStageK);
    launch_logits<true>(a, a.pitch, st);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    const DxArgs d = {a.q, a.w, c, L.direct() ? reinterpret_cast<unsigned char*>(dx) : reinterpret_cast<unsigned char*>(sums),
                      a.T, a.V, a.H, a.pitch, L.dx.parts, (int)L.dx.kp};
    const int out = L.direct() ? 0 : p == 0 ? 1 : 2;
    switch (L.dx.side) {
      case 256: launch_dx<DxTile256>(d, out, st); break;
      case 128: launch_dx<DxTile128>(d, out, st); break;
      case 64: launch_dx<DxTile64>(d, out, st); break;
      default: launch_dx<DxTile32>(d, out, st); break;
    }
    if ((err = hipGetLastError()) != hipSuccess) return err;
    launch_dw(a.q, xc, reinterpret_cast<unsigned char*>(dw) + v0 * h.H * (dw_bf16 ? 2 : 4), dw_bf16, a.T, a.V, a.H,
              a.pitch, st);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  if (!L.direct()) {
    const int64_t count = h.T * h.H;
    hipLaunchKernelGGL(head_dx_sum_kernel, dim3((unsigned)ceil_div(count, 8 * 256)), dim3(256), 0, st, sums, c, dx, count,
                       h.H, L.dx.parts);
  }
  return hipGetLastError();
}

}  // namespace beam
