// Orthogonalised update of weight matrices (gfx950): the Newton-Schulz iteration of the Muon optimiser,
//   X <- G / (|G|_F + eps);   A = X X^T,  X <- a X + (b A + c A^2) X,   `steps` times,
// with X taken along its shorter side (a tall G is transposed on the way in and out, as
// p(X X^T) X = X p(X^T X)).
//
// Number formats. The products run on the 16-bit matrix cores with FP32 sums, on fp16 rather than
// bf16 (three more bits at the same rate; every matrix is scaled by a power of two that puts its
// entries in fp16's range). X is kept as a pair of fp16, hi + lo: the products take hi, the term a X
// both. Without lo, each step would add a rounding error in every direction, and directions in which
// G is weak are amplified by up to a^steps (about 480 for the usual coefficients): a rank-one G came
// out 10% wrong with fp16 alone and 0.03% with the pair. B is stored as B + s I with s = -(b + c), its
// value on converged directions: entries then shrink as X converges, and their rounding with them
// (the update takes s back off X exactly). Measured against 64 bits before the last rounding to bf16
// (which is 0.17%): 0.05 - 0.2%.
//
// Where |G|_F is far under eps, X starts far under 1 and would sink below fp16's smallest values (at
// |G|_F = 1e-5 eps the result was 2% off, from 1e-7 eps on zero). Each matrix therefore holds X times
// a power of two of its own, 2^j, chosen anew at every step from a bound u on X's singular values:
// j = 0 from u = 1/2 on, else 2^j u in [1/2, 1). u starts as |G|_F / (|G|_F + eps); a step takes a
// singular value v to p(v) = a v + b v^3 + c v^5, and u to the largest |p| up to u. A then holds 4^j
// times its values, B and the update undo that exactly.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gemm_tile.h"

namespace beam {

constexpr float kGramScale = 256.f;     // A and B hold 2^8 times their values

// X holds 2^k times its values, 2^k about sqrt(longer side): a matrix of orthonormal rows has entries
// of about 1 / sqrt(longer side).
static float x_scale(int n_long) {
  float s = 1.f;
  while (s * s < (float)n_long) s *= 2.f;
  return s;
}

// 2^-j for a bound u >= 0 on X's norm; NaN gives 1.
constexpr int kMaxShift = 100;
__device__ __forceinline__ float ns_unit(float u) {
  const int e = (int)(__float_as_uint(u) >> 23 & 255) - 126;   // u < 2^e; subnormals -126
  return __uint_as_float((uint32_t)(127 + min(max(e, -kMaxShift), 0)) << 23);
}
__device__ __forceinline__ float pow2_inverse(float unit) {   // of a power of two
  return __uint_as_float((254u << 23) - __float_as_uint(unit));
}
// p and its extrema: |p| is peak[i] at at[i] > 0 (at: infinite where there is none).
struct NsCurve {
  float a, b, c, at[2], peak[2];
};
static NsCurve ns_curve(float a, float b, float c) {
  NsCurve p{a, b, c, {INFINITY, INFINITY}, {0.f, 0.f}};
  // a + 3 b t + 5 c t^2 = 0, t = v^2, by the larger root's form without cancellation
  const double d = 9.0 * b * b - 20.0 * (double)a * c;
  const double q = -0.5 * (3.0 * b + std::copysign(std::sqrt(std::max(d, 0.0)), (double)b));
  const double roots[2] = {c != 0.f ? q / (5.0 * c) : 0.0, q != 0.0 ? a / q : 0.0};
  if (d >= 0.0)
    for (int i = 0; i < 2; ++i)
      if (roots[i] > 0.0 && std::isfinite(roots[i])) {
        const double t = roots[i], v = std::sqrt(t);
        p.at[i] = (float)v;
        p.peak[i] = (float)std::fabs(v * (a + t * (b + t * c)));
      }
  return p;
}
// The bound after a step. Past 2 it stays there (p reaches past 2 up to 2), and j with it at zero.
__device__ __forceinline__ float ns_next_bound(float u, const NsCurve& p) {
  const float t = u * u;
  float v = fabsf(u * (p.a + t * (p.b + t * p.c)));
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (p.at[i] < u) v = fmaxf(v, p.peak[i]);
  return fminf(v, 2.f);
}

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16)
              : reinterpret_cast<const float*>(p)[i];
}

// Eight consecutive values, the first at a multiple of 8.
__device__ __forceinline__ void load8(const void* p, int64_t i, bool bf16, float* v) {
  if (bf16) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = bf16_lo(w[q]);
      v[2 * q + 1] = bf16_hi(w[q]);
    }
  } else {
    const auto* f = reinterpret_cast<const floatx4*>(reinterpret_cast<const float*>(p) + i);
    const floatx4 a = f[0], b = f[1];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = a[q];
      v[q + 4] = b[q];
    }
  }
}

// Partial sums of squares, in 64 bits so that no finite input overflows or vanishes. Matrices of a
// multiple of 8 values are read 16 bytes (fp32: 32) at a time.
__global__ __launch_bounds__(256) void ns_norm_kernel(const void* __restrict__ g, int g_bf16,
                                                      int64_t count, double* __restrict__ parts) {
  __shared__ double red[4];
  const int64_t base = (int64_t)blockIdx.y * count;
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  double s = 0.0;
  if ((count & 7) == 0) {
    for (int64_t i = first; i < count / 8; i += step) {
      float v[8];
      load8(g, base + 8 * i, g_bf16, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) s += (double)v[q] * v[q];
    }
  } else {
    for (int64_t i = first; i < count; i += step) {
      const double v = load_as_f32(g, base + i, g_bf16);
      s += v * v;
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    parts[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = ((red[0] + red[1]) + red[2]) + red[3];
}

// hi + lo = G * scale * 2^j / (norm + eps), laid out [m][ld] along the shorter side, zeros in the
// padding, and units[mat][k] = 2^-j of every step k. 64 x 64 tiles through LDS.
__global__ __launch_bounds__(256) void ns_init_kernel(const void* __restrict__ g, int g_bf16,
                                                      int rows, int cols, int tall, int m, int ld,
                                                      const double* __restrict__ parts, int n_parts,
                                                      float scale, float eps, int steps,
                                                      NsCurve curve, float* __restrict__ units,
                                                      _Float16* __restrict__ hi,
                                                      _Float16* __restrict__ lo) {
  __shared__ float tile[64][65];
  const int lane = threadIdx.x & 63;
  const int64_t mat = blockIdx.z;
  double s = 0.0;
#pragma unroll
  for (int p = 0; p < kNormParts / 64; ++p)
    if (64 * p + lane < n_parts) s += parts[mat * n_parts + 64 * p + lane];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
  const double den = sqrt(s) + (double)eps;
  double mul = den > 0.0 ? (double)scale / den : 0.0;   // a zero matrix stays zero
  float u = (float)(mul * sqrt(s)) * (1.f / scale);
  mul *= pow2_inverse(ns_unit(u));
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    for (int k = 0; k < steps; ++k) {
      units[mat * kNsMaxSteps + k] = ns_unit(u);
      u = ns_next_bound(u, curve);
    }
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;   // tile origin in X
  // X(r, c) = G(r, c), or G(c, r) when tall; the tile's rows of G are gr0.., its columns gc0..
  const int gr0 = tall ? c0 : r0, gc0 = tall ? r0 : c0;
  const bool by8 = (cols & 7) == 0;   // then rows start at multiples of 8 values
#pragma unroll
  for (int it = 0; it < 2; ++it) {   // a thread reads eight values of one row of G
    const int i = it * 32 + (threadIdx.x >> 3), c8 = 8 * (threadIdx.x & 7);
    const int gr = gr0 + i, gc = gc0 + c8;
    float v[8] = {};
    if (gr < rows && gc < cols) {
      const int64_t at = mat * rows * cols + (int64_t)gr * cols + gc;
      if (by8) {
        load8(g, at, g_bf16, v);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (gc + q < cols) v[q] = load_as_f32(g, at + q, g_bf16);
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float x = (float)(v[q] * mul);
      if (tall)
        tile[c8 + q][i] = x;
      else
        tile[i][c8 + q] = x;
    }
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    const int i = it * 32 + (threadIdx.x >> 3), c8 = 8 * (threadIdx.x & 7);
    const int r = r0 + i, c = c0 + c8;
    if (r < m && c < ld) {   // ld % 8 == 0; columns n .. ld - 1 lie outside G: zero
      f16x8 h, l;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float x = tile[i][c8 + q];
        h[q] = (_Float16)x;
        l[q] = (_Float16)(x - (float)h[q]);
      }
      const int64_t at = (mat * m + r) * ld + c;
      *reinterpret_cast<f16x8*>(hi + at) = h;
      *reinterpret_cast<f16x8*>(lo + at) = l;
    }
  }
}

// Two values rounded to fp16, to nearest even.
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, (f16x2{(_Float16)a, (_Float16)b}));
}
__device__ __forceinline__ f16x8 load_f16x8(const _Float16* p) {
  return *reinterpret_cast<const f16x8*>(p);
}

// Lane b of each four holds row b of a 4 x 4 matrix of 16-bit values (r0: columns 0, 1; r1: 2, 3);
// afterwards it holds column b.
__device__ __forceinline__ u32x2 quad_transpose(uint32_t r0, uint32_t r1, int lane) {
  auto from = [](uint32_t v, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, decltype(ctrl)::value, 0xf, 0xf, true);
  };
  using Xor1 = std::integral_constant<int, 0xB1>;   // quad_perm 1, 0, 3, 2
  using Xor2 = std::integral_constant<int, 0x4E>;   // quad_perm 2, 3, 0, 1
  const uint32_t sel = lane & 1 ? 0x03020706u : 0x05040100u;
  const uint32_t s0 = __builtin_amdgcn_perm(from(r0, Xor1{}), r0, sel);
  const uint32_t s1 = __builtin_amdgcn_perm(from(r1, Xor1{}), r1, sel);
  const bool low = (lane & 2) == 0;
  const uint32_t t = from(low ? s1 : s0, Xor2{});
  return low ? u32x2{s0, t} : u32x2{t, s1};
}

// Row i, column j <= i of the lower triangle's tile t.
__device__ __forceinline__ void triangle_tile(int t, int& i, int& j) {
  i = (int)((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);
  while (i * (i + 1) / 2 > t) --i;
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  j = t - i * (i + 1) / 2;
}

// D = X X^T of `x` [m][ld] (contraction over k values of each row): tiles on or under the diagonal,
// written to both halves of out [m][mp], the mirrored one in 8-byte pieces after a 4 x 4 transpose
// between neighbouring lanes (both halves through LDS in long rows: 14 us a 256 x 256 tile slower).
//   POLY = false: out = D * c0                               (x = hi: A)
//   POLY = true:  out = b x + D * c0 + ident on the diagonal (x = A:  B + s I), with A's factor 4^j
//                 taken out of b and c0 (`unit` points to the step's 2^-j of the first matrix)
template <class S, bool POLY>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void ns_gram_kernel(
    const _Float16* __restrict__ x, _Float16* __restrict__ out, int m, int mp, int ld, int k,
    int per, int total, float c0, float b, float ident, const float* __restrict__ unit) {
  static_assert(S::BM == S::BN, "square tiles");
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int v = xcd_tile(blockIdx.x, total);
  if (v < 0) return;
  const int mat = v / per;
  if constexpr (POLY) {
    const float i1 = unit[(int64_t)mat * kNsMaxSteps], i2 = i1 * i1;   // 4^-j
    b *= i2;
    c0 = c0 * i2 * i2;
  }
  int ti, tj;
  triangle_tile(v % per, ti, tj);
  const int row0 = uniform(ti) * S::BM, col0 = uniform(tj) * S::BN;
  const _Float16* xm = x + (int64_t)mat * m * ld;
  const int64_t ldb = (int64_t)ld * 2;
  OperandLoader<S::BM, S::kWaves, false> la;
  OperandLoader<S::BN, S::kWaves, false> lb;
  const auto* xb = reinterpret_cast<const unsigned char*>(xm);
  la.init({xb + row0 * ldb, ldb, min(S::BM, m - row0), 0}, wave, lane);
  lb.init({xb + col0 * ldb, ldb, min(S::BN, m - col0), 0}, wave, lane);
  floatx4 acc[S::FM][S::FN];
  tile_zero<S>(acc);
  tile_kloop<S, false, false, true, S::FM>(la, lb, k, smem, wave, lane, acc);
  _Float16* om = out + (int64_t)mat * m * mp;
  // A's values of half the row sub-tiles are read together, ahead of their use: one at a time, their
  // latencies took as long as the products
  const int g = lane >> 4;
  const int dn0 = col0 + 16 * (wave % S::WN * S::FN) + 4 * g;
  constexpr int kBatch = S::FM / 2;
#pragma unroll
  for (int i0 = 0; i0 < S::FM; i0 += kBatch) {
    f16x4 a[kBatch][S::FN];
    if constexpr (POLY) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int j = 0; j < S::FN; ++j) {
          const int r = row0 + 16 * S::row_tile(wave / S::WN, i0 + i) + (lane & 15);
          const int c = dn0 + 16 * j;
          // outside the matrix any value inside it does: its result is not stored
          a[i][j] = *reinterpret_cast<const f16x4*>(xm + (int64_t)min(r, m - 1) * ld +
                                                    min(c, mp - 4));
        }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        const int r = row0 + 16 * S::row_tile(wave / S::WN, i0 + i) + (lane & 15);
        const int c = dn0 + 16 * j;
        floatx4 v = acc[i0 + i][j] * c0;   // zero in rows and columns from m on
        if constexpr (POLY) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[q] += b * (float)a[i][j][q] + (r == c + q ? ident : 0.f);
            if (r >= m || c + q >= m) v[q] = 0.f;
          }
        }
        const u32x2 h{pack_f16(v.x, v.y), pack_f16(v.z, v.w)};
        if (r < m && c < mp) *reinterpret_cast<u32x2*>(om + (int64_t)r * mp + c) = h;
        if (row0 != col0) {
          const u32x2 t = quad_transpose(h.x, h.y, lane);   // row c + lane % 4, columns r - r % 4 ..
          const int mr = c + (lane & 3), mc = r - (lane & 3);
          if (mr < m && mc < mp) *reinterpret_cast<u32x2*>(om + (int64_t)mr * mp + mc) = t;
        }
      }
  }
}

// Part of A's sums for a matrix whose tiles leave most CUs idle: the contraction is cut into `parts`
// of kp values, and part p of tile t goes to sums[(mat * per + t) * parts + p] (BM x BN fp32).
template <class S>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void ns_gram_part_kernel(
    const _Float16* __restrict__ x, float* __restrict__ sums, int m, int ld, int k, int per,
    int parts, int kp) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = blockIdx.x % parts, tile = blockIdx.x / parts % per;
  const int mat = blockIdx.x / parts / per;
  int ti, tj;
  triangle_tile(tile, ti, tj);
  const int row0 = uniform(ti) * S::BM, col0 = uniform(tj) * S::BN;
  const int64_t ldb = (int64_t)ld * 2;
  const auto* xb = reinterpret_cast<const unsigned char*>(x + (int64_t)mat * m * ld + part * kp);
  OperandLoader<S::BM, S::kWaves, false> la;
  OperandLoader<S::BN, S::kWaves, false> lb;
  // (a part's last row may reach past the matrix by the offset of the part: its loads past k are
  // kept out by k, not by the buffer's end)
  la.init({xb + row0 * ldb, ldb, min(S::BM, m - row0), 0}, wave, lane);
  lb.init({xb + col0 * ldb, ldb, min(S::BN, m - col0), 0}, wave, lane);
  floatx4 acc[S::FM][S::FN];
  tile_zero<S>(acc);
  tile_kloop<S, false, false, true, S::FM>(la, lb, min(kp, k - part * kp), smem, wave, lane, acc);
  float* o = sums + (int64_t)blockIdx.x * (S::BM * S::BN);
  tile_rows<S, S::FM, 4>(
      smem, wave, lane,
      [&](int i, int j, unsigned char* p) { *reinterpret_cast<floatx4*>(p) = acc[i][j]; },
      [&](int m, int n, const unsigned char* p) {
        *reinterpret_cast<floatx4*>(o + m * S::BN + n) = *reinterpret_cast<const floatx4*>(p);
      });
}

// A = c0 * the parts' sum, in part order, to both halves. A workgroup per quarter of a tile.
template <class S>
__global__ __launch_bounds__(256) void ns_gram_sum_kernel(const float* __restrict__ sums,
                                                          _Float16* __restrict__ out, int m, int mp,
                                                          int per, int parts, float c0) {
  const int lane = threadIdx.x & 63;
  const int tile = blockIdx.x / 4 % per, mat = blockIdx.x / 4 / per;
  int ti, tj;
  triangle_tile(tile, ti, tj);
  constexpr int kQuads = S::BN / 4;   // runs of four columns of a row
  static_assert(S::BM * kQuads == 4 * 256, "one run a thread");
  // 16 rows by 4 runs a wave, as a sub-tile's accumulators lie
  const int sub = blockIdx.x % 4 * 4 + (threadIdx.x >> 6);
  const int dm = sub / (S::BN / 16) * 16 + (lane & 15);
  const int dn = sub % (S::BN / 16) * 16 + 4 * (lane >> 4);
  const float* p = sums + ((int64_t)mat * per + tile) * parts * (S::BM * S::BN) + dm * S::BN + dn;
  floatx4 v = *reinterpret_cast<const floatx4*>(p);
#pragma unroll 8
  for (int i = 1; i < parts; ++i)
    v += *reinterpret_cast<const floatx4*>(p + (int64_t)i * (S::BM * S::BN));
  v = v * c0;
  _Float16* om = out + (int64_t)mat * m * mp;
  const int r = ti * S::BM + dm, c = tj * S::BN + dn;
  const u32x2 h{pack_f16(v.x, v.y), pack_f16(v.z, v.w)};
  if (r < m && c < mp) *reinterpret_cast<u32x2*>(om + (int64_t)r * mp + c) = h;
  if (ti != tj) {
    const u32x2 t = quad_transpose(h.x, h.y, lane);
    const int mr = c + (lane & 3), mc = r - (lane & 3);
    if (mr < m && mc < mp) *reinterpret_cast<u32x2*>(om + (int64_t)mr * mp + mc) = t;
  }
}

// X' = c_lo lo + c_hi hi + c_prod (B + s I) hi, as hi' + lo', or, in the last step, rounded to bf16
// into `out` in G's own layout; `rescale` is the next step's 2^j over this one's (in the last step, 2^-j
// times c_out).
template <class S, bool LAST>
__device__ __forceinline__ void ns_update_tile(
    const _Float16* __restrict__ bmat, const _Float16* __restrict__ hi, _Float16* lo,
    _Float16* __restrict__ hi_out, uint16_t* __restrict__ out, int m, int mp, int n, int ld,
    float c_prod, float c_hi, float c_lo, float rescale, int tall, int mat, int row0, int col0,
    unsigned char* smem, int wave, int lane) {
  const int64_t x0 = (int64_t)mat * m * ld;
  OperandLoader<S::BM, S::kWaves, false> la;
  OperandLoader<S::BN, S::kWaves, true> lb;
  la.init({reinterpret_cast<const unsigned char*>(bmat + (int64_t)mat * m * mp) +
               (int64_t)row0 * mp * 2,
           (int64_t)mp * 2, min(S::BM, m - row0), 0},
          wave, lane);
  lb.init({reinterpret_cast<const unsigned char*>(hi + x0 + col0), (int64_t)ld * 2, 0,
           (ld - col0) * 2},
          wave, lane);
  floatx4 acc[S::FM][S::FN];
  tile_zero<S>(acc);
  tile_kloop<S, false, true, true, S::FM>(la, lb, m, smem, wave, lane, acc);
  if constexpr (LAST) {
    if (tall) {   // G's rows are X's columns: as the accumulators lie, 4 x 4 transposed between lanes
      const int r0 = row0 + (lane & 15), c0 = col0 + 16 * (wave % S::WN * S::FN) + 4 * (lane >> 4);
      f16x4 h[S::FM][S::FN], l[S::FM][S::FN];
      auto fetch = [&](int i) {   // clamped into the matrix; outside, the result is not stored
        const int r = min(r0 + 16 * S::row_tile(wave / S::WN, i), m - 1);
#pragma unroll
        for (int j = 0; j < S::FN; ++j) {
          const int64_t at = x0 + (int64_t)r * ld + min(c0 + 16 * j, ld - 4);
          h[i][j] = *reinterpret_cast<const f16x4*>(hi + at);
          l[i][j] = *reinterpret_cast<const f16x4*>(lo + at);
        }
      };
      uint16_t* o = out + (int64_t)mat * m * n;
      constexpr int kAhead = S::FM < 2 ? S::FM : 2;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(i);
#pragma unroll
      for (int i = 0; i < S::FM; ++i) {
        if (i + kAhead < S::FM) fetch(i + kAhead);
        const int r = r0 + 16 * S::row_tile(wave / S::WN, i) - (lane & 3);
#pragma unroll
        for (int j = 0; j < S::FN; ++j) {
          floatx4 v;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            v[q] = rescale * (c_prod * acc[i][j][q] + c_hi * (float)h[i][j][q] +
                              c_lo * (float)l[i][j][q]);
          // row c + lane % 4 of G's layout, columns r .. r + 3
          const u32x2 t = quad_transpose(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w), lane);
          const int c = c0 + 16 * j + (lane & 3);
          if (c >= n || r >= m) continue;
          const int64_t at = (int64_t)c * m + r;
          if ((m & 3) == 0) {
            *reinterpret_cast<u32x2*>(o + at) = t;
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (r + q < m) o[at + q] = (uint16_t)(t[q >> 1] >> (16 * (q & 1)));
          }
        }
      }
      return;
    }
  }
  // in row order, four values a lane; hi and lo of the next two sub-tiles' rows are under way while
  // one's are used
  constexpr int kChunks = S::FN * 4, kRows = 64 / kChunks, kParts = 16 / kRows;
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int dr = lane / kChunks, c = col0 + wn * S::FN * 16 + lane % kChunks * 4;
  auto place = [&](int i, int p) {   // clamped into the matrix; outside, the result is not stored
    const int r = row0 + 16 * S::row_tile(wm, i) + p * kRows + dr;
    return x0 + (int64_t)min(r, m - 1) * ld + min(c, ld - 4);
  };
  f16x4 h[S::FM][kParts], l[S::FM][kParts];
  auto fetch = [&](int i) {
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      h[i][p] = *reinterpret_cast<const f16x4*>(hi + place(i, p));
      l[i][p] = *reinterpret_cast<const f16x4*>(lo + place(i, p));
    }
  };
  constexpr int kAhead = S::FM < 2 ? S::FM : 2;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(i);
  int step = 0;   // sub-tile and part that the next get is for: get is called in that order
  tile_rows<S, S::FM, 4>(
      smem, wave, lane,
      [&](int i, int j, unsigned char* p) {
        if (j == 0 && i + kAhead < S::FM) fetch(i + kAhead);
        *reinterpret_cast<floatx4*>(p) = acc[i][j];
      },
      [&](int dm, int dn, const unsigned char* p) {
        const int i = step / kParts, part = step % kParts;
        ++step;
        const int r = row0 + dm;
        floatx4 v = *reinterpret_cast<const floatx4*>(p);
        const f16x4 hv = h[i][part], lv = l[i][part];
        if (r >= m || c >= ld) return;   // ld % 8 == 0: four columns are all in or all out
#pragma unroll
        for (int q = 0; q < 4; ++q)   // zero in columns n .. ld - 1
          v[q] = rescale * (c_prod * v[q] + c_hi * (float)hv[q] + c_lo * (float)lv[q]);
        if constexpr (!LAST) {
          const int64_t at = x0 + (int64_t)r * ld + c;
          const f16x4 nh{(_Float16)v.x, (_Float16)v.y, (_Float16)v.z, (_Float16)v.w};
          f16x4 nl;
#pragma unroll
          for (int q = 0; q < 4; ++q) nl[q] = (_Float16)(v[q] - (float)nh[q]);
          *reinterpret_cast<f16x4*>(hi_out + at) = nh;
          *reinterpret_cast<f16x4*>(lo + at) = nl;
        } else if ((n & 3) == 0) {   // 8-byte aligned rows, four columns in or out
          if (c < n)
            *reinterpret_cast<u32x2*>(out + ((int64_t)mat * m + r) * n + c) =
                u32x2{pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)};
        } else {
          uint16_t* o = out + (int64_t)mat * m * n;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (c + q < n) o[(int64_t)r * n + c + q] = (uint16_t)pack_bf16(v[q], 0.f);
        }
      });
}

template <class S, bool LAST>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void ns_update_kernel(
    const _Float16* __restrict__ bmat, const _Float16* __restrict__ hi, _Float16* lo,
    _Float16* __restrict__ hi_out, uint16_t* __restrict__ out, int m, int mp, int n, int ld,
    int n_mtiles, int n_ctiles, int total, float c_prod, float c_hi, float c_lo, float c_out,
    int tall, const float* __restrict__ unit) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int half;
  const int v = xcd_tile_halves<S>(blockIdx.x, total, half);
  if (v < 0) return;
  const int mat = v / (n_mtiles * n_ctiles), t = v % (n_mtiles * n_ctiles);
  const int row0 = t % n_mtiles * S::BM, col0 = t / n_mtiles * S::BN;
  const float* const u = unit + (int64_t)mat * kNsMaxSteps;
  const float rescale = LAST ? c_out * u[0] : u[0] * pow2_inverse(u[1]);   // exact
  if constexpr (kHalves<S>) {
    if (half >= 0) {
      const int c = col0 + half * (S::BN / 2);
      if (c < ld)
        ns_update_tile<HalfTile<S>, LAST>(bmat, hi, lo, hi_out, out, m, mp, n, ld, c_prod, c_hi, c_lo,
                                          rescale, tall, mat, row0, c, smem, wave, lane);
      return;
    }
  }
  ns_update_tile<S, LAST>(bmat, hi, lo, hi_out, out, m, mp, n, ld, c_prod, c_hi, c_lo, rescale, tall,
                          mat, row0, col0, smem, wave, lane);
}

// Small matrices: all steps in one launch, a workgroup a matrix of up to 16 MT rows and 128 NJ columns.
// X stays in registers in 32 bits (wave w holds column tiles w, w + 8, ...), its fp16 half for the
// products in LDS, where A and B lie too; each wave computes an eighth of their sub-tiles. The
// formats and scales are those above, with X itself in lo's place. Bound by latency: one matrix, five
// steps (in brackets a launch a product), 64 x 512 31 us (80), 64 x 1024 55 (85), 128 x 256 43 (80),
// 128 x 384 61 (86); 500 of 128 x 384 133 (415). Larger ones need more registers or LDS than a CU has.
constexpr int kSmallWaves = 8;

struct NsSmallArgs {
  const void* g;
  uint16_t* out;
  int g_bf16, tall, m, n, steps;
  NsCurve curve;
  float ident, eps, scale;
};

template <int MT, int NJ>
__global__ __launch_bounds__(64 * kSmallWaves) void ns_small_kernel(NsSmallArgs p) {
  constexpr int kM = 16 * MT;
  constexpr int kPitch = 2 * 128 * NJ + 16, kSquarePitch = 2 * kM + 16;   // bytes
  constexpr int kSquare = kM * kSquarePitch;
  constexpr bool kOneSquare = MT > 4;   // LDS holds one of A and B
  __shared__ __attribute__((aligned(16))) unsigned char
      smem[kM * kPitch + (kOneSquare ? 1 : 2) * kSquare + 8 * kSmallWaves];
  unsigned char* const xs = smem;
  unsigned char* const as = xs + kM * kPitch;
  unsigned char* const bs = kOneSquare ? as : as + kSquare;
  double* const red = reinterpret_cast<double*>(bs + kSquare);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r15 = lane & 15, g = lane >> 4;
  const int m = p.m, n = p.n;
  const int64_t base = (int64_t)blockIdx.x * m * n;
  const int tiles = (n + 31) / 32 * 2;   // 16-column tiles, whole steps of 32
  auto col_tile = [&](int j) { return j * kSmallWaves + wave; };

  // x[i][j]: rows 16 i + lane % 16, columns 16 col_tile(j) + 4 (lane / 16) + 0..3
  floatx4 x[MT][NJ];
  double s = 0.0;
  const bool by4 = !p.tall && (n & 3) == 0;   // then four columns are all in or all out, and aligned
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int r = 16 * i + r15, c = 16 * col_tile(j) + 4 * g;
      x[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
      if (r >= m || c >= n) continue;
      if (by4) {
        const int64_t at = base + (int64_t)r * n + c;
        if (p.g_bf16) {
          const u32x2 v = *reinterpret_cast<const u32x2*>(reinterpret_cast<const uint16_t*>(p.g) + at);
          x[i][j] = floatx4{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
        } else {
          x[i][j] = *reinterpret_cast<const floatx4*>(reinterpret_cast<const float*>(p.g) + at);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c + q < n)
            x[i][j][q] =
                load_as_f32(p.g, base + (p.tall ? (int64_t)(c + q) * m + r : (int64_t)r * n + c + q),
                            p.g_bf16);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) s += (double)x[i][j][q] * x[i][j][q];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
  if (lane == 0) red[wave] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < kSmallWaves; ++w) s += red[w];
  const double den = sqrt(s) + (double)p.eps;
  double mul = den > 0.0 ? (double)p.scale / den : 0.0;   // a zero matrix stays zero
  const float back = 1.f / p.scale;
  float bound = uniform((float)(mul * sqrt(s)) * back);
  float unit = uniform(ns_unit(bound));   // 2^-j
  mul *= pow2_inverse(unit);
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v = x[i][j][q];
        asm volatile("" : "+v"(v));   // or the 64-bit values of the sum above stay in registers
        x[i][j][q] = (float)(v * mul);
      }

  // the wave's sub-tiles of A and B: T of a row
  constexpr int T = MT * MT / kSmallWaves, kRowWaves = MT / T;
  const int r = 16 * (wave / kRowWaves) + r15, ct = wave % kRowWaves * T;
  auto frag = [&](const unsigned char* at) { return *reinterpret_cast<const intx4*>(at); };
  for (int step = 0; step < p.steps; ++step) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (col_tile(j) < tiles)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          *reinterpret_cast<u32x2*>(xs + (16 * i + r15) * kPitch + 32 * col_tile(j) + 8 * g) =
              u32x2{pack_f16(x[i][j].x, x[i][j].y), pack_f16(x[i][j].z, x[i][j].w)};
    __syncthreads();
    // A
    floatx4 d[T] = {};
#pragma unroll 2
    for (int k = 0; k < tiles / 2; ++k) {
      const intx4 fa = frag(xs + r * kPitch + 64 * k + 16 * g);
#pragma unroll
      for (int t = 0; t < T; ++t)
        d[t] = tile_mma<true>(
            frag(xs + (16 * (ct + t) + r15) * kPitch + 64 * k + 16 * g), fa, d[t]);
    }
    const float c0 = kGramScale / (p.scale * p.scale);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int c = 16 * (ct + t) + 4 * g;
      *reinterpret_cast<u32x2*>(as + r * kSquarePitch + 2 * c) =
          u32x2{pack_f16(d[t].x * c0, d[t].y * c0), pack_f16(d[t].z * c0, d[t].w * c0)};
    }
    __syncthreads();
    // B + s I
    const float i2 = unit * unit, pb = uniform(p.curve.b * i2),
                pc = uniform(p.curve.c / kGramScale * i2 * i2);
    u32x2 h[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int c = 16 * (ct + t) + 4 * g;
      floatx4 e = {};
#pragma unroll
      for (int k = 0; k < kM / 32; ++k)
        e = tile_mma<true>(
            frag(as + (16 * (ct + t) + r15) * kSquarePitch + 64 * k + 16 * g),
            frag(as + r * kSquarePitch + 64 * k + 16 * g), e);
      const f16x4 a = *reinterpret_cast<const f16x4*>(as + r * kSquarePitch + 2 * c);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        e[q] = pc * e[q] + pb * (float)a[q] + (r == c + q ? p.ident * kGramScale : 0.f);
      h[t] = u32x2{pack_f16(e.x, e.y), pack_f16(e.z, e.w)};
    }
    if constexpr (kOneSquare) __syncthreads();   // A is read
#pragma unroll
    for (int t = 0; t < T; ++t)
      *reinterpret_cast<u32x2*>(bs + r * kSquarePitch + 32 * (ct + t) + 8 * g) = h[t];
    __syncthreads();
    // X
    const bool last = step + 1 == p.steps;
    bound = ns_next_bound(bound, p.curve);
    const float next = last ? 1.f : uniform(ns_unit(bound)), rescale = unit * pow2_inverse(next);   // exact
    const float c_prod = rescale / kGramScale, ca = rescale * p.curve.a, cs = rescale * p.ident;
    unit = next;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (col_tile(j) >= tiles) continue;
      floatx4 u[MT] = {};
#pragma unroll
      for (int k = 0; k < kM / 32; ++k) {
        // columns across the contraction: transposing reads of rows 32 k + 8 g + 0..3 and 4..7
        const unsigned char* at = xs + (32 * k + 8 * g + (r15 >> 2)) * kPitch +
                                  32 * col_tile(j) + 8 * (r15 & 3);
        const u32x2 lo = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at));
        const u32x2 hi = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * kPitch)));
        const intx4 fx{(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
#pragma unroll
        for (int i = 0; i < MT; ++i)
          u[i] = tile_mma<true>(fx, frag(bs + (16 * i + r15) * kSquarePitch + 64 * k + 16 * g), u[i]);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float v = x[i][j][q], h = (float)(_Float16)v;
          // a X - s hi + (B + s I) hi, or, in the last step, (a - s) X + (B + s I) hi
          x[i][j][q] = u[i][q] * c_prod + ca * v - cs * (last ? v : h);
        }
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int ro = 16 * i + r15, co = 16 * col_tile(j) + 4 * g;
      if (ro >= m || co >= n) continue;
      const floatx4 v = x[i][j] * back;
      if (by4) {
        *reinterpret_cast<u32x2*>(p.out + base + (int64_t)ro * n + co) =
            u32x2{pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)};
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (co + q < n)
            p.out[base + (p.tall ? (int64_t)(co + q) * m + ro : (int64_t)ro * n + co + q)] =
                (uint16_t)pack_bf16(v[q], 0.f);
      }
    }
  }
}

template <class F>
static void with_ns_small(int m, int n, F&& f) {
  using std::integral_constant;
  if (m <= 64)
    n <= 512 ? f(integral_constant<int, 4>{}, integral_constant<int, 4>{})
             : f(integral_constant<int, 4>{}, integral_constant<int, 8>{});
  else
    n <= 256 ? f(integral_constant<int, 8>{}, integral_constant<int, 2>{})
             : f(integral_constant<int, 8>{}, integral_constant<int, 3>{});
}

// ---- host side -----------------------------------------------------------------------------------
hipError_t launch_orthogonalise(const void* g, bool g_bf16, uint16_t* out, int n_mats, int rows,
                                int cols, int steps, const float* coeffs, float eps, char* ws,
                                hipStream_t st) {
  const NsLayout L = ns_layout(n_mats, rows, cols);
  double* norm_parts = reinterpret_cast<double*>(ws + L.parts);
  float* units = reinterpret_cast<float*>(ws + L.units);
  _Float16* hi[2] = {reinterpret_cast<_Float16*>(ws + L.hi[0]),
                     reinterpret_cast<_Float16*>(ws + L.hi[1])};
  _Float16* lo = reinterpret_cast<_Float16*>(ws + L.lo);
  _Float16* gram = reinterpret_cast<_Float16*>(ws + L.gram);
  _Float16* poly = reinterpret_cast<_Float16*>(ws + L.poly);
  const float a = coeffs[0], b = coeffs[1], c = coeffs[2];
  const NsCurve curve = ns_curve(a, b, c);
  const float sx = x_scale(L.n);
  const float ident = std::round(-(b + c) * 4.f) / 4.f;   // exact in fp16 at the stored scale
  if (ns_is_small(L.m, L.n)) {
    with_ns_small(L.m, L.n, [&](auto mt, auto nj) {
      hipLaunchKernelGGL((ns_small_kernel<decltype(mt)::value, decltype(nj)::value>), dim3(n_mats),
                         dim3(64 * kSmallWaves), 0, st,
                         NsSmallArgs{g, out, g_bf16, L.tall, L.m, L.n, steps, curve, ident, eps, sx});
    });
    return hipGetLastError();
  }
  const int64_t count = (int64_t)rows * cols;
  const int n_parts = ns_norm_parts(count);
  hipLaunchKernelGGL(ns_norm_kernel, dim3(n_parts, n_mats), dim3(256), 0, st, g, g_bf16, count,
                     norm_parts);
  hipLaunchKernelGGL(ns_init_kernel,
                     dim3((unsigned)ceil_div(L.ld, 64), (unsigned)ceil_div(L.m, 64), n_mats),
                     dim3(256), 0, st, g, g_bf16, rows, cols, L.tall, L.m, L.ld, norm_parts,
                     n_parts, sx, eps, steps, curve, units, hi[0], lo);
  const GramParts split = gram_parts(n_mats, L.m, L.n);
  auto gram_tiles = [&](int side) { return n_mats * ns_triangle(ceil_div(L.m, side)); };
  for (int s = 0; s < steps; ++s) {
    const float c0 = kGramScale / (sx * sx);
    if (split.parts > 1) {
      using S = NsTile64;
      float* sums = reinterpret_cast<float*>(ws + L.sums);
      const int per = (int)ns_triangle(ceil_div(L.m, 64));
      hipLaunchKernelGGL((ns_gram_part_kernel<S>), dim3((unsigned)(n_mats * per * split.parts)),
                         dim3(S::kThreads), 0, st, hi[0], sums, L.m, L.ld, L.n, per, split.parts, split.kp);
      hipLaunchKernelGGL((ns_gram_sum_kernel<S>), dim3((unsigned)(n_mats * per * 4)), dim3(256), 0,
                         st, sums, gram, L.m, L.mp, per, split.parts, c0);
    } else {
      with_ns_tile(false, L.n, gram_tiles, [&](auto tile) {
        using S = decltype(tile);
        hipLaunchKernelGGL((ns_gram_kernel<S, false>), dim3((unsigned)xcd_workgroups(gram_tiles(S::BM))),
                           dim3(S::kThreads), 0, st, hi[0], gram, L.m, L.mp, L.ld, L.n,
                           (int)ns_triangle(ceil_div(L.m, S::BM)), (int)gram_tiles(S::BM), c0, 0.f,
                           0.f, nullptr);
      });
    }
    with_ns_tile(false, L.m, gram_tiles, [&](auto tile) {
      using S = decltype(tile);
      hipLaunchKernelGGL((ns_gram_kernel<S, true>), dim3((unsigned)xcd_workgroups(gram_tiles(S::BM))),
                         dim3(S::kThreads), 0, st, gram, poly, L.m, L.mp, L.mp, L.m,
                         (int)ns_triangle(ceil_div(L.m, S::BM)), (int)gram_tiles(S::BM), c / kGramScale, b,
                         ident * kGramScale, units + s);
    });
    auto update_tiles = [&](int side) { return n_mats * ceil_div(L.m, side) * ceil_div(L.ld, side); };
    with_ns_tile(true, L.m, update_tiles, [&](auto tile) {
      using S = decltype(tile);
      const int mt = (int)ceil_div(L.m, S::BM), ct = (int)ceil_div(L.ld, S::BN);
      auto update = [&](auto last) {
        // lo takes a in every step but the last, a - s there: the error is B lo, which vanishes in
        // weak directions, or (B + s I) lo, which vanishes in converged ones; only the last step's
        // error is not amplified in the weak ones
        constexpr bool kLast = decltype(last)::value;
        hipLaunchKernelGGL((ns_update_kernel<S, kLast>), dim3((unsigned)xcd_workgroups_halves<S>(update_tiles(S::BM))),
                           dim3(S::kThreads), 0, st, poly, hi[0], lo, hi[1], out, L.m, L.mp, L.n,
                           L.ld, mt, ct, (int)update_tiles(S::BM), 1.f / kGramScale, a - ident, kLast ? a - ident : a,
                           1.f / sx, L.tall, units + s);
      };
      if (s + 1 == steps)
        update(std::true_type{});
      else
        update(std::false_type{});
    });
    std::swap(hi[0], hi[1]);
  }
  return hipGetLastError();
}

}  // namespace beam
