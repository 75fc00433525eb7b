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
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gemm_tile.h"

namespace beam {

constexpr int kNormParts = 64;          // partial sums of squares of a matrix
constexpr float kGramScale = 256.f;     // A and B hold 2^8 times their values

// X holds 2^k times its values, 2^k about sqrt(longer side): a matrix of orthonormal rows has entries
// of about 1 / sqrt(longer side).
static float x_scale(int n_long) {
  float s = 1.f;
  while (s * s < (float)n_long) s *= 2.f;
  return s;
}

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, bool bf16) {
  return bf16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16)
              : reinterpret_cast<const float*>(p)[i];
}

// Partial sums of squares, in 64 bits so that no finite input overflows or vanishes.
__global__ __launch_bounds__(256) void ns_norm_kernel(const void* __restrict__ g, int g_bf16,
                                                      int64_t count, double* __restrict__ parts) {
  __shared__ double red[4];
  const int64_t base = (int64_t)blockIdx.y * count;
  double s = 0.0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count;
       i += (int64_t)gridDim.x * 256) {
    const double v = load_as_f32(g, base + i, g_bf16);
    s += v * v;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    parts[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = ((red[0] + red[1]) + red[2]) + red[3];
}

// hi + lo = G * scale / (norm + eps), laid out [m][ld] along the shorter side, zeros in the padding.
// 64 x 64 tiles through LDS.
__global__ __launch_bounds__(256) void ns_init_kernel(const void* __restrict__ g, int g_bf16,
                                                      int rows, int cols, int tall, int m, int ld,
                                                      const double* __restrict__ parts,
                                                      float scale, float eps,
                                                      _Float16* __restrict__ hi,
                                                      _Float16* __restrict__ lo) {
  __shared__ float tile[64][65];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t mat = blockIdx.z;
  double s = parts[mat * kNormParts + lane];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
  const double den = sqrt(s) + (double)eps;
  const double mul = den > 0.0 ? (double)scale / den : 0.0;   // a zero matrix stays zero
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;   // tile origin in X
  for (int i = wave; i < 64; i += 4) {
    // X(r, c) = G(r, c), or G(c, r) when tall: `lane` runs along G's rows either way
    const int gr = tall ? c0 + i : r0 + i, gc = (tall ? r0 : c0) + lane;
    float v = 0.f;
    if (gr < rows && gc < cols)
      v = (float)(load_as_f32(g, mat * rows * cols + (int64_t)gr * cols + gc, g_bf16) * mul);
    if (tall)
      tile[lane][i] = v;
    else
      tile[i][lane] = v;
  }
  __syncthreads();
  for (int i = wave; i < 64; i += 4) {
    const int r = r0 + i, c = c0 + lane;
    if (r < m && c < ld) {
      const float v = tile[i][lane];   // columns n .. ld - 1 lie outside G: zero
      const _Float16 h = (_Float16)v;
      const int64_t at = (mat * m + r) * ld + c;
      hi[at] = h;
      lo[at] = (_Float16)(v - (float)h);
    }
  }
}

__device__ __forceinline__ f16x4 to_f16x4(floatx4 v) {
  return f16x4{(_Float16)v.x, (_Float16)v.y, (_Float16)v.z, (_Float16)v.w};
}
__device__ __forceinline__ floatx4 from_f16x4(f16x4 v) {
  return floatx4{(float)v.x, (float)v.y, (float)v.z, (float)v.w};
}

// D = X X^T of `x` [m][ld] (contraction over k values of each row): tiles on or under the diagonal,
// written to both halves.
//   POLY = false: out = D * c0                               (x = hi: A)
//   POLY = true:  out = b x + D * c0 + ident on the diagonal (x = A:  B + s I)
template <class S, bool POLY>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void ns_gram_kernel(
    const _Float16* __restrict__ x, _Float16* __restrict__ out, int m, int mp, int ld, int k,
    int n_tiles, int n_mats, float c0, float b, float ident) {
  static_assert(S::BM == S::BN, "square tiles");
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = n_tiles * (n_tiles + 1) / 2;
  const int mat = blockIdx.x / per, t = blockIdx.x % per;
  int i = (int)((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);   // row i of the triangle holds t
  while (i * (i + 1) / 2 > t) --i;
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  const int j = t - i * (i + 1) / 2;
  const int row0 = i * S::BM, col0 = j * S::BN;
  const _Float16* xm = x + (int64_t)mat * m * ld;
  const int64_t ldb = (int64_t)ld * 2;
  OperandLoader<S::BM, S::kWaves, false, S::KT> la;
  OperandLoader<S::BN, S::kWaves, false, S::KT> lb;
  const auto* xb = reinterpret_cast<const unsigned char*>(xm);
  la.init({xb + row0 * ldb, ldb, min(S::BM, m - row0), 0}, wave, lane);
  lb.init({xb + col0 * ldb, ldb, min(S::BN, m - col0), 0}, wave, lane);
  floatx4 acc[S::FM][S::FN];
  tile_zero<S>(acc);
  tile_kloop<S, false, false, true, S::FM>(la, lb, k, smem, wave, lane, acc);
  _Float16* om = out + (int64_t)mat * m * mp;
  tile_for_each<S, S::FM>(acc, wave, lane, [&](int dm, int dn, floatx4 d) {
    const int r = row0 + dm, c = col0 + dn;
    if (r >= mp || c >= mp) return;
    floatx4 v = d * c0;   // zero in rows and columns m .. mp - 1
    if (POLY && r < m) {
      v = v + b * from_f16x4(*reinterpret_cast<const f16x4*>(xm + (int64_t)r * ld + c));
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (r == c + q) v[q] += ident;
    }
    const f16x4 h = to_f16x4(v);
    if (r < m) *reinterpret_cast<f16x4*>(om + (int64_t)r * mp + c) = h;
    if (i != j) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c + q < m) om[(int64_t)(c + q) * mp + r] = h[q];
    }
  });
}

// X' = a lo + (a - s) hi + (B + s I) hi, as hi' + lo', or, in the last step, rounded to bf16 into
// `out` in G's own layout.
template <class S, bool LAST>
__global__ __launch_bounds__(S::kThreads, S::kLdsBytes <= 80 * 1024 ? 2 : 1) void ns_update_kernel(
    const _Float16* __restrict__ bmat, const _Float16* __restrict__ hi, _Float16* lo,
    _Float16* __restrict__ hi_out, uint16_t* __restrict__ out, int m, int mp, int n, int ld,
    int n_mtiles, int n_ctiles, int n_mats, float c_prod, float c_hi, float c_lo, float c_out,
    int tall) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[S::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = n_mtiles * n_ctiles;
  const int mat = blockIdx.x / per, t = blockIdx.x % per;
  const int row0 = t % n_mtiles * S::BM, col0 = t / n_mtiles * S::BN;
  const int64_t x0 = (int64_t)mat * m * ld;
  OperandLoader<S::BM, S::kWaves, false, S::KT> la;
  OperandLoader<S::BN, S::kWaves, true, S::KT> lb;
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
  tile_for_each<S, S::FM>(acc, wave, lane, [&](int dm, int dn, floatx4 d) {
    const int r = row0 + dm, c = col0 + dn;
    if (r >= m || c >= ld) return;
    const int64_t at = x0 + (int64_t)r * ld + c;
    const floatx4 h = from_f16x4(*reinterpret_cast<const f16x4*>(hi + at));
    const floatx4 l = from_f16x4(*reinterpret_cast<const f16x4*>(lo + at));
    const floatx4 v = c_prod * d + c_hi * h + c_lo * l;   // zero in columns n .. ld - 1
    if constexpr (!LAST) {
      const f16x4 nh = to_f16x4(v);
      *reinterpret_cast<f16x4*>(hi_out + at) = nh;
      *reinterpret_cast<f16x4*>(lo + at) = to_f16x4(v - from_f16x4(nh));
    } else {
      const int64_t o0 = (int64_t)mat * m * n;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c + q < n)
          out[o0 + (tall ? (int64_t)(c + q) * m + r : (int64_t)r * n + c + q)] =
              (uint16_t)f32_to_bf16_bits(c_out * v[q]);
    }
  });
}

NsLayout ns_layout(int64_t n_mats, int rows, int cols) {
  NsLayout L;
  L.tall = rows > cols;
  L.m = std::min(rows, cols);
  L.n = std::max(rows, cols);
  L.mp = (L.m + 7) / 8 * 8;
  L.ld = (L.n + 7) / 8 * 8;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) & ~size_t(255);
    return o;
  };
  const size_t x = 2 * (size_t)n_mats * L.m * L.ld, a = 2 * (size_t)n_mats * L.m * L.mp;
  L.parts = take(sizeof(double) * kNormParts * (size_t)n_mats);
  L.hi[0] = take(x);
  L.hi[1] = take(x);
  L.lo = take(x);
  L.gram = take(a);
  L.poly = take(a);
  L.total = off;
  return L;
}

using NsTile = TileShape<128, 128, 2, 2, 2, 2>;

bool ns_grid_fits(int64_t n_mats, int rows, int cols) {
  const int64_t mt = ceil_div(std::min(rows, cols), 128), ct = ceil_div(std::max(rows, cols), 128);
  return n_mats <= 65535 && n_mats * mt * std::max(ct, (mt + 1) / 2) < (int64_t(1) << 31);
}

hipError_t launch_orthogonalise(const void* g, bool g_bf16, uint16_t* out, int n_mats, int rows,
                                int cols, int steps, const float* coeffs, float eps, char* ws,
                                hipStream_t st) {
  const NsLayout L = ns_layout(n_mats, rows, cols);
  double* parts = reinterpret_cast<double*>(ws + L.parts);
  _Float16* hi[2] = {reinterpret_cast<_Float16*>(ws + L.hi[0]),
                     reinterpret_cast<_Float16*>(ws + L.hi[1])};
  _Float16* lo = reinterpret_cast<_Float16*>(ws + L.lo);
  _Float16* gram = reinterpret_cast<_Float16*>(ws + L.gram);
  _Float16* poly = reinterpret_cast<_Float16*>(ws + L.poly);
  const float a = coeffs[0], b = coeffs[1], c = coeffs[2];
  const float sx = x_scale(L.n);
  const float ident = std::round(-(b + c) * 4.f) / 4.f;   // exact in fp16 at the stored scale
  hipLaunchKernelGGL(ns_norm_kernel, dim3(kNormParts, n_mats), dim3(256), 0, st, g, g_bf16,
                     (int64_t)rows * cols, parts);
  hipLaunchKernelGGL(ns_init_kernel,
                     dim3((unsigned)ceil_div(L.ld, 64), (unsigned)ceil_div(L.m, 64), n_mats),
                     dim3(256), 0, st, g, g_bf16, rows, cols, L.tall, L.m, L.ld, parts, sx, eps,
                     hi[0], lo);
  using S = NsTile;
  const int mt = (int)ceil_div(L.m, S::BM), ct = (int)ceil_div(L.ld, S::BN);
  const dim3 gram_grid((unsigned)((int64_t)n_mats * mt * (mt + 1) / 2));
  const dim3 upd_grid((unsigned)((int64_t)n_mats * mt * ct));
  for (int s = 0; s < steps; ++s) {
    hipLaunchKernelGGL((ns_gram_kernel<S, false>), gram_grid, dim3(S::kThreads), 0, st, hi[0], gram,
                       L.m, L.mp, L.ld, L.n, mt, n_mats, kGramScale / (sx * sx), 0.f, 0.f);
    hipLaunchKernelGGL((ns_gram_kernel<S, true>), gram_grid, dim3(S::kThreads), 0, st, gram, poly,
                       L.m, L.mp, L.mp, L.m, mt, n_mats, c / kGramScale, b, ident * kGramScale);
    auto update = [&](auto last) {
      hipLaunchKernelGGL((ns_update_kernel<S, decltype(last)::value>), upd_grid, dim3(S::kThreads),
                         0, st, poly, hi[0], lo, hi[1], out, L.m, L.mp, L.n, L.ld, mt, ct, n_mats,
                         1.f / kGramScale, a - ident, a, 1.f / sx, L.tall);
    };
    if (s + 1 == steps)
      update(std::true_type{});
    else
      update(std::false_type{});
    std::swap(hi[0], hi[1]);
  }
  return hipGetLastError();
}

}  // namespace beam
