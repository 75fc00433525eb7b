// Gradient of the sublayer boundary (gfx950), the backward pass of boundary.hip: next norm -> residual
// add -> output norm, with both norm weights' gradients.
//
// Per token t, roundings passed through as the identity, h' taken as the forward stored it
// ([V] §MoE and residual stream; [S] §Sandwich Normalization and Depth-Scaled Residuals):
//   r2 = 1 / sqrt(mean(h'^2) + eps), g = dx' * gamma_next
//   dh'' = dh' + r2 * (g - h' * r2^2 * mean(g h'));  dgamma_next += dx' * h' * r2
//   dh = alpha * dh'',  dp = beta * dh''
//   r1 = 1 / sqrt(mean(u^2) + eps), u = bf16(y), q = dp * gamma_post
//   dy = r1 * (q - u * r1^2 * mean(q u));  dgamma_post += dp * u * r1
// Two reductions a token: sum h'^2, g h', u^2 together, then q u. A workgroup walks tokens
// blockIdx, + gridDim, ... and keeps its part of both weight gradients in registers; the parts go to
// the workspace and a second launch adds them in workgroup order (deterministic, no atomics).
#include <algorithm>
#include <type_traits>

#include "device_common.h"

namespace beam {

constexpr int kBwdThreads = 256;
constexpr int kBwdMaxParts = 1024;   // workgroups of the first launch
static_assert(kBoundaryMaxHidden == 16 * 4 * kBwdThreads, "register chunks cover every row");

__device__ __forceinline__ floatx4 load_bf16x4(const uint16_t* p) {
  const u32x2 v = *reinterpret_cast<const u32x2*>(p);
  return floatx4{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
}
__device__ __forceinline__ void store_bf16x4(uint16_t* p, floatx4 v) {
  u32x2 o;
  o.x = f32_to_bf16_bits(v.x) | (f32_to_bf16_bits(v.y) << 16);
  o.y = f32_to_bf16_bits(v.z) | (f32_to_bf16_bits(v.w) << 16);
  *reinterpret_cast<u32x2*>(p) = o;
}
__device__ __forceinline__ float dot4(floatx4 a, floatx4 b) {
  return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// CH: chunks of 4 values a thread holds (hidden <= CH * 1024)
template <int CH, bool Y_BF16, bool HAS_DH>
__global__ __launch_bounds__(kBwdThreads) void boundary_bwd_kernel(
    const void* __restrict__ y, const uint16_t* __restrict__ h, const float* __restrict__ gp,
    const float* __restrict__ gn, const uint16_t* dh_in, const uint16_t* __restrict__ dx,
    void* __restrict__ dy, uint16_t* dh_out, float* __restrict__ parts, int64_t T, int H,
    float alpha, float beta, float eps) {
  __shared__ float red[2][4][4];   // [token parity][value][wave]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  floatx4 acc_p[CH], acc_n[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) acc_p[j] = acc_n[j] = floatx4{0.f, 0.f, 0.f, 0.f};
  int par = 0;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x, par ^= 1) {
    floatx4 hv[CH], xv[CH], uv[CH], dv[CH];
    float shh = 0.f, sgh = 0.f, suu = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = 4 * (tid + kBwdThreads * j);
      hv[j] = xv[j] = uv[j] = dv[j] = floatx4{0.f, 0.f, 0.f, 0.f};
      if (c >= H) continue;
      const int64_t at = t * H + c;
      hv[j] = load_bf16x4(h + at);
      xv[j] = load_bf16x4(dx + at);
      if constexpr (Y_BF16) {
        uv[j] = load_bf16x4(reinterpret_cast<const uint16_t*>(y) + at);
      } else {
        const floatx4 v = *reinterpret_cast<const floatx4*>(reinterpret_cast<const float*>(y) + at);
        uv[j] = floatx4{bf16_round(v.x), bf16_round(v.y), bf16_round(v.z), bf16_round(v.w)};
      }
      if constexpr (HAS_DH) dv[j] = load_bf16x4(dh_in + at);
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = 4 * (tid + kBwdThreads * j);
      if (c >= H) continue;
      const floatx4 g = *reinterpret_cast<const floatx4*>(gn + c);
      shh += dot4(hv[j], hv[j]);
      sgh += dot4(xv[j] * g, hv[j]);
      suu += dot4(uv[j], uv[j]);
    }
    shh = wave_sum(shh);
    sgh = wave_sum(sgh);
    suu = wave_sum(suu);
    float(*rd)[4] = red[par];
    if (lane == 0) {
      rd[0][wave] = shh;
      rd[1][wave] = sgh;
      rd[2][wave] = suu;
    }
    __syncthreads();
    const float inv_h = 1.0f / (float)H;
    shh = ((rd[0][0] + rd[0][1]) + rd[0][2]) + rd[0][3];
    sgh = ((rd[1][0] + rd[1][1]) + rd[1][2]) + rd[1][3];
    suu = ((rd[2][0] + rd[2][1]) + rd[2][2]) + rd[2][3];
    const float r2 = 1.0f / sqrtf(shh * inv_h + eps), r1 = 1.0f / sqrtf(suu * inv_h + eps);
    const float k2 = r2 * r2 * (sgh * inv_h);
    float squ = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = 4 * (tid + kBwdThreads * j);
      if (c >= H) continue;
      const floatx4 g = *reinterpret_cast<const floatx4*>(gn + c);
      const floatx4 p = *reinterpret_cast<const floatx4*>(gp + c);
      acc_n[j] += xv[j] * (hv[j] * r2);
      const floatx4 d = dv[j] + r2 * (xv[j] * g - hv[j] * k2);
      store_bf16x4(dh_out + t * H + c, alpha * d);
      const floatx4 dp = beta * d;
      acc_p[j] += dp * (uv[j] * r1);
      dv[j] = dp * p;
      squ += dot4(dv[j], uv[j]);
    }
    squ = wave_sum(squ);
    if (lane == 0) rd[3][wave] = squ;
    __syncthreads();
    squ = ((rd[3][0] + rd[3][1]) + rd[3][2]) + rd[3][3];
    const float k1 = r1 * r1 * (squ * inv_h);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = 4 * (tid + kBwdThreads * j);
      if (c >= H) continue;
      const floatx4 o = r1 * (dv[j] - uv[j] * k1);
      if constexpr (Y_BF16)
        store_bf16x4(reinterpret_cast<uint16_t*>(dy) + t * H + c, o);
      else
        *reinterpret_cast<floatx4*>(reinterpret_cast<float*>(dy) + t * H + c) = o;
    }
  }
  float* mine = parts + (int64_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = 4 * (tid + kBwdThreads * j);
    if (c >= H) continue;
    *reinterpret_cast<floatx4*>(mine + c) = acc_p[j];
    *reinterpret_cast<floatx4*>(mine + H + c) = acc_n[j];
  }
}

// dgamma[c] = sum over the parts, 64 columns a workgroup: 16 rows of 64 threads each add every 16th
// part, then the 16 sums in order.
constexpr int kReduceRows = 16;
__global__ __launch_bounds__(64 * kReduceRows) void gamma_reduce_kernel(
    const float* __restrict__ parts, int n_parts, float* __restrict__ dgp, float* __restrict__ dgn,
    int H) {
  __shared__ float sums[kReduceRows][64];
  const int lane = threadIdx.x & 63, row = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;   // 2 H is a multiple of 64
  float s = 0.f;
  for (int p = row; p < n_parts; p += kReduceRows) s += parts[(int64_t)p * 2 * H + c];
  sums[row][lane] = s;
  __syncthreads();
  if (row == 0) {
    for (int r = 1; r < kReduceRows; ++r) s += sums[r][lane];
    if (c < H)
      dgp[c] = s;
    else
      dgn[c - H] = s;
  }
}

int boundary_bwd_parts(int64_t T) { return (int)std::min<int64_t>(T, kBwdMaxParts); }

hipError_t launch_boundary_bwd(const BoundaryBwdArgs& a, int64_t T, int H, hipStream_t st) {
  const int n_parts = boundary_bwd_parts(T);
  auto go = [&](auto ch_tag) {
    constexpr int CH = decltype(ch_tag)::value;
    auto run = [&](auto yb, auto dh) {
      hipLaunchKernelGGL((boundary_bwd_kernel<CH, decltype(yb)::value, decltype(dh)::value>),
                         dim3(n_parts), dim3(kBwdThreads), 0, st, a.y, a.h, a.gamma_post,
                         a.gamma_next, a.d_h_in, a.d_x, a.d_y, a.d_h, a.parts, T, H, a.alpha,
                         a.beta, a.eps);
    };
    if (a.y_bf16)
      a.d_h_in ? run(std::true_type{}, std::true_type{}) : run(std::true_type{}, std::false_type{});
    else
      a.d_h_in ? run(std::false_type{}, std::true_type{})
               : run(std::false_type{}, std::false_type{});
  };
  const int need = (int)ceil_div(H, 4 * kBwdThreads);
  if (need <= 1)
    go(std::integral_constant<int, 1>{});
  else if (need <= 2)
    go(std::integral_constant<int, 2>{});
  else if (need <= 3)
    go(std::integral_constant<int, 3>{});
  else if (need <= 5)
    go(std::integral_constant<int, 5>{});
  else if (need <= 8)
    go(std::integral_constant<int, 8>{});
  else
    go(std::integral_constant<int, 16>{});
  hipLaunchKernelGGL(gamma_reduce_kernel, dim3(2 * H / 64), dim3(64 * kReduceRows), 0, st, a.parts,
                     n_parts, a.d_gamma_post, a.d_gamma_next, H);
  return hipGetLastError();
}

}  // namespace beam
