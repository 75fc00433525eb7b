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
// Two reductions a token: sum h'^2, g h', u^2 together, then q u. Memory-bound: T H (2 y + 8) bytes.
// A workgroup walks tokens blockIdx, + gridDim, ..., holding a token packed in registers while the
// next one's loads are under way, and keeps its part of both weight gradients in registers; the
// parts go to the workspace and a second launch adds them in workgroup order (deterministic, no
// atomics).
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "train_rules.h"

namespace beam {

static_assert(kBoundaryMaxHidden == 4 * 4 * 1024, "the widest kernel's chunks cover every row");

__device__ __forceinline__ floatx4 unpack_bf16(u32x2 v) {
  return floatx4{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
}
__device__ __forceinline__ u32x2 pack_bf16(floatx4 v) {
  return u32x2{pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)};
}
__device__ __forceinline__ u32x2 pack_bf16(u32x2 v) { return v; }
__device__ __forceinline__ float dot4(floatx4 a, floatx4 b) {
  return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// Barrier that waits for LDS but not, as __syncthreads() would, for the next token's loads.
__device__ __forceinline__ void bwd_barrier() {
  __builtin_amdgcn_s_waitcnt(kLgkmZero);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// TH threads, each with CH chunks of 4 values of the row (hidden <= 4 TH CH). AHEAD: the next token's
// loads and both weights stay in registers (about 230 at CH = 5: two waves a SIMD, 100 KB of loads
// in flight a CU); the widest rows leave no registers for that.
template <int TH, int CH, bool AHEAD, bool Y_BF16, bool HAS_DH>
__global__ __launch_bounds__(TH) void boundary_bwd_kernel(
    const void* __restrict__ y, const uint16_t* __restrict__ h, const float* __restrict__ gp,
    const float* __restrict__ gn, const uint16_t* dh_in, const uint16_t* __restrict__ dx,
    void* __restrict__ dy, uint16_t* dh_out, float* __restrict__ parts, int64_t T, int H,
    float alpha, float beta, float eps) {
  using YChunk = std::conditional_t<Y_BF16, u32x2, floatx4>;
  constexpr int NW = TH / 64;
  __shared__ float red[2][4][NW];   // [token parity][value][wave]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  floatx4 acc_p[CH], acc_n[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) acc_p[j] = acc_n[j] = floatx4{0.f, 0.f, 0.f, 0.f};
  u32x2 nh[CH], nx[CH], nd[CH];   // the next token
  YChunk ny[CH];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = 4 * (tid + TH * j);
      nh[j] = nx[j] = nd[j] = u32x2{0, 0};
      ny[j] = YChunk{};
      if (c >= H) continue;
      const int64_t at = t * H + c;
      nh[j] = *reinterpret_cast<const u32x2*>(h + at);
      nx[j] = *reinterpret_cast<const u32x2*>(dx + at);
      ny[j] = *reinterpret_cast<const YChunk*>(reinterpret_cast<const char*>(y) +
                                               at * (Y_BF16 ? 2 : 4));
      if constexpr (HAS_DH) nd[j] = *reinterpret_cast<const u32x2*>(dh_in + at);
    }
  };
  auto waves_sum = [](const float* v) {
    float a = v[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) a += v[w];
    return a;
  };
  if (AHEAD && blockIdx.x < T) fetch(blockIdx.x);
  int par = 0;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x, par ^= 1) {
    u32x2 hv[CH], xv[CH], uv[CH], dv[CH];
    float shh = 0.f, sgh = 0.f, suu = 0.f;
    if constexpr (!AHEAD) {
      asm volatile("" : "+s"(gp), "+s"(gn));   // keeps the weights' loads inside the loop
      fetch(t);
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      hv[j] = nh[j];
      xv[j] = nx[j];
      dv[j] = nd[j];
      uv[j] = pack_bf16(ny[j]);   // u = bf16(y)
    }
    if (AHEAD && t + gridDim.x < T) fetch(t + gridDim.x);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = 4 * (tid + TH * j);
      if (c >= H) continue;
      const floatx4 g = *reinterpret_cast<const floatx4*>(gn + c);
      const floatx4 hf = unpack_bf16(hv[j]), uf = unpack_bf16(uv[j]);
      shh += dot4(hf, hf);
      sgh += dot4(unpack_bf16(xv[j]) * g, hf);
      suu += dot4(uf, uf);
    }
    shh = wave_sum(shh);
    sgh = wave_sum(sgh);
    suu = wave_sum(suu);
    float(*rd)[NW] = red[par];
    if (lane == 0) {
      rd[0][wave] = shh;
      rd[1][wave] = sgh;
      rd[2][wave] = suu;
    }
    bwd_barrier();
    const float inv_h = 1.0f / (float)H;
    shh = waves_sum(rd[0]);
    sgh = waves_sum(rd[1]);
    suu = waves_sum(rd[2]);
    const float r2 = 1.0f / sqrtf(shh * inv_h + eps), r1 = 1.0f / sqrtf(suu * inv_h + eps);
    const float k2 = r2 * r2 * (sgh * inv_h);
    floatx4 q[CH];
    float squ = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = 4 * (tid + TH * j);
      if (c >= H) continue;
      const floatx4 g = *reinterpret_cast<const floatx4*>(gn + c);
      const floatx4 p = *reinterpret_cast<const floatx4*>(gp + c);
      const floatx4 hf = unpack_bf16(hv[j]), xf = unpack_bf16(xv[j]), uf = unpack_bf16(uv[j]);
      acc_n[j] += xf * (hf * r2);
      const floatx4 d = unpack_bf16(dv[j]) + r2 * (xf * g - hf * k2);
      *reinterpret_cast<u32x2*>(dh_out + t * H + c) = pack_bf16(alpha * d);
      const floatx4 dp = beta * d;
      acc_p[j] += dp * (uf * r1);
      q[j] = dp * p;
      squ += dot4(q[j], uf);
    }
    squ = wave_sum(squ);
    if (lane == 0) rd[3][wave] = squ;
    bwd_barrier();
    squ = waves_sum(rd[3]);
    const float k1 = r1 * r1 * (squ * inv_h);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = 4 * (tid + TH * j);
      if (c >= H) continue;
      const floatx4 o = r1 * (q[j] - unpack_bf16(uv[j]) * k1);
      if constexpr (Y_BF16)
        *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(dy) + t * H + c) = pack_bf16(o);
      else
        *reinterpret_cast<floatx4*>(reinterpret_cast<float*>(dy) + t * H + c) = o;
    }
  }
  float* mine = parts + (int64_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = 4 * (tid + TH * j);
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
#pragma unroll 8
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

hipError_t launch_boundary_bwd(const BoundaryBwdArgs& a, int64_t T, int H, hipStream_t st) {
  const int n_parts = boundary_bwd_parts(T, H);
  auto reduce = [&]() {
    hipLaunchKernelGGL(gamma_reduce_kernel, dim3(2 * H / 64), dim3(64 * kReduceRows), 0, st, a.parts,
                       n_parts, a.d_gamma_post, a.d_gamma_next, H);
  };
  auto go = [&](auto th_tag, auto ch_tag) {
    constexpr int TH = decltype(th_tag)::value, CH = decltype(ch_tag)::value;
    auto run = [&](auto yb, auto dh) {
      hipLaunchKernelGGL((boundary_bwd_kernel<TH, CH, TH <= 512, decltype(yb)::value,
                                              decltype(dh)::value>),
                         dim3(n_parts), dim3(TH), 0, st, a.y, a.h, a.gamma_post, a.gamma_next,
                         a.d_h_in, a.d_x, a.d_y, a.d_h, a.parts, T, H, a.alpha, a.beta, a.eps);
    };
    if (a.y_bf16)
      a.d_h_in ? run(std::true_type{}, std::true_type{}) : run(std::true_type{}, std::false_type{});
    else
      a.d_h_in ? run(std::false_type{}, std::true_type{})
               : run(std::false_type{}, std::false_type{});
  };
  if (n_parts == 0) {   // no tokens: the weights' gradients are sums over nothing
    reduce();
    return hipGetLastError();
  }
  const int th = boundary_bwd_threads(H), need = (int)ceil_div(H, 4 * th);
  auto chunks = [&](auto th_tag) {
    if (need <= 1)
      go(th_tag, std::integral_constant<int, 1>{});
    else if (need <= 2)
      go(th_tag, std::integral_constant<int, 2>{});
    else if (need <= 3)
      go(th_tag, std::integral_constant<int, 3>{});
    else if (need <= 4)
      go(th_tag, std::integral_constant<int, 4>{});
    else
      go(th_tag, std::integral_constant<int, 5>{});
  };
  if (th == 256)
    chunks(std::integral_constant<int, 256>{});
  else if (th == 512)   // need is 3 to 5
    need <= 3   ? go(std::integral_constant<int, 512>{}, std::integral_constant<int, 3>{})
    : need <= 4 ? go(std::integral_constant<int, 512>{}, std::integral_constant<int, 4>{})
                : go(std::integral_constant<int, 512>{}, std::integral_constant<int, 5>{});
  else   // need is 3 or 4
    need <= 3 ? go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 3>{})
              : go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
  reduce();
  return hipGetLastError();
}

}  // namespace beam
