// AdamW step over many tensors at once (gfx950): the weights that the orthogonalised update is not for
// (norms, router, embedding, head) beside it in an optimiser.
//
//   g = grad * grad_scale,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// States in FP32, or in 8 bits: E4M3 values of a scale (amax / 448) that 256 of them share, v by its root,
// which halves its range and gives the divisor twice its digits. m, v, the roots and the values they are
// rounded to are single FP32 operations, each correctly rounded (no fused multiply-adds), so that equal
// inputs give equal states on any machine; p alone uses the hardware's reciprocal (1 ulp).
//
// 8-bit states and bf16 weights round to nearest or, with a seed, up or down at random, in proportion: a
// state that shrinks by 0.05% a step, or an update under 2^-9 of its weight, is lost by rounding to
// nearest (half a step of E4M3 is 3 to 6%). A root above zero stays above zero, else the next update of a
// value far below its block's largest would be divided by eps.
//
// Bound by memory: 28 bytes a value (FP32 weights and states, bf16 gradients and copies), 10 with 8-bit
// states and bf16 weights. A wave takes kUnroll blocks of 256 values, all of its loads issued ahead; a lane
// has four consecutive values of a block, so a block's amax is one wave reduction. Pointers travel in the
// kernel's arguments (no table on the device that a step would have to upload), kAdamwTensors a launch.
#include "device_common.h"
#include "step_rules.h"

namespace beam {

namespace {

struct AdamwBatch {
  AdamwTensor t[kAdamwTensors];
  int32_t first[kAdamwTensors];   // first chunk of each tensor (past the last: the grid's size)
  int32_t base256[kAdamwTensors];   // blocks of 256 values before it in the whole list
};
static_assert(sizeof(AdamwBatch) + sizeof(AdamwScalars) <= 4096, "kernel arguments");

__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// Four E4M3 codes of v (values in a register each) and back.
__device__ __forceinline__ uint32_t pack_e4m3(const floatx4 v) {
  int d = __builtin_amdgcn_cvt_pk_fp8_f32(v.x, v.y, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v.z, v.w, d, true);
}
__device__ __forceinline__ floatx4 unpack_e4m3(uint32_t c) {
  return floatx4{__builtin_amdgcn_cvt_f32_fp8((int)c, 0), __builtin_amdgcn_cvt_f32_fp8((int)c, 1),
                 __builtin_amdgcn_cvt_f32_fp8((int)c, 2), __builtin_amdgcn_cvt_f32_fp8((int)c, 3)};
}

// |x| / scale as an E4M3 value (sign of x), or its stochastic rounding with 16 random bits.
template <bool NOISE, bool ROOT>
__device__ __forceinline__ float to_e4m3(float x, float inv, uint32_t bits16) {
#pragma clang fp contract(off)
  float t = fabsf(x) * inv;
  t = t > 448.f ? 448.f : t;   // NaN stays
  float q;
  if constexpr (NOISE) {
    const int e = max((int)(__float_as_uint(t) >> 23) - 127, -6);
    const float up = __uint_as_float((uint32_t)(130 - e) << 23), down = __uint_as_float((uint32_t)(124 + e) << 23);
    q = floorf(t * up + (float)bits16 * 0x1p-16f) * down;
    q = q > 448.f ? 448.f : q;
  } else {
    q = t;   // the conversion rounds to nearest even
  }
  if constexpr (ROOT) q = x > 0.f && q < 0x1p-9f ? 0x1p-9f : q;
  return copysignf(q, x);
}

template <bool P_BF16, bool G_BF16, bool Q8, bool COPY, bool NOISE>
__global__ __launch_bounds__(kAdamwThreads) void adamw_kernel(AdamwBatch b, AdamwScalars s) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int chunk = blockIdx.x;
  // the last tensor whose first chunk is not behind this one
  static_assert(kAdamwTensors <= 64, "a tensor a lane");
  const int first = b.first[lane < kAdamwTensors ? lane : 0];
  const uint64_t begun = __ballot(lane < kAdamwTensors && first <= chunk);
  const int which = 63 - __clzll((long long)begun);
  const AdamwTensor t = b.t[which];
  const int64_t block0 = (int64_t)(chunk - b.first[which]) * kAdamwChunkBlocks + wave * kAdamwUnroll;

  float gs = 1.f;
  if (s.grad_scale) {
    gs = *s.grad_scale;
    if (!(fabsf(gs) <= 3.4028235e38f)) return;   // a step with gradients out of range is left out
  }
  float lr = s.lr, correction = s.correction, root_scale = s.root_scale, decay = s.decay;
  uint32_t key = s.key;
  if (s.step) {
    const int now = *s.step;
    correction = 1.f / -expm1f((float)now * s.log_beta1);
    root_scale = 1.f / sqrtf(-expm1f((float)now * s.log_beta2));
    key = mix32(s.key + (uint32_t)now);
  }
  if (s.lr_now) {
    lr = *s.lr_now;
    decay = 1.f - lr * s.weight_decay;
  }
  const float step_size = lr * correction;

  struct Loaded {
    floatx4 p, m, v;
    u32x2 pb, gb;
    floatx4 gf;
    uint32_t mc, vc;
    float ms, vs;
  };
  Loaded in[kAdamwUnroll];
  auto at = [&](int u) { return (block0 + u) * 256 + 4 * lane; };
#pragma unroll
  for (int u = 0; u < kAdamwUnroll; ++u) {
    const int64_t i = at(u);
    if (i + 4 > t.count) continue;   // the last values, one by one below
    if constexpr (P_BF16)
      in[u].pb = *reinterpret_cast<const u32x2*>((const uint16_t*)t.param + i);
    else
      in[u].p = *reinterpret_cast<const floatx4*>((const float*)t.param + i);
    if constexpr (G_BF16)
      in[u].gb = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>((const uint16_t*)t.grad + i));
    else
      in[u].gf = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>((const float*)t.grad + i));
    if constexpr (Q8) {
      in[u].mc = *reinterpret_cast<const uint32_t*>((const uint8_t*)t.m + i);
      in[u].vc = *reinterpret_cast<const uint32_t*>((const uint8_t*)t.v + i);
    } else {
      in[u].m = *reinterpret_cast<const floatx4*>((const float*)t.m + i);
      in[u].v = *reinterpret_cast<const floatx4*>((const float*)t.v + i);
    }
  }
  if constexpr (Q8) {
#pragma unroll
    for (int u = 0; u < kAdamwUnroll; ++u)
      if ((block0 + u) * 256 < t.count) {
        in[u].ms = t.m_scale[block0 + u];
        in[u].vs = t.v_scale[block0 + u];
      }
  }
#pragma unroll
  for (int u = 0; u < kAdamwUnroll; ++u) {
    if ((block0 + u) * 256 >= t.count) break;   // wave-uniform
    const int64_t i = at(u);
    const int have = (int)(t.count - i < 4 ? (t.count - i < 0 ? 0 : t.count - i) : 4);
    floatx4 p, g, m, v;
    if (have == 4) {
      p = P_BF16 ? floatx4{bf16_lo(in[u].pb.x), bf16_hi(in[u].pb.x), bf16_lo(in[u].pb.y), bf16_hi(in[u].pb.y)}
                 : in[u].p;
      g = G_BF16 ? floatx4{bf16_lo(in[u].gb.x), bf16_hi(in[u].gb.x), bf16_lo(in[u].gb.y), bf16_hi(in[u].gb.y)}
                 : in[u].gf;
      m = Q8 ? unpack_e4m3(in[u].mc) : in[u].m;
      v = Q8 ? unpack_e4m3(in[u].vc) : in[u].v;
    } else {
      p = g = m = v = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        if (c >= have) break;
        p[c] = P_BF16 ? __uint_as_float((uint32_t)((const uint16_t*)t.param)[i + c] << 16)
                      : ((const float*)t.param)[i + c];
        g[c] = G_BF16 ? __uint_as_float((uint32_t)((const uint16_t*)t.grad)[i + c] << 16)
                      : ((const float*)t.grad)[i + c];
        m[c] = Q8 ? __builtin_amdgcn_cvt_f32_fp8((int)((const uint8_t*)t.m)[i + c], 0) : ((const float*)t.m)[i + c];
        v[c] = Q8 ? __builtin_amdgcn_cvt_f32_fp8((int)((const uint8_t*)t.v)[i + c], 0) : ((const float*)t.v)[i + c];
      }
    }
    floatx4 root;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float gc = g[c] * gs;
      float mc = m[c], vc = v[c];
      if constexpr (Q8) {
        mc = mc * in[u].ms;
        vc = vc * in[u].vs;
        vc = vc * vc;
      }
      mc = mc * s.beta1 + gc * s.rest1;
      vc = vc * s.beta2 + (gc * gc) * s.rest2;
      const float r = sqrtf(vc);
      p[c] = p[c] * decay - step_size * (mc * __builtin_amdgcn_rcpf(r * root_scale + s.eps));
      m[c] = mc;
      v[c] = vc;
      root[c] = r;
    }
    uint32_t bits[4] = {0, 0, 0, 0};
    if constexpr (NOISE) {
      const uint64_t n = ((uint64_t)b.base256[which] + (uint64_t)(block0 + u)) * 256 + 4 * lane;
      const uint32_t k = mix32(key + (uint32_t)(n >> 32));
#pragma unroll
      for (int c = 0; c < 4; ++c) bits[c] = mix32(((uint32_t)n + c) ^ k);
    }
    u32x2 pb;
    if constexpr (P_BF16) {
      if constexpr (NOISE) {
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t f = __float_as_uint(p[c]);
          // infinities and NaN keep their bits
          w[c] = (f & 0x7F800000u) == 0x7F800000u ? f >> 16 : (f + (mix32(bits[c] ^ 0x9E3779B9u) & 0xFFFFu)) >> 16;
        }
        pb = u32x2{w[0] | w[1] << 16, w[2] | w[3] << 16};
      } else {
        pb = u32x2{pack_bf16(p.x, p.y), pack_bf16(p.z, p.w)};
      }
    }
    uint32_t mcode = 0, vcode = 0;
    if constexpr (Q8) {
      // values behind the tensor's end are zero and below every amax
      const float am = fmaxf(wave_max(fmaxf(fmaxf(fabsf(m.x), fabsf(m.y)), fmaxf(fabsf(m.z), fabsf(m.w)))), 0x1p-100f);
      const float av = fmaxf(wave_max(fmaxf(fmaxf(root.x, root.y), fmaxf(root.z, root.w))), 0x1p-100f);
      const float im = 448.f / am, iv = 448.f / av;
      floatx4 qm, qv;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        qm[c] = to_e4m3<NOISE, false>(m[c], im, bits[c] & 0xFFFFu);
        qv[c] = to_e4m3<NOISE, true>(root[c], iv, bits[c] >> 16);
      }
      mcode = pack_e4m3(qm);
      vcode = pack_e4m3(qv);
      if (lane == 0) {
        t.m_scale[block0 + u] = am / 448.f;
        t.v_scale[block0 + u] = av / 448.f;
      }
    }
    if (have == 4) {
      if constexpr (P_BF16)
        *reinterpret_cast<u32x2*>((uint16_t*)t.param + i) = pb;
      else
        *reinterpret_cast<floatx4*>((float*)t.param + i) = p;
      if constexpr (COPY)
        *reinterpret_cast<u32x2*>((uint16_t*)t.copy + i) = u32x2{pack_bf16(p.x, p.y), pack_bf16(p.z, p.w)};
      if constexpr (Q8) {
        *reinterpret_cast<uint32_t*>((uint8_t*)t.m + i) = mcode;
        *reinterpret_cast<uint32_t*>((uint8_t*)t.v + i) = vcode;
      } else {
        *reinterpret_cast<floatx4*>((float*)t.m + i) = m;
        *reinterpret_cast<floatx4*>((float*)t.v + i) = v;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        if (c >= have) break;
        if constexpr (P_BF16)
          ((uint16_t*)t.param)[i + c] = (uint16_t)(pb[c / 2] >> 16 * (c & 1));
        else
          ((float*)t.param)[i + c] = p[c];
        if constexpr (COPY) ((uint16_t*)t.copy)[i + c] = (uint16_t)pack_bf16(p[c], 0.f);
        if constexpr (Q8) {
          ((uint8_t*)t.m)[i + c] = (uint8_t)(mcode >> 8 * c);
          ((uint8_t*)t.v)[i + c] = (uint8_t)(vcode >> 8 * c);
        } else {
          ((float*)t.m)[i + c] = m[c];
          ((float*)t.v)[i + c] = v[c];
        }
      }
    }
  }
}

template <class F>
void pick(bool v, F&& f) {
  v ? f(std::true_type{}) : f(std::false_type{});
}

}  // namespace

hipError_t launch_adamw(const AdamwTensor* tensors, int n, bool p_bf16, bool g_bf16, bool q8, bool copy,
                        bool noise, const AdamwScalars& s, hipStream_t st) {
  AdamwBatch b;
  int used = 0;
  int64_t chunks = 0, base = 0;
  hipError_t err = hipSuccess;
  auto flush = [&]() {
    if (used == 0) return;
    for (int i = used; i < kAdamwTensors; ++i) b.first[i] = INT32_MAX;
    pick(p_bf16, [&](auto pb) {
      pick(g_bf16, [&](auto gb) {
        pick(q8, [&](auto q) {
          pick(copy && !p_bf16, [&](auto cp) {
            pick(noise && (q8 || p_bf16), [&](auto nz) {
              constexpr bool P = decltype(pb)::value, Q = decltype(q)::value, C = decltype(cp)::value,
                             N = decltype(nz)::value;
              if constexpr (!(P && C) && (!N || P || Q))
                hipLaunchKernelGGL((adamw_kernel<P, decltype(gb)::value, Q, C, N>), dim3((unsigned)chunks),
                                   dim3(kAdamwThreads), 0, st, b, s);
            });
          });
        });
      });
    });
    err = hipGetLastError();
    used = 0;
    chunks = 0;
  };
  for (int i = 0; i < n && err == hipSuccess; ++i) {
    const int64_t mine = adamw_chunks(tensors[i].count);
    if (mine == 0) continue;
    if (used == kAdamwTensors || chunks + mine > kAdamwMostChunks) flush();
    b.t[used] = tensors[i];
    b.first[used] = (int32_t)chunks;
    b.base256[used] = (int32_t)base;
    ++used;
    chunks += mine;
    base += ceil_div(tensors[i].count, 256);
  }
  if (err == hipSuccess) flush();
  return err;
}

}  // namespace beam
