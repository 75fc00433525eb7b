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
// Bound by memory: 28 bytes a value (FP32 weights and states, bf16 gradients and copies: 4e8 values in 1.98 to 2.03 ms,
// 5.6 TB/s), 10 with 8-bit states and bf16 weights (0.78 to 0.82 ms, 5.0 TB/s, where the arithmetic of the roundings,
// some 85 instructions a value, is near it). A wave takes kAdamwUnroll blocks of 256 values, all of its loads issued
// ahead and non-temporal, as its stores (2.12 ms with the default policy); a lane has four consecutive values of a
// block. The eight maxima of a wave's blocks are reduced together, each step halving what a lane holds, and their eight
// reciprocals and eight scales are one division, a lane each (1.10 ms with a reduction and four divisions a block, and
// codes rounded by floor and the conversion).
//
// A workgroup finds its tensor in a table that the caller keeps on the device (one launch for a whole list: 208 tensors
// of 5120 values 8.3 to 8.8 us), or, without one, in the kernel's arguments, kAdamwTensors a launch (24 us; with other
// gradients a call the checks of 208 tensors in Python take 118).
#include "device_common.h"
#include "step_rules.h"

namespace beam {

namespace {

struct AdamwBatch {
  AdamwEntry t[kAdamwTensors];
};
static_assert(sizeof(AdamwBatch) + sizeof(AdamwScalars) + 16 <= 4096, "kernel arguments");

// Pointers out of a table are to global memory (the compiler would take the slower flat accesses).
template <class T>
__device__ __forceinline__ __attribute__((address_space(1))) T* global_at(const void* p, int64_t i) {
  return (__attribute__((address_space(1))) T*)p + i;
}

// Four E4M3 codes of v, rounded to nearest even, and back.
__device__ __forceinline__ uint32_t pack_e4m3(const floatx4 v) {
  int d = __builtin_amdgcn_cvt_pk_fp8_f32(v.x, v.y, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v.z, v.w, d, true);
}
__device__ __forceinline__ floatx4 unpack_e4m3(uint32_t c) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  return floatx4{lo[0], lo[1], hi[0], hi[1]};
}

// sqrt of four values a lane, correctly rounded: the hardware's is off by an ulp at most, and the residue says
// which way. Where a value of the wave is under 2^-96 but not zero the residue would lose its bits.
__device__ __forceinline__ floatx4 roots_of(const floatx4 v) {
  floatx4 r;
  uint32_t least = 0xFFFFFFFFu;
#pragma unroll
  for (int c = 0; c < 4; ++c) least = min(least, __float_as_uint(v[c]) - 1);   // zero wraps round
  if (__any(least < 0x0F800000u - 1)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) r[c] = sqrtf(v[c]);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float s = __builtin_amdgcn_sqrtf(v[c]);
      const float down = __uint_as_float(__float_as_uint(s) - 1), up = __uint_as_float(__float_as_uint(s) + 1);
      const float low = __builtin_fmaf(-down, s, v[c]) <= 0.f ? down : s;
      r[c] = __builtin_fmaf(-up, s, v[c]) > 0.f ? up : low;
    }
  }
  return r;
}

// The E4M3 codes of four x / scale, inv = 1 / scale, a root's above zero for an x above zero. With NOISE each takes
// 16 random bits: times 2^-120 a float's bits are an E4M3 code and 20 more, below 2^-6 too (FP32's subnormals line
// up with E4M3's there, t rounded to 2^-29), so the random bits are added in front of what is cut off.
template <bool NOISE, bool ROOT>
__device__ __forceinline__ uint32_t e4m3_codes(const floatx4 x, float inv, const uint32_t (&bits16)[4]) {
#pragma clang fp contract(off)
  floatx4 t;
#pragma unroll
  for (int c = 0; c < 4; ++c) t[c] = fminf(fabsf(x[c]) * inv, 448.f);   // a NaN's block has a NaN for its scale
  if constexpr (NOISE) {
    uint32_t codes = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t q = (__float_as_uint(t[c] * 0x1p-120f) + (bits16[c] << 4)) >> 20;
      if constexpr (ROOT)
        q = max(q, min(__float_as_uint(x[c]), 1u));
      else
        q |= __float_as_uint(x[c]) >> 24 & 0x80u;
      codes |= q << 8 * c;
    }
    return codes;
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      t[c] = ROOT ? (x[c] > 0.f && t[c] < 0x1p-9f ? 0x1p-9f : t[c]) : copysignf(t[c], x[c]);
    return pack_e4m3(t);
  }
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, kCtrl, 0xF, 0xF, false);
}

// Wave maxima of eight values a lane (magnitudes as their bits: NaN above all): lane l ends with that of
// value l / 8.
__device__ __forceinline__ uint32_t wave_maxima(uint32_t (&v)[8], int lane) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {   // lanes 0-31 keep k, 32-63 k + 4
    const auto r = __builtin_amdgcn_permlane32_swap((int)v[k], (int)v[k + 4], false, false);
    v[k] = max((uint32_t)r[0], (uint32_t)r[1]);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {   // even rows of 16 keep k, odd ones k + 2
    const auto r = __builtin_amdgcn_permlane16_swap((int)v[k], (int)v[k + 2], false, false);
    v[k] = max((uint32_t)r[0], (uint32_t)r[1]);
  }
  const bool high = lane & 8;
  uint32_t m = max(high ? v[1] : v[0], dpp<0x128>(high ? v[0] : v[1]));   // eight lanes round the row
  m = max(m, dpp<0x141>(m));         // mirrored halves of a row
  m = max(m, dpp<0xB1>(m));          // pairs
  return max(m, dpp<0x4E>(m));       // and pairs of pairs
}

struct AdamwNumbers {
  float gs, step_size, root_scale, decay;
  uint32_t key;
};

// kAdamwUnroll blocks of a tensor from block0 on, `left` values (with FULL all of them).
template <bool P_BF16, bool G_BF16, bool Q8, bool COPY, bool NOISE, bool FULL>
__device__ __forceinline__ void adamw_wave(const AdamwEntry& e, int64_t block0, int left, const AdamwNumbers& a,
                                           const AdamwScalars& s, int lane) {
#pragma clang fp contract(off)
  constexpr int U = kAdamwUnroll;
  const int64_t i0 = block0 * 256;
  auto* const param32 = global_at<float>(e.t.param, i0);
  auto* const param16 = global_at<uint16_t>(e.t.param, i0);
  auto* const grad32 = global_at<const float>(e.t.grad, i0);
  auto* const grad16 = global_at<const uint16_t>(e.t.grad, i0);
  auto* const m32 = global_at<float>(e.t.m, i0);
  auto* const v32 = global_at<float>(e.t.v, i0);
  auto* const m8 = global_at<uint8_t>(e.t.m, i0);
  auto* const v8 = global_at<uint8_t>(e.t.v, i0);
  auto* const copy16 = global_at<uint16_t>(e.t.copy, i0);
#define BEAM_AT(type, p, i) (*(__attribute__((address_space(1))) type*)((p) + (i)))
  struct Loaded {
    floatx4 p, m, v, gf;
    u32x2 pb, gb;
    uint32_t mc, vc;
  };
  Loaded in[U];
  // values of the lane's four in block u
  auto have = [&](int u) { return FULL ? 4 : min(max(left - (256 * u + 4 * lane), 0), 4); };
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = 256 * u + 4 * lane;
    if (!FULL && have(u) < 4) continue;   // the last values, one by one below
    if constexpr (P_BF16)
      in[u].pb = __builtin_nontemporal_load(&BEAM_AT(const u32x2, param16, i));
    else
      in[u].p = __builtin_nontemporal_load(&BEAM_AT(const floatx4, param32, i));
    if constexpr (G_BF16)
      in[u].gb = __builtin_nontemporal_load(&BEAM_AT(const u32x2, grad16, i));
    else
      in[u].gf = __builtin_nontemporal_load(&BEAM_AT(const floatx4, grad32, i));
    if constexpr (Q8) {
      in[u].mc = __builtin_nontemporal_load(&BEAM_AT(const uint32_t, m8, i));
      in[u].vc = __builtin_nontemporal_load(&BEAM_AT(const uint32_t, v8, i));
    } else {
      in[u].m = __builtin_nontemporal_load(&BEAM_AT(const floatx4, m32, i));
      in[u].v = __builtin_nontemporal_load(&BEAM_AT(const floatx4, v32, i));
    }
  }
  // a lane's scale: of m and of the root in turn, of block lane / 16
  auto* const scale = Q8 ? global_at<float>(lane & 8 ? e.t.v_scale : e.t.m_scale, block0 + (lane >> 4)) : nullptr;
  const bool scaled = Q8 && (FULL || 256 * (lane >> 4) < left);
  int scale_bits = 0;
  if (scaled) scale_bits = __float_as_int(*scale);

  floatx4 m_new[U], root[U];
  uint32_t bits[U][4], most[2 * U] = {};   // of the blocks behind the tensor's end too
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!FULL && 256 * u >= left) break;   // wave-uniform
    const int i = 256 * u + 4 * lane, n = have(u);
    floatx4 p, g, m, v;
    if (FULL || n == 4) {
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
        if (c >= n) break;
        p[c] = P_BF16 ? __uint_as_float((uint32_t)param16[i + c] << 16) : param32[i + c];
        g[c] = G_BF16 ? __uint_as_float((uint32_t)grad16[i + c] << 16) : grad32[i + c];
        m[c] = Q8 ? __builtin_amdgcn_cvt_f32_fp8((int)m8[i + c], 0) : m32[i + c];
        v[c] = Q8 ? __builtin_amdgcn_cvt_f32_fp8((int)v8[i + c], 0) : v32[i + c];
      }
    }
    if constexpr (Q8) {
      const float ms = __int_as_float(__builtin_amdgcn_readlane(scale_bits, 16 * u));
      const float vs = __int_as_float(__builtin_amdgcn_readlane(scale_bits, 16 * u + 8));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        m[c] = m[c] * ms;
        v[c] = v[c] * vs;
        v[c] = v[c] * v[c];
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float gc = g[c] * a.gs;
      m[c] = m[c] * s.beta1 + gc * s.rest1;
      v[c] = v[c] * s.beta2 + (gc * gc) * s.rest2;
    }
    root[u] = roots_of(v);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float d = __builtin_fmaf(root[u][c], a.root_scale, s.eps);
      p[c] = __builtin_fmaf(-a.step_size, m[c] * __builtin_amdgcn_rcpf(d), p[c] * a.decay);
    }
    m_new[u] = m;
    if constexpr (Q8) {   // values behind the tensor's end are zero
      most[2 * u] = max(max(abs_bits(m.x), abs_bits(m.y)), max(abs_bits(m.z), abs_bits(m.w)));
      most[2 * u + 1] = max(max(abs_bits(root[u].x), abs_bits(root[u].y)), max(abs_bits(root[u].z), abs_bits(root[u].w)));
    }
    if constexpr (NOISE) {
      const uint64_t number = ((uint64_t)(uint32_t)e.base256 + (uint64_t)(block0 + u)) * 256;   // wave-uniform
      const uint32_t k = mix32(a.key + (uint32_t)(number >> 32));
#pragma unroll
      for (int c = 0; c < 4; ++c) bits[u][c] = mix32(((uint32_t)number + 4 * lane + c) ^ k);
    }
    u32x2 pb;
    if constexpr (P_BF16) {
      if constexpr (NOISE) {
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t f = __float_as_uint(p[c]);
          const uint32_t cut = (f & 0x7F800000u) == 0x7F800000u ? 0u : 0xFFFFu;   // infinities and NaN stay
          w[c] = f + (mix32(bits[u][c] ^ 0x9E3779B9u) & cut);
        }
        pb = u32x2{w[0] >> 16 | (w[1] & 0xFFFF0000u), w[2] >> 16 | (w[3] & 0xFFFF0000u)};
      } else {
        pb = u32x2{pack_bf16(p.x, p.y), pack_bf16(p.z, p.w)};
      }
    }
    if (FULL || n == 4) {
      if constexpr (P_BF16)
        __builtin_nontemporal_store(pb, &BEAM_AT(u32x2, param16, i));
      else
        __builtin_nontemporal_store(p, &BEAM_AT(floatx4, param32, i));
      if constexpr (COPY) __builtin_nontemporal_store(u32x2{pack_bf16(p.x, p.y), pack_bf16(p.z, p.w)}, &BEAM_AT(u32x2, copy16, i));
      if constexpr (!Q8) {
        __builtin_nontemporal_store(m, &BEAM_AT(floatx4, m32, i));
        __builtin_nontemporal_store(v, &BEAM_AT(floatx4, v32, i));
      }
    } else {
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        if (c >= n) break;
        if constexpr (P_BF16)
          param16[i + c] = (uint16_t)(pb[c / 2] >> 16 * (c & 1));
        else
          param32[i + c] = p[c];
        if constexpr (COPY) copy16[i + c] = (uint16_t)pack_bf16(p[c], 0.f);
        if constexpr (!Q8) {
          m32[i + c] = m[c];
          v32[i + c] = v[c];
        }
      }
    }
  }
  if constexpr (Q8) {
    const float amax = __uint_as_float(max(wave_maxima(most, lane), 0x0D800000u));   // at least 2^-100
    const bool second = lane & 1;
    const float ratio = (second ? amax : 448.f) / (second ? 448.f : amax);
    if (scaled && (lane & 7) == 1) *scale = ratio;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!FULL && 256 * u >= left) break;   // wave-uniform
      const float im = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ratio), 16 * u));
      const float iv = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ratio), 16 * u + 8));
      uint32_t low[4] = {}, high[4] = {};
      if constexpr (NOISE) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          low[c] = bits[u][c] & 0xFFFFu;
          high[c] = bits[u][c] >> 16;
        }
      }
      const uint32_t mcode = e4m3_codes<NOISE, false>(m_new[u], im, low);
      const uint32_t vcode = e4m3_codes<NOISE, true>(root[u], iv, high);
      const int i = 256 * u + 4 * lane, n = have(u);
      if (FULL || n == 4) {
        __builtin_nontemporal_store(mcode, &BEAM_AT(uint32_t, m8, i));
        __builtin_nontemporal_store(vcode, &BEAM_AT(uint32_t, v8, i));
      } else {
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          if (c >= n) break;
          m8[i + c] = (uint8_t)(mcode >> 8 * c);
          v8[i + c] = (uint8_t)(vcode >> 8 * c);
        }
      }
    }
  }
#undef BEAM_AT
}

template <bool P_BF16, bool G_BF16, bool Q8, bool COPY, bool NOISE>
__global__ __launch_bounds__(kAdamwThreads) void adamw_kernel(AdamwBatch b, const unsigned char* __restrict__ table,
                                                             int n, AdamwScalars s) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int chunk = blockIdx.x;
  AdamwEntry e;
  if (table) {
    // a table of another list than the launch's: nothing is done outside it, and nothing at all to other types
    const AdamwTableHead head = *reinterpret_cast<const AdamwTableHead*>(table);
    if (chunk >= head.chunks || head.entries != n || head.types != adamw_types(P_BF16, G_BF16, Q8, COPY)) return;
    const auto* const entries = reinterpret_cast<const AdamwEntry*>(table + sizeof(AdamwTableHead));
    const auto* const map = reinterpret_cast<const int32_t*>(entries + n);
    e = entries[__builtin_amdgcn_readfirstlane(map[chunk])];
  } else {   // the last tensor whose first chunk is not behind this one
    static_assert(kAdamwTensors <= 64, "a tensor a lane");
    const uint64_t begun = __ballot(lane < n && b.t[lane < n ? lane : 0].first <= chunk);
    e = b.t[63 - __clzll((long long)begun)];
  }
  const AdamwTensor& t = e.t;
  const int64_t block0 = (int64_t)(chunk - e.first) * kAdamwChunkBlocks + wave * kAdamwUnroll;

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

  static_assert(kAdamwUnroll == 4, "eight maxima a wave");
  const int64_t left = t.count - block0 * 256;   // values from the wave's first on
  if (left <= 0) return;
  const AdamwNumbers numbers = {gs, step_size, root_scale, decay, key};
  if (left >= kAdamwUnroll * 256)
    adamw_wave<P_BF16, G_BF16, Q8, COPY, NOISE, true>(e, block0, kAdamwUnroll * 256, numbers, s, lane);
  else
    adamw_wave<P_BF16, G_BF16, Q8, COPY, NOISE, false>(e, block0, (int)left, numbers, s, lane);
}

template <class F>
void pick(bool v, F&& f) {
  v ? f(std::true_type{}) : f(std::false_type{});
}

}  // namespace

hipError_t launch_adamw(const AdamwTensor* tensors, int n, const void* table, bool p_bf16, bool g_bf16, bool q8,
                        bool copy, bool noise, const AdamwScalars& s, hipStream_t st) {
  auto go = [&](const AdamwBatch& b, const void* tab, int count, int64_t chunks) {
    pick(p_bf16, [&](auto pb) {
      pick(g_bf16, [&](auto gb) {
        pick(q8, [&](auto q) {
          pick(copy, [&](auto cp) {
            pick(noise && (q8 || p_bf16), [&](auto nz) {
              constexpr bool P = decltype(pb)::value, Q = decltype(q)::value, C = decltype(cp)::value,
                             N = decltype(nz)::value;
              if constexpr (!(P && C) && (!N || P || Q))   // the others are refused, or not asked for
                hipLaunchKernelGGL((adamw_kernel<P, decltype(gb)::value, Q, C, N>), dim3((unsigned)chunks),
                                   dim3(kAdamwThreads), 0, st, b, reinterpret_cast<const unsigned char*>(tab), count, s);
            });
          });
        });
      });
    });
    return hipGetLastError();
  };
  AdamwBatch b = {};
  if (table) {
    int entries = 0;
    int64_t chunks = 0;
    for (int i = 0; i < n; ++i) {
      entries += tensors[i].count > 0;
      chunks += adamw_chunks(tensors[i].count);
    }
    if (chunks <= kAdamwMostChunks) return go(b, table, entries, chunks);
  }
  int used = 0;
  int64_t chunks = 0, base = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t mine = adamw_chunks(tensors[i].count);
    if (mine == 0) continue;
    if (used == kAdamwTensors || chunks + mine > kAdamwMostChunks) {
      const hipError_t err = go(b, nullptr, used, chunks);
      if (err != hipSuccess) return err;
      used = 0;
      chunks = 0;
    }
    b.t[used++] = {tensors[i], (int32_t)chunks, (int32_t)base};
    chunks += mine;
    base += ceil_div(tensors[i].count, 256);
  }
  return used ? go(b, nullptr, used, chunks) : hipSuccess;
}

}  // namespace beam
