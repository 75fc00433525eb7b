// Products of few rows (gfx950): a workgroup's eight waves split the contraction of one block of up to 32 rows by two
// runs of 16 weight rows, and their sums meet in LDS. Where the tiles of gemm_tile.h are fewer than the CUs, their
// chain of stages is what such a call takes; here a wave has an eighth of it, in kNarrowAhead turns at once. Bound by
// reading the weights with few bytes in flight: one row, 5120 -> 2560 of the gated products, 52 MB in 17.4 us out of
// memory (3.0 TB/s, tiles 32), in 13.7 out of the last-level cache (tiles 29); rows' fragments are read again by each
// workgroup, so blocks of 32 rows end where tiles begin to fill the CUs.
#pragma once

#include "gemm_tile.h"
#include "step_rules.h"

namespace beam {

constexpr int kNarrowSums = 2 * 2 * kNarrowWaves * 64;   // floatx4 of LDS

// v[p] of wave i < NV: for row 16 i + lane % 16 of x the products with the weight rows 4 (lane / 16) + 0..3 of run p, run
// 1 `run1` bytes behind run 0; false in the other waves. NV: sub-tiles of 16 rows. Rows lie K values apart, and those
// past x_bytes and w_bytes (under 2^31) read as zero, as does k past K (a multiple of 8).
//
// Fragments go from memory to registers: turn t is 64 values of k, 128 bytes of a row, turns dealt to the waves one by
// one, 1 KB of a row by the eight.
template <int NV>
__device__ __forceinline__ bool narrow_products(const unsigned char* __restrict__ x, uint32_t x_bytes,
                                                const unsigned char* __restrict__ w, uint32_t w_bytes, uint32_t run1,
                                                int K, floatx4* red, int wave, int lane, floatx4 (&v)[2]) {
  const uint32_t ld = 2 * (uint32_t)K, row = (lane & 15) * ld;
  const unsigned char* const xb = uniform(x);
  const unsigned char* const wb = uniform(w);
  floatx4 acc[NV][2];
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i][0] = acc[i][1] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int turns = (K + 63) >> 6;
  for (int t0 = wave; t0 < turns; t0 += kNarrowWaves * kNarrowAhead) {
    intx4 wf[kNarrowAhead][2][2], xf[kNarrowAhead][2][NV];
#pragma unroll
    for (int a = 0; a < kNarrowAhead; ++a)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int k = 64 * (t0 + kNarrowWaves * a) + 32 * s + 8 * (lane >> 4);
        const uint32_t at = row + 2 * (uint32_t)k, past = k < K ? 0u : 0x80000000u;
        wf[a][s][0] = __builtin_bit_cast(intx4, buffer_load16<0>(wb, w_bytes, at | past, 0));
        wf[a][s][1] = __builtin_bit_cast(intx4, buffer_load16<0>(wb, w_bytes, (at + run1) | past, 0));
#pragma unroll
        for (int i = 0; i < NV; ++i)
          xf[a][s][i] = __builtin_bit_cast(intx4, buffer_load16<0>(xb, x_bytes, (at + 16 * i * ld) | past, 0));
      }
    __builtin_amdgcn_sched_barrier(0);   // all of them before the first product
#pragma unroll
    for (int a = 0; a < kNarrowAhead; ++a)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int p = 0; p < 2; ++p) acc[i][p] = tile_mma<false>(wf[a][s][p], xf[a][s][i], acc[i][p]);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p) red[((i * 2 + p) * kNarrowWaves + wave) * 64 + lane] = acc[i][p];
  __syncthreads();
  if (wave >= NV) return false;
#pragma unroll
  for (int p = 0; p < 2; ++p) {   // in the waves' order
    const floatx4* const mine = red + (wave * 2 + p) * kNarrowWaves * 64 + lane;
    v[p] = mine[0];
#pragma unroll
    for (int k = 1; k < kNarrowWaves; ++k) v[p] += mine[k * 64];
  }
  return true;
}

}  // namespace beam
