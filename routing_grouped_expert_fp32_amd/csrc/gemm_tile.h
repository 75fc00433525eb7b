// Tile products D = A B^T of 16-bit operands with FP32 accumulation (gfx950), the core of the grouped
// training products and of the orthogonalised update.
//
// D[m][n] = sum_k A(m, k) B(n, k) for a BM x BN tile. Either operand is stored along the contraction
// (each row a run of k: "row" operands) or across it (each row one k, a run of m or n: "column"
// operands), so the four products Y = X W^T, dX = dY W, dW = dY^T X and X X^T all read their operands
// where they lie, without a transposed copy.
//   * A stage carries 64 values of k. Both kinds reach LDS by 16-byte direct loads, 1 KB a wave
//     instruction. Row operands: [rows][64 k], chunk c of row r at c ^ (r & 7), fragments by 16-byte
//     reads (8 consecutive k of one row). Column operands: [64 k][rows], the 32-byte unit u of row k
//     at u ^ f(k), f = (k & 3) | (k >> 3 & 1) << 2, fragments by transposing 8-byte reads
//     (ds_read_b64_tr_b16: 16 lanes hand in 4 rows x 16 columns and take a column each); the eight
//     rows that half a wave touches lie on distinct banks.
//   * Past an operand's rows, or past k, loads fall outside their buffer and leave zeros in LDS, so
//     no size needs to divide the tile. Rows are multiples of 8 values (16-byte chunks).
//   * The MFMA takes the B fragment first, so a lane ends with four consecutive n of one m, and the
//     epilogue stores 8 or 16 bytes a lane.
#pragma once

#include "device_common.h"

namespace beam {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kTileK = 64;   // values of k in a stage (128 bytes)

// Workgroup tile of BM x BN, WM x WN waves, ST stages of LDS.
template <int BM_, int BN_, int WM_, int WN_, int ST_>
struct TileShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int FM = BM / 16 / WM, FN = BN / 16 / WN;   // 16 x 16 sub-tiles of a wave
  static constexpr int kABytes = BM * 2 * kTileK, kBBytes = BN * 2 * kTileK;
  static constexpr int kLdsBytes = ST * (kABytes + kBBytes);
  static_assert(kLdsBytes <= 160 * 1024, "LDS budget");
  static_assert(FM * 16 * WM == BM && FN * 16 * WN == BN, "whole sub-tiles");
};

// One operand of a tile, wave-uniform.
struct TileOperand {
  const unsigned char* base;   // first value of the tile
  int64_t ld;                  // bytes from one stored row to the next
  int32_t rows;                // row operands: rows that exist
  int32_t tail;                // column operands: bytes from base to the end of its own row
};

// Direct loads of one operand's stages (ROWS = BM or BN).
template <int ROWS, int WAVES, bool COL>
struct OperandLoader {
  static constexpr int L = ROWS / 8 / WAVES;   // 1 KB loads of a wave in a stage
  static_assert(L * 8 * WAVES == ROWS, "loads split evenly over waves");
  static constexpr int kRowChunks = COL ? ROWS / 8 : 8;       // 16-byte chunks of a stored row
  static constexpr int kLoadRows = 64 / kRowChunks;           // stored rows of a load
  static_assert(!COL || ROWS >= 128, "the swizzle needs eight 32-byte units a row");
  TileOperand op;
  uint32_t voff[L];
  int kofs;   // row operands: first k of this lane's chunk within a stage

  __device__ __forceinline__ void init(const TileOperand& o, int wave, int lane) {
    op = o;
    const int slot = lane % kRowChunks, lr = lane / kRowChunks;
    kofs = 8 * (slot ^ (lr & 7));
#pragma unroll
    for (int q = 0; q < L; ++q) {
      const int row = (wave * L + q) * kLoadRows + lr;
      if constexpr (COL) {
        const int f = (row & 3) | ((row >> 1) & 4);
        voff[q] = (uint32_t)(row * op.ld + (slot ^ (f << 1)) * 16);
      } else {
        voff[q] = (uint32_t)(row * op.ld + kofs * 2);
      }
    }
  }

  // stage kt of a contraction over k values into the LDS ring slot at dst
  __device__ __forceinline__ void issue(int kt, int64_t k, unsigned char* dst, int wave) const {
    if constexpr (COL) {
      const int64_t left = k - (int64_t)kt * kTileK;
      const int rows = left < kTileK ? (int)left : kTileK;
      const unsigned char* base = op.base + (int64_t)kt * kTileK * op.ld;
      const uint32_t bytes = rows > 0 ? (uint32_t)((rows - 1) * op.ld + op.tail) : 0u;
#pragma unroll
      for (int q = 0; q < L; ++q)
        buffer_load_lds16<0>(base, bytes, voff[q], 0, (lds_void_t*)(dst + (wave * L + q) * 1024));
    } else {
      const uint32_t bytes = (uint32_t)(op.rows * op.ld);
      // chunks past k: an offset past every buffer (a tile's rows are under 2 GiB)
      const uint32_t past = (int64_t)kt * kTileK + kofs < k ? 0u : 0x80000000u;
#pragma unroll
      for (int q = 0; q < L; ++q)
        buffer_load_lds16<0>(op.base, bytes, voff[q] | past, (uint32_t)kt * (2 * kTileK),
                             (lds_void_t*)(dst + (wave * L + q) * 1024));
    }
  }
};

// Fragment reads of one operand from a ring slot: the wave's COUNT sub-tiles (16 rows of the tile)
// first, first + STEP, ...; step s is 32 of the stage's 64 k. Lane l holds row l % 16,
// k = 32 s + 8 (l / 16) + 0..7.
template <int ROWS, int COUNT, int STEP, bool COL>
struct FragReader {
  int off[COL ? COUNT : 2];

  __device__ __forceinline__ void init(int first, int lane) {
    const int r = lane & 15, g = lane >> 4;
    if constexpr (COL) {
      const int f = (r >> 2) | ((g & 1) << 2);
#pragma unroll
      for (int i = 0; i < COUNT; ++i)
        off[i] = (8 * g + (r >> 2)) * (2 * ROWS) + (r & 3) * 8 + (((first + STEP * i) ^ f) << 5);
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        off[s] = first * 2048 + r * 128 + (((4 * s + g) ^ (r & 7)) << 4);
    }
  }
  __device__ __forceinline__ intx4 read(const unsigned char* slot, int i, int s) const {
    if constexpr (COL) {
      const unsigned char* p = slot + s * (32 * 2 * ROWS) + off[i];
      const u32x2 lo = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
      const u32x2 hi = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * 2 * ROWS)));
      return intx4{(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
    } else {
      return *reinterpret_cast<const intx4*>(slot + i * (STEP * 2048) + off[s]);
    }
  }
};

template <bool F16>
__device__ __forceinline__ floatx4 tile_mma(intx4 a, intx4 b, floatx4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Barrier without the fence of __syncthreads(), which would wait for every load in flight.
__device__ __forceinline__ void tile_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The loop over k of one tile. acc[i][j] is sub-tile (wm + WM i, wn FN + j); NV of the wave's FM row
// sub-tiles hold rows, the others' accumulators are left alone.
template <class S, bool ACOL, bool BCOL, bool F16, int NV>
__device__ __forceinline__ void tile_kloop(const OperandLoader<S::BM, S::kWaves, ACOL>& la,
                                           const OperandLoader<S::BN, S::kWaves, BCOL>& lb,
                                           int64_t k, unsigned char* smem, int wave, int lane,
                                           floatx4 (&acc)[S::FM][S::FN]) {
  FragReader<S::BM, NV, S::WM, ACOL> ra;
  FragReader<S::BN, S::FN, 1, BCOL> rb;
  ra.init(wave / S::WN, lane);
  rb.init(wave % S::WN * S::FN, lane);
  const int nk = (int)((k + kTileK - 1) / kTileK);
  unsigned char* const aring = smem;
  unsigned char* const bring = smem + S::ST * S::kABytes;
  constexpr int kPerStage = OperandLoader<S::BM, S::kWaves, ACOL>::L +
                            OperandLoader<S::BN, S::kWaves, BCOL>::L;
  static_assert((S::ST - 1) * kPerStage < 64, "vmcnt range");
#pragma unroll
  for (int p = 0; p < S::ST - 1; ++p)
    if (p < nk) {
      la.issue(p, k, aring + p * S::kABytes, wave);
      lb.issue(p, k, bring + p * S::kBBytes, wave);
    }
  for (int kt = 0; kt < nk; ++kt) {
    // the wave's own loads of stage kt have landed; after the barrier everyone's have, and everyone
    // is done reading the slot that stage kt + ST - 1 takes
    if (kt + S::ST - 2 < nk)
      __builtin_amdgcn_s_waitcnt(vmcnt_imm((S::ST - 2) * kPerStage));
    else
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    tile_barrier();
    const int nx = kt + S::ST - 1;
    if (nx < nk) {
      la.issue(nx, k, aring + (nx % S::ST) * S::kABytes, wave);
      lb.issue(nx, k, bring + (nx % S::ST) * S::kBBytes, wave);
    }
    const unsigned char* sa = aring + (kt % S::ST) * S::kABytes;
    const unsigned char* sb = bring + (kt % S::ST) * S::kBBytes;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      intx4 bf[S::FN], af[NV];
#pragma unroll
      for (int j = 0; j < S::FN; ++j) bf[j] = rb.read(sb, j, s);
#pragma unroll
      for (int i = 0; i < NV; ++i) af[i] = ra.read(sa, i, s);
      __builtin_amdgcn_sched_barrier(0);   // all reads ahead of the MFMA chain
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < S::FN; ++j) acc[i][j] = tile_mma<F16>(bf[j], af[i], acc[i][j]);
    }
  }
}

// Walks a tile's accumulators: f(m, n, v) with v = D[m][n .. n + 3], m and n within the tile.
template <class S, int NV, class F>
__device__ __forceinline__ void tile_for_each(const floatx4 (&acc)[S::FM][S::FN], int wave,
                                              int lane, F&& f) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < S::FN; ++j)
      f(16 * (wave / S::WN + S::WM * i) + (lane & 15),
        16 * (wave % S::WN * S::FN + j) + 4 * (lane >> 4), acc[i][j]);
}

// Four consecutive values to bf16 or fp32 at element offset `at` (8- or 16-byte aligned).
template <bool OUT_BF16>
__device__ __forceinline__ void store4(void* out, int64_t at, floatx4 v) {
  if constexpr (OUT_BF16) {
    u32x2 o;
    o.x = f32_to_bf16_bits(v.x) | (f32_to_bf16_bits(v.y) << 16);
    o.y = f32_to_bf16_bits(v.z) | (f32_to_bf16_bits(v.w) << 16);
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(out) + at) = o;
  } else {
    *reinterpret_cast<floatx4*>(reinterpret_cast<float*>(out) + at) = v;
  }
}

}  // namespace beam
