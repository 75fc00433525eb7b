// Tile products D = A B^T of 16-bit operands with FP32 accumulation (gfx950), the core of the grouped
// training products and of the orthogonalised update.
//
// D[m][n] = sum_k A(m, k) B(n, k) for a BM x BN tile. Either operand is stored along the contraction
// (each row a run of k: "row" operands) or across it (each row one k, a run of m or n: "column"
// operands), so the four products Y = X W^T, dX = dY W, dW = dY^T X and X X^T all read their operands
// where they lie, without a transposed copy.
//   * A stage carries 64 values of k. Both kinds reach LDS by 16-byte direct loads, 1 KB a wave
//     instruction. Row operands: [rows][64 k], chunk c of row r at c ^ (r & 7), fragments by 16-byte
//     reads (8 consecutive k of one row). Column operands: [k][rows], the 32-byte unit u of row k
//     at u ^ f(k), f = (k & 3) | (k >> 3 & 1) << 2 (64 rows: its upper two bits, two stored rows being
//     256 bytes), fragments by transposing 8-byte reads
//     (ds_read_b64_tr_b16: 16 lanes hand in 4 rows x 16 columns and take a column each); the eight
//     rows that half a wave touches lie on distinct banks.
//   * Past an operand's rows, or past k, loads fall outside their buffer and leave zeros in LDS, so
//     no size needs to divide the tile. Rows are multiples of 8 values (16-byte chunks).
//   * The MFMA takes the B fragment first, so a lane ends with four consecutive n of one m, and the
//     epilogue stores 8 or 16 bytes a lane.
#pragma once

#include "device_common.h"
#include "train_rules.h"

namespace beam {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Wave-uniform values that the compiler would otherwise keep in vector registers, where a buffer
// descriptor made from them costs a loop around every load.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float uniform(float v) {
  return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v)));
}
template <class T>
__device__ __forceinline__ T* uniform(T* p) {
  const uint64_t u = (uint64_t)p;
  return (T*)((uint64_t)(uint32_t)uniform((int)(uint32_t)u) |
              (uint64_t)(uint32_t)uniform((int)(uint32_t)(u >> 32)) << 32);
}

// One operand of a tile, wave-uniform.
struct TileOperand {
  const unsigned char* base;   // first value of the tile
  int64_t ld;                  // bytes from one stored row to the next
  int32_t rows;                // row operands: rows that exist
  int32_t tail;                // column operands: bytes from base to the end of its own row
};

// f(k) of a column operand, from k & 3 and bit 3 of k
template <int ROWS>
__device__ __forceinline__ int column_swizzle(int low, int bit3) {
  return ROWS >= 128 ? low | bit3 << 2 : low >> 1 | bit3 << 1;
}

// Direct loads of one operand's stages (ROWS = BM or BN).
template <int ROWS, int WAVES, bool COL>
struct OperandLoader {
  static constexpr int L = ROWS * kStageK / 512 / WAVES;   // 1 KB loads of a wave in a stage
  static_assert(L * 512 * WAVES == ROWS * kStageK, "loads split evenly over waves");
  static constexpr int kRowChunks = COL ? ROWS / 8 : 8;       // 16-byte chunks of a stored row
  static constexpr int kLoadRows = 64 / kRowChunks;           // stored rows of a load
  static_assert(!COL || (ROWS >= 64 && (ROWS & (ROWS - 1)) == 0), "the swizzle permutes 4 or 8 units");
  TileOperand op;
  uint32_t voff[L];
  bool stream = false;   // read once: non-temporal loads
  int kofs;   // row operands: first k of this lane's chunk within a stage

  __device__ __forceinline__ void init(const TileOperand& o, int wave, int lane) {
    init(o, wave, lane, [](int row) { return row; });
  }
  // row operands: row r of the tile is stored row at(r) from `base` (op.rows: one past the last of them)
  template <class At>
  __device__ __forceinline__ void init(const TileOperand& o, int wave, int lane, At&& at) {
    op = o;
    const int slot = lane % kRowChunks, lr = lane / kRowChunks;
    kofs = 8 * (slot ^ (lr & 7));
#pragma unroll
    for (int q = 0; q < L; ++q) {
      const int row = (wave * L + q) * kLoadRows + lr;
      if constexpr (COL) {
        const int f = column_swizzle<ROWS>(row & 3, (row >> 3) & 1);
        voff[q] = (uint32_t)(row * op.ld + (slot ^ (f << 1)) * 16);
      } else {
        voff[q] = (uint32_t)(at(row) * op.ld + kofs * 2);
      }
    }
  }

  // stage kt of a contraction over k values into the LDS ring slot at dst
  __device__ __forceinline__ void issue(int kt, int64_t k, unsigned char* dst, int wave) const {
    if (stream)
      issue_as<kCachePolicyNT>(kt, k, dst, wave);
    else
      issue_as<0>(kt, k, dst, wave);
  }
  template <int kAux>
  __device__ __forceinline__ void issue_as(int kt, int64_t k, unsigned char* dst, int wave) const {
    if constexpr (COL) {
      const int64_t left = k - (int64_t)kt * kStageK;
      const int rows = left < kStageK ? (int)left : kStageK;
      const unsigned char* base = uniform(op.base + (int64_t)kt * kStageK * op.ld);
      const uint32_t bytes =
          (uint32_t)uniform(rows > 0 ? (int)((rows - 1) * op.ld + op.tail) : 0);
#pragma unroll
      for (int q = 0; q < L; ++q)
        buffer_load_lds16<kAux>(base, bytes, voff[q], 0, (lds_void_t*)(dst + (wave * L + q) * 1024));
    } else {
      const uint32_t bytes = (uint32_t)(op.rows * op.ld);
      // chunks past k: an offset past every buffer (a tile's rows are under 2 GiB)
      const uint32_t past = (int64_t)kt * kStageK + kofs < k ? 0u : 0x80000000u;
#pragma unroll
      for (int q = 0; q < L; ++q)
        buffer_load_lds16<kAux>(op.base, bytes, voff[q] | past, (uint32_t)kt * (2 * kStageK),
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
      const int f = column_swizzle<ROWS>(r >> 2, g & 1);
#pragma unroll
      for (int i = 0; i < COUNT; ++i)
        off[i] = (8 * g + (r >> 2)) * (2 * ROWS) + (r & 3) * 8 + (((first + STEP * i) ^ f) << 5);
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        off[s] = first * 2048 + r * 128 + (((4 * s + g) ^ (r & 7)) << 4);
    }
  }
  // __restrict__: without it the compiler takes a transposing read to alias the direct loads in flight
  // and waits for all of them first (vmcnt 0 in every stage; the input gradient ran 20% slower)
  __device__ __forceinline__ intx4 read(const unsigned char* __restrict__ slot, int i, int s) const {
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

// One wave's side of a stage: its fragments and their schedule. A stage is NV positions a step: position p
// multiplies row sub-tile p % NV in step p / NV; acc[i][j] is sub-tile (row_tile(wm, i), wn FN + j). NV of
// the wave's FM row sub-tiles hold rows, the others' accumulators are left alone.
//
// Fragments are read ahead of their MFMAs, the row operand's AHEAD positions, the other's one step.
// Once the last AHEAD positions' fragments of a stage are in registers, its slot is free: there, and
// not at the stage's end, stands its one barrier (`turn`), so the reads of the next stage run under
// this one's last MFMAs.
template <class S, bool ACOL, bool BCOL, bool F16, int NV>
struct TileStage {
  static constexpr int STEPS = kStageK / 32, P = STEPS * NV, AHEAD = NV < 4 ? NV : 4;
  FragReader<S::BM, NV, S::WM, ACOL> ra;
  FragReader<S::BN, S::FN, 1, BCOL> rb;
  intx4 af[P + AHEAD], bf[STEPS + 1][S::FN];   // the next stage's first ones at the end

  __device__ __forceinline__ void init(int wave, int lane) {
    ra.init(S::row_tile(wave / S::WN, 0), lane);
    rb.init(wave % S::WN * S::FN, lane);
  }
  // the first fragments of the first stage, which has landed in the slots sa, sb
  __device__ __forceinline__ void start(const unsigned char* sa, const unsigned char* sb) {
#pragma unroll
    for (int j = 0; j < S::FN; ++j) bf[0][j] = rb.read(sb, j, 0);
#pragma unroll
    for (int p = 0; p < AHEAD; ++p) af[p] = ra.read(sa, p, 0);
  }
  // multiplies the stage in sa, sb; `turn` waits until the next one has landed in na, nb (behind the
  // last stage the fragments read from there are not used) and issues further loads
  template <class Turn>
  __device__ __forceinline__ void run(const unsigned char* sa, const unsigned char* sb,
                                      const unsigned char* na, const unsigned char* nb, Turn&& turn,
                                      floatx4 (&acc)[S::FM][S::FN]) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int s = p / NV;
      if (p == P - AHEAD) turn();
      if (p + AHEAD < P)
        af[p + AHEAD] = ra.read(sa, (p + AHEAD) % NV, (p + AHEAD) / NV);
      else
        af[p + AHEAD] = ra.read(na, (p + AHEAD) % NV, (p + AHEAD - P) / NV);
      // the other operand's next step, spread over the last positions of this one
      constexpr int kBEach = (S::FN + AHEAD - 1) / AHEAD;
      const int q = p % NV - (NV - AHEAD);
      if (q >= 0) {
#pragma unroll
        for (int j = q * kBEach; j < (q + 1) * kBEach && j < S::FN; ++j) {
          if (s + 1 < STEPS)
            bf[s + 1][j] = rb.read(sb, j, s + 1);
          else
            bf[STEPS][j] = rb.read(nb, j, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < S::FN; ++j)
        acc[p % NV][j] = tile_mma<F16>(bf[s][j], af[p], acc[p % NV][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < S::FN; ++j) bf[0][j] = bf[STEPS][j];
#pragma unroll
    for (int p = 0; p < AHEAD; ++p) af[p] = af[P + p];
  }
};

template <class S>
__device__ __forceinline__ void tile_zero(floatx4 (&acc)[S::FM][S::FN]) {
#pragma unroll
  for (int i = 0; i < S::FM; ++i)
#pragma unroll
    for (int j = 0; j < S::FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
}

// The loop over k of one tile.
template <class S, bool ACOL, bool BCOL, bool F16, int NV>
__device__ __forceinline__ void tile_kloop(const OperandLoader<S::BM, S::kWaves, ACOL>& la,
                                           const OperandLoader<S::BN, S::kWaves, BCOL>& lb,
                                           int64_t k, unsigned char* smem, int wave, int lane,
                                           floatx4 (&acc)[S::FM][S::FN]) {
  const int nk = (int)((k + kStageK - 1) / kStageK);
  if (nk == 0) return;
  unsigned char* const aring = smem;
  unsigned char* const bring = smem + S::AST * S::kABytes;
  constexpr int LA = OperandLoader<S::BM, S::kWaves, ACOL>::L;
  constexpr int LB = OperandLoader<S::BN, S::kWaves, BCOL>::L;
  static_assert(S::BST * (LA + LB) < 64, "vmcnt range");
  // a wave's loads are issued, and counted, in the order A(t), B(t + BST - AST): behind the loads of
  // stage t + 1 came B's of that turn, if B runs ahead, and both operands' of AST - 2 turns
  constexpr int kBehind = (S::AST - 2) * (LA + LB) + (S::BST > S::AST ? LB : 0);
  auto issue_a = [&](int st) { la.issue(st, k, aring + (st % S::AST) * S::kABytes, wave); };
  auto issue_b = [&](int st) { lb.issue(st, k, bring + (st % S::BST) * S::kBBytes, wave); };
#pragma unroll
  for (int p = 0; p < S::BST; ++p) {
    if (p < S::AST && p < nk) issue_a(p);
    if (p < nk) issue_b(p);
  }
  if (nk >= S::BST)
    __builtin_amdgcn_s_waitcnt(vmcnt_imm((S::AST - 1) * LA + (S::BST - 1) * LB));
  else
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  tile_barrier();
  TileStage<S, ACOL, BCOL, F16, NV> stage;
  stage.init(wave, lane);
  stage.start(aring, bring);
  int ia = 0, ib = 0;   // ring slots of the stage
  for (int kt = 0; kt < nk; ++kt) {
    const int ja = ia + 1 == S::AST ? 0 : ia + 1, jb = ib + 1 == S::BST ? 0 : ib + 1;
    stage.run(aring + ia * S::kABytes, bring + ib * S::kBBytes, aring + ja * S::kABytes,
              bring + jb * S::kBBytes,
              [&]() {
                // own reads of this stage are done; own loads of the next one have landed
                if (kt + S::BST <= nk)
                  __builtin_amdgcn_s_waitcnt(vmcnt_imm(kBehind) & kLgkmZero);
                else
                  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0) & kLgkmZero);
                tile_barrier();
                if (kt + S::AST < nk) la.issue(kt + S::AST, k, aring + ia * S::kABytes, wave);
                if (kt + S::BST < nk) lb.issue(kt + S::BST, k, bring + ib * S::kBBytes, wave);
              },
              acc);
    ia = ja;
    ib = jb;
  }
}

// Hands a tile's accumulators (NV row sub-tiles a wave) on in row order: put(i, j, p) writes the lane's
// four values of acc[i][j] (column 16 j + 4 (lane / 16) of the wave's columns) to LDS at p, kSize
// bytes each, and get(m, n, p) takes the 16 bytes at p, the values of row m from column n on (of the
// tile). A wave's rows of one sub-tile lie in LDS as 16 rows 16 bytes apart from a multiple of
// 256 (no bank conflicts); `smem` is the tile's ring, which nobody reads or fills any more: the last
// stage's barrier stands behind its last reads.
//
// A CU stores 35 GB/s in runs of 64 bytes, as the accumulators lie, and 140 GB/s in long rows: a
// 256 x 256 fp32 tile takes 7.3 us or 1.9 (measured with one workgroup a CU, 8 to 256 CUs).
template <class S, int NV, int kSize, class Put, class Get>
__device__ __forceinline__ void tile_rows(unsigned char* smem, int wave, int lane, Put&& put,
                                          Get&& get) {
  constexpr int kRow = S::FN * 16 * kSize, kPitch = kRow + 16, kBuf = 16 * kPitch;
  static_assert(S::kWaves * 2 * kBuf <= S::kLdsBytes, "staging fits the ring");
  // lanes of a row (the last ones idle where its chunks are no power of two), rows an instruction
  constexpr int kChunks = kRow / 16;
  constexpr int kLanes = kChunks <= 4 ? 4 : kChunks <= 8 ? 8 : kChunks <= 16 ? 16 : 32;
  constexpr int kRows = 64 / kLanes;
  static_assert(kChunks <= kLanes && kRows <= 16, "whole rows");
  unsigned char* const mine = smem + wave * 2 * kBuf;
  const int wm = wave / S::WN, wn = wave % S::WN;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    unsigned char* const buf = mine + (i & 1) * kBuf;
#pragma unroll
    for (int j = 0; j < S::FN; ++j)
      put(i, j, buf + (lane & 15) * kPitch + (16 * j + 4 * (lane >> 4)) * kSize);
    // the lanes read each other's values: the compiler keeps the order (no instruction)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int p = 0; p < 16 / kRows; ++p) {
      const int r = p * kRows + lane / kLanes, c = lane % kLanes;
      if (kChunks == kLanes || c < kChunks)
        get(16 * S::row_tile(wm, i) + r, wn * S::FN * 16 + c * (16 / kSize),
            buf + r * kPitch + 16 * c);
    }
  }
}

// Stores a tile's accumulators: rows m < rows and columns n < cols, cols a multiple of 8, of the tile
// whose first value is at `out`, `ld` bytes from row to row (a tile's rows under 2 GiB). Lanes
// outside are dropped by the buffer's bounds.
template <class S, int NV, bool OUT_BF16>
__device__ __forceinline__ void tile_store(const floatx4 (&acc)[S::FM][S::FN], void* out, int64_t ld,
                                           int rows, int cols, unsigned char* smem, int wave,
                                           int lane) {
  constexpr int kSize = OUT_BF16 ? 2 : 4;
  const uint32_t bytes = (uint32_t)((min(rows, S::BM) - 1) * ld + min(cols, S::BN) * kSize);
  const auto rsrc =
      __builtin_amdgcn_make_buffer_rsrc(uniform(out), (short)0, uniform((int)bytes), 0x00020000);
  tile_rows<S, NV, kSize>(
      smem, wave, lane,
      [&](int i, int j, unsigned char* p) {
        const floatx4 v = acc[i][j];
        if constexpr (OUT_BF16)
          *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)};
        else
          *reinterpret_cast<floatx4*>(p) = v;
      },
      [&](int m, int n, const unsigned char* p) {
        const uint32_t off = (uint32_t)(m * ld + n * kSize);
        __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const u32x4*>(p), rsrc,
                                               m < rows && n < cols ? off : 0x80000000u, 0, 0);
      });
}

}  // namespace beam
