// Host-side rules of the operators that close a training step (gfx950): tiles, launch and workspace sizes
// of the gated products, of the head's loss and of the AdamW step. Plain C++, as train_rules.h.
#pragma once

#include "train_rules.h"

namespace beam {

// ---- gated products grouped by expert ----
// A tile's columns are half gate, half up, in sub-tiles of 16 in turn, so each wave needs an even
// number of them: every tile of the grouped products but the 32 x 64 one. The products' rule (train_rules.h), over
// the 2 F rows of the weights. Measured (us) 32 x 128, 64 x 64, 128 x 128, then 128, 192, 256, 320 x 256, the rule's
// choice last: 32 experts of 5120 -> 2560, 32 rows in all 181, 175, 181, 174, 181, 195, 233: 181; 2048 rows 472, 455,
// 348, 302, 310, 327, 367: 307; 8192 rows 1304, 988, 670, 591, 549, 520, 423 to 517: the last; 279 rows of one expert, 4152 ->
// 1056: 27, 25, 50, 41, 54, 60, 92: 25. Over 27 random calls the rule's choice took 6% more than the best tile.
template <class S>
constexpr int kGatedCols = S::BN / 2;
template <class F>
void with_gated_tile(int64_t R, int64_t E, int64_t Fw, int64_t K, bool keep, F&& f) {
  const RowsCall call(R, E, 2 * Fw, K, R * (Fw * (keep ? 6e-6 : 2e-6)));
  with_least([&](auto s) { return call.us(s); }, f, TileStream{}, Tile64{}, TilePair{}, Tile128{}, Tile192{},
             Tile256Deep{}, Tile320{});
}

// Few rows of few experts make few tiles, each a chain of stages: blocks of 32 rows by kNarrowCols hidden values instead,
// the contraction split over a workgroup's waves, where those are at most one and a half a CU and the chain is long.
// Measured (us, the tiles first, on weights out of memory, then on weights that the last call left in the cache): one
// row, 5120 -> 2560, 160 blocks, 31.8, 17.4, then 29.4, 13.7; 8 rows, 4624 -> 944, 59: 29.9, 16.5, 22.2, 10.7; 4 rows, 4096
// -> 4096, 256: 27.5, 17.6, 25.8, 15.3; one row or so of each of 4 experts, 5120 -> 2560, 320 to 640: 33.5, 35.3, 32.2,
// 28.1; 16 rows, 4096 -> 8192, 512: 32.2, 37.3, 29.7, 31.7; 20 rows of 16 experts, 2048 -> 704, 528: 18.1, 24.4, 15.6, 22.0;
// 128 rows, 4096 -> 1024, 256: 26.7, 21.2, 22.7, 19.5; 16 rows, 2048 -> 1024, 64: 14.1, 9.7, 11.5, 8.7; 30 rows, 1024 ->
// 2560, 160: 9.1, 9.6, 7.7, 8.2. Turns of a wave at once: five; with eight the first three are, in the cache, 15.7, 12.8
// and 13.4 (fewer of them past the end of most contractions).
constexpr int kNarrowWaves = 8, kNarrowAhead = 5, kNarrowCols = 16;
bool gated_is_narrow(int64_t R, int64_t E, int64_t Fw, int64_t K);

// The gradient's tiles: F columns, contraction over the hidden width; 10 bytes a value beside dy. Measured as above,
// 32 x 64 second: 32 experts of 5120 -> 2560, 2048 rows 257, 361, 258, 211, 171, 175, 185, 215: 175; 32768 rows 2136,
// 4024, 1881, 1121, 1102, 1002, 975, 899: 899; 9 rows of 9 experts, 4688 -> 624: 30, 25, 29, 59, 38, 42, 61, 71: 25.
// Over 18 random calls 3% more than the best tile.
template <class F>
void with_gated_bwd_tile(int64_t R, int64_t E, int64_t Fw, int64_t H, F&& f) {
  const RowsCall call(R, E, Fw, H, R * (Fw * 10e-6));
  with_least([&](auto s) { return call.us(s); }, f, TileStream{}, TileLone{}, Tile64{}, TilePair{}, Tile128{},
             Tile192{}, Tile256Deep{}, Tile320{});
}
// Partial sums of the scales' gradient: one for the columns of a wave, or of a wave of its half tile.
template <class S>
constexpr int kScaleCols = kHalves<S> ? S::FN * 8 : S::FN * 16;
constexpr int kLeastScaleCols = 16;
inline int64_t gated_scale_parts(int64_t Fw) { return ceil_div(Fw, kLeastScaleCols); }

// ---- loss of the output head ----
// Logits: the grouped products' rule for one expert of V columns, by tile shape; `store`: their gradient is
// stored, in bf16. Measured (us, the loss, tiles as for the gated products, the rule's choice last): one token, 131072 x
// 5120: 208, 222, 213, 197, 197, 205, 269: 208; 755 tokens, 23413 x 3624: 369, 284, 198, 172, 146, 171, 177: 154;
// 2499, 39407 x 2784: 1240, 944, 603, 625, 571, 539, 478: 478; the gradient's logits of 154, 72560 x 720: 59, 46, 43,
// 45, 39, 40, 41: 39. Over 16 random calls of the loss 8% more than the best tile.
template <class F>
void with_head_tile(int64_t T, int64_t V, int64_t H, bool store, F&& f) {
  const RowsCall call(T, 1, V, H, store ? T * (V * 2e-6) : 0.0);
  with_least([&](auto s) { return call.us(s); }, f, TileStream{}, Tile64{}, TilePair{}, Tile128{}, Tile192{},
             Tile256Deep{}, Tile320{});
}
// Few tokens and columns (`end` of them, to the pitch for the gradient): blocks of 32 tokens by kNarrowLogits columns
// as for the gated products, where they are at most one a CU. Measured (us, the loss's logits, then the gradient's, the
// tiles first, on weights out of memory): one token, 1000 x 1280, 32 blocks, 9.8, 7.1 and 9.6, 6.6; 2, 300 x 5120, 10:
// 29.7, 15.8 and 30.4, 16.0; 8, 4096 x 4096, 128: 26.2, 15.7 and 25.3, 15.9; 32 of them 26.3, 21.6 and 25.4, 21.8; 16, 8192
// x 5120, 256: 33.7, 23.9 and 32.7, 24.3; 32, 8000 x 1600, 250: 12.8, 11.7 and 12.0, 11.5; 128, 2048 x 4096, 256: 27.9, 20.6
// and 26.2, 20.4. 384 blocks: one, 12288 x 5120 35.2, 34.1 and 38.8, 39.7; 32, 12288 x 2048 16.4, 24.0 and 15.7, 23.4; 64,
// 6144 x 5120 35.9, 45.0 and 33.8, 46.3. On weights that the last call left in the cache the tiles gain more: the
// gradient's are ahead of two of these blocks (32 tokens: 17.7, 18.7 and 9.1, 10.0), the loss's of none.
constexpr int kNarrowLogits = 32;
inline bool head_is_narrow(int64_t T, int64_t end, int64_t H) {
  return H >= 1280 && ceil_div(T, 32) * ceil_div(end, kNarrowLogits) <= kGroupedCus;
}
// Column slots of a row's partial sums: one a tile, two where a tile may be split.
template <class S>
int64_t head_slots(int64_t V) {
  return ceil_div(V, S::BN) * (kHalves<S> ? 2 : 1);
}

// Gradient of x: tiles of T x H, the contraction over a piece of the vocabulary cut into `parts` runs of
// `kp` values (whole stages), each with FP32 sums of its own that are added in order: by a model of the time (full
// rounds of workgroups, a tile's ends and stages, the sums' traffic). Measured (us, with the addition): 154 x 720, 72560
// columns: 128 x 128 in 43 parts 35, in 21 41, 256 x 256 in 85 39, 64 x 64 in 43 46, 32 x 128 in 17 44; 2048 x 4096,
// 65536: 256 x 256 in 2 parts 868, in 1 1470, in 4 922, 128 x 128 in 1 1013; 256 x 5120, 131072: 256 x 256 in 12
// parts 368, in 13 (a second round) 580; 9 x 2264, 15625: 64 x 64 in 21 parts 15.6, 32 x 128 in 14 15.9, 128 x 128 in
// 28 16.5.
struct HeadDxPlan {
  int side;       // tile: 256, 128 or 64 square, 32: 32 x 128
  int parts;
  int64_t kp;
};
using DxTile256 = TileShape<256, 256, 2, 4, 2, 2>;
using DxTile128 = TileShape<128, 128, 2, 2, 2, 2>;
using DxTile64 = TileShape<64, 64, 1, 2, 3, 3>;
using DxTile32 = TileShape<32, 128, 1, 4, 4, 4>;
HeadDxPlan head_dx_plan(int64_t T, int64_t H, int64_t cols);

// Workspace of the loss (byte offsets): partial maxima and sums [slots][T], the targets' logits [T].
struct HeadLayout {
  size_t at_target = 0, total = 0;
  int64_t slots = 0;
};
HeadLayout head_layout(int64_t T, int64_t V, int64_t H);
// Workspace of its gradient: a piece of the logits' gradient over c, [T][pitch] bf16; c and its inverse without
// d_loss [2][T]; bf16(c x) [T][H]; the sums of dx [parts][T][H] FP32 unless one part of one piece is all there is.
struct HeadBwdLayout {
  int64_t cols = 0, pieces = 0, pitch = 0;   // columns of a piece; its row length
  HeadDxPlan dx = {};
  size_t c = 0, xc = 0, sums = 0, total = 0;
  bool direct() const { return pieces == 1 && dx.parts == 1; }
};
// Columns of a piece: what 512 MiB of dz hold, but 32768 where 4 GiB do (each piece reads and writes T x H sums of dx,
// 8 bytes against 2 columns' products: 3% of a piece of 32768), and never under 512 (16 GiB of 2^24 tokens). 4096
// tokens, 131072 x 5120, in pieces of 256 MiB, 512 MiB, 1 GiB: 13.5, 13.3, 13.25 ms.
constexpr int64_t kHeadPieceBytes = int64_t(512) << 20, kHeadMostBytes = int64_t(4) << 30;
constexpr int64_t kHeadPieceCols = 32768, kHeadLeastCols = 512;
HeadBwdLayout head_bwd_layout(int64_t T, int64_t V, int64_t H);
bool head_grid_fits(int64_t T, int64_t V, int64_t H);

// ---- AdamW step ----
// A workgroup's chunk: kAdamwUnroll blocks of 256 values a wave. Tensors of a launch without a table: what the
// kernel's arguments (4 KB) hold. A table: its head, an entry for each tensor that has values, each chunk's entry.
struct AdamwTableHead {
  int32_t entries, chunks, types, unused;   // types: adamw_types
};
// The random bits of stochastic rounding: the published integer hash lowbias32 of seed, step and the value's number.
constexpr uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}
// The types that a table's arrays have, which a launch of others must not follow. From one on: a table of zeros has none.
constexpr int32_t adamw_types(bool p_bf16, bool g_bf16, bool q8, bool copy) {
  return 1 + (p_bf16 ? 1 : 0) + (g_bf16 ? 2 : 0) + (q8 ? 4 : 0) + (copy ? 8 : 0);
}
struct AdamwEntry {
  AdamwTensor t;
  int32_t first;     // its first chunk
  int32_t base256;   // blocks of 256 values before it in the whole list
};
constexpr int kAdamwThreads = 256, kAdamwUnroll = 4, kAdamwChunkBlocks = kAdamwThreads / 64 * kAdamwUnroll;
constexpr int kAdamwTensors = 54;
static_assert(sizeof(AdamwEntry) == 72, "one layout on host and device");
constexpr int64_t kAdamwMostChunks = (int64_t(1) << 32) / kAdamwThreads - 1;   // threads of a launch
constexpr int64_t kAdamwMostValues = kAdamwMostChunks * kAdamwChunkBlocks * 256;
inline int64_t adamw_chunks(int64_t count) { return ceil_div(count, kAdamwChunkBlocks * 256); }

bool gated_grid_fits(int64_t R, int64_t E, int64_t Fw, int64_t K);
bool gated_bwd_grid_fits(int64_t R, int64_t E, int64_t Fw, int64_t H);

}  // namespace beam
