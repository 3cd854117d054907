// experts_kernel.cuh -- parameters shared by the host side (moe.cu) and the
// kernel of the products grouped by expert (experts_kernel.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace agg {

// The products of the kernel.  "Wide" is the output's contiguous dimension,
// the MMA's M; "rows" its N.
enum ExpertsOp : int {
  kOpForward = 0,   // y[r][n]  = sum_k x[r][k] w[e][k][n]     wide n, rows r, over k
  kOpInput = 1,     // dx[r][k] = sum_n dy[r][n] w[e][k][n]    wide k, rows r, over n
  kOpWeight = 2,    // dw[e][k][n] = sum_r x[r][k] dy[r][n]    wide n, rows k, over e's rows r
  kOpFp8 = 3,       // y[r][n] with e4m3 operands and scales   wide n, rows r, over k
  kOpFp8Long = 4,   // the same with rows as the MMA's M (chosen by the launcher)
  kOpFp4 = 5,       // y[r][n] with e2m1 operands and e8m0 scales, over k
};

constexpr int kXWide = 256;    // a pair's tile: 256 of the wide dimension
constexpr int kXRows = 256;    // and up to 256 rows,
constexpr int kXFewRows = 64;  // or up to 64 where groups are short
constexpr int kXRows4 = 224;   // e2m1: up to 224 (two accumulators of 224 leave TMEM columns for the scales)
constexpr int kXRowBoxes = 4;  // box heights of the row operand: a quarter of half a tile, in whole 8 rows, to all of it
__host__ __device__ constexpr int box_step(int tile_rows) { return (tile_rows / 8 + 7) / 8 * 8; }
__host__ __device__ constexpr int box_height(int tile_rows, int boxes) {
  return kXRowBoxes * box_step(tile_rows) > tile_rows / 2 && boxes == kXRowBoxes ? tile_rows / 2
                                                                               : boxes * box_step(tile_rows);
}
constexpr int kXSub = 2;       // k-blocks of 128 bytes per stage of the ring
constexpr int kXEpiWarps = 16;
constexpr int kCopyWarps = 2, kPassWarps = 4;
// TMA warp, MMA warp, epilogue warps; the weight gradient's zeroing warp, the scale warp
// of e4m3, or those of e2m1, two that copy and four that pass on.
__host__ __device__ constexpr int threads_of(int op) {
  return 32 * (2 + kXEpiWarps + (op == kOpForward || op == kOpInput ? 0 : op == kOpFp4 ? kCopyWarps + kPassWarps : 1));
}
constexpr int kXGroup = 8;     // row tiles that share the weights they read (tile order)

struct ExpertsParams {
  CUtensorMap tm_w;              // the wide operand
  CUtensorMap tm_r[kXRowBoxes];  // the row operand, by box height (weight gradient: of 128 and of 64 columns)
  const int32_t* offsets;        // [E + 1], or null: one group of all rows
  int32_t E;
  int32_t rows;                  // rows of the inputs
  int32_t wide;                  // extent of the wide dimension
  int32_t red;                   // length of the sums (weight gradient: unused)
  int32_t out_rows;              // weight gradient: output rows per expert (K)
  int32_t step, row_tiles;       // weight gradient: output rows of a tile, 256 or 128; tiles of K
  uint32_t inv_group, inv_expert;  // floor((2^32 - 1) / n): n tiles of 8 row tiles, n of an expert (weight gradient)
  int32_t w_blk, r_blk;          // operand described in blocks of 128 bytes (one load a stage), or not (two)
  int32_t segment;               // k-blocks per accumulator (e4m3: 1)
  int32_t bf16;                  // operands are bfloat16 (otherwise fp16)
  int32_t out_type;              // ElemType of the output
  int32_t rows32;                // 16-bit output whose rows start at multiples of 32 bytes
  void* out;
  int64_t ldo;
  const float* xs;               // e4m3: row scales [KB][rows]
  const float* ws;               // e4m3: weight scales [E][NB][KB]
  float* partials;               // split sums: [unit][warps of the pair][columns][32 lanes]
  uint32_t* arrivals;            // [tile][warps of the pair], zero between runs
  int32_t max_units;             // units the workspace holds (0: never split)
  uint32_t* status;              // [4]: status word and detail of a wait that ran out, which ends the waits
                                 // of later runs too; the same of bad offsets, which concern their run alone
  uint64_t timeout_ns;
  // (here, so that what the other products read stays where it was: further in, the e4m3 kernel
  // of long groups spilt more registers, and 8192 rows on 32 experts took 344 us instead of 336)
  const uint32_t* xs4;           // e2m1: row scales, four to a word, [ceil(K / 128)][rows]
  uint32_t inv_stages;           // e2m1: floor((2^32 - 1) / stages of a sum)
  CUtensorMap tm_s;              // e2m1: the weights' scales, pieces of 128 rows x 4 scales side by side
};

// A unit of a split sum: each warp's columns x 32 lanes of floats.
constexpr int64_t split_unit_bytes(bool few) {
  return 2 * kXEpiWarps * (static_cast<int64_t>(few ? kXFewRows : kXRows) / 4) * 32 * 4;
}

// Prices of splitting a sum, in k-blocks of its variant: once a round, and for each part
// (choose_split says what they stand for).
struct SplitPrice {
  int32_t once, part;
};
__host__ __device__ constexpr SplitPrice split_price(int op, bool short_tiles) {
  return op == kOpFp8 ? SplitPrice{9, 1}
         : op == kOpFp8Long ? SplitPrice{9, 3}
         : op == kOpFp4 ? SplitPrice{short_tiles ? 7 : 9, short_tiles ? 1 : 3}
         : op == kOpWeight ? SplitPrice{14, short_tiles ? 3 : 5}  // half tiles, whole ones
                           : SplitPrice{14, short_tiles ? 2 : 5};
}
constexpr int kMaxSplit = 16, kMinPart = 4;  // parts of a sum; k-blocks of a part

constexpr uint32_t kStatusOffsets = 16;  // status word: offsets decrease or leave [0, rows]

// Kernel attributes; the number of CTA pairs that are resident at once.
cudaError_t experts_prepare(int* pairs);
cudaError_t launch_experts(const ExpertsParams& p, int op, bool few, int grid,
                           cudaStream_t stream);

}  // namespace agg
