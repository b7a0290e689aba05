// matvec.cuh -- matrix products for a few tokens (at most 16), where reading the weights is the
// whole cost: bf16 weights (the feed-forward block's small batches) and 4-bit weights with group
// scales (one matrix, or the routed and shared experts of a decode batch).
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMvTokens = 16;    // tokens of one launch
constexpr int kMvRows = 16;      // output rows of a unit (the MMA's M)
constexpr int kInt4Cols = 128;   // columns of a block of 4-bit codes
constexpr int kMvMaxSlots = kMvTokens * kMaxTopK;

// ---- the 4-bit format ------------------------------------------------------------------------
// w[r][c] = scale[r][c / group] * (code[r][c] - zero[r][c / group]), code and zero 0..15 (zero 8
// where a matrix has none), scale bf16, group 32, 64 or 128.
// Codes are laid out for the MMA's A fragments: blocks of 16 rows x 128 columns (1024 bytes), row tiles
// outermost, each two halves of 64 columns (512 bytes). In a half, lane 4 q + c of a warp owns 16 bytes:
// the columns 32 h + 8 c .. 32 h + 8 c + 7 (h = 0, 1) of rows q and q + 8. Its 32-bit word 2 h + i holds,
// for the columns k = 32 h + 8 c + 4 i + {0, 1, 2, 3}: bits 4 n .. 4 n + 3 for n = 0..7 are
//   (q, k), (q + 8, k), (q, k + 2), (q + 8, k + 2), (q, k + 1), (q + 8, k + 1), (q, k + 3), (q + 8, k + 3)
// so that one mask of both half words gives two neighbouring columns of a row.
// Scales: per row tile, then per block, then per q = 0..7, then per group of the block, the entries of
// rows q and q + 8, so that a lane's entries lie together. An entry is the bf16 scale, or, with zero
// points, the scale (low half word) and bf16(128 + zero) (high half word). Groups past the last column
// have entries too.
__host__ __device__ inline int64_t int4_row_tiles(int64_t rows) { return (rows + kMvRows - 1) / kMvRows; }
__host__ __device__ inline int64_t int4_blocks(int64_t cols) { return (cols + kInt4Cols - 1) / kInt4Cols; }
__host__ __device__ inline int64_t int4_code_bytes(int64_t rows, int64_t cols) {
  return int4_row_tiles(rows) * int4_blocks(cols) * (kMvRows * kInt4Cols / 2);
}
__host__ __device__ inline int64_t int4_scale_bytes(int64_t rows, int64_t cols, int group, bool zeros) {
  return int4_row_tiles(rows) * int4_blocks(cols) * (kInt4Cols / group) * kMvRows * (zeros ? 4 : 2);
}
// Entry of (row r of the tile, group g) among a tile's.
__host__ __device__ inline int int4_scale_at(int r, int g, int group) {
  const int n = kInt4Cols / group;
  return (g / n) * kMvRows * n + (r & 7) * 2 * n + (g % n) * 2 + (r >> 3);
}

// One or two matrices of equal shape (two: up and gate), bf16 [R][K] or 4-bit.
struct MvMatrix {
  const void* w[2];
  const void* scales[2];
  int32_t R, K;          // of one expert's matrix
};

struct MvArgs {
  MvMatrix m;            // routed experts' matrices one after another, or the one matrix
  MvMatrix shared;       // R (up) or K (down) 0: no shared expert
  const uint16_t* x;     // bf16 activations, row stride ldx
  int64_t ldx;
  int32_t T;             // 1..16
  int32_t group;         // 4-bit: columns a scale covers
  int32_t early;         // weights, ids and topk_w may be read before the kernel in front is done
  // experts
  const int32_t* ids;    // [T][k], entries outside [0, E) are skipped
  const float* topk_w;   // [T][k]
  int32_t E, k;
  int32_t capacity;      // tokens an expert takes, the lowest first (0: all)
  // results
  void* out;             // row stride ldo
  int64_t ldo;
  int32_t out_bf16;
  uint16_t* u;           // dual, one matrix: also the pre-activations (or null), row stride ldo
  uint16_t* g;
};

// kind: what a unit of 16 rows is
enum MvKind : int {
  kMvOne = 0,      // one matrix (dual: a pair): out[t] = W x_t (dual: SwiGLU)
  kMvUp = 1,       // dual, per expert hit: h of its tokens, a row each (experts and tokens in rising
                   // order), and of the shared expert at rows T * k + t
  kMvDown = 2,     // sum over the experts hit (and the shared one): out[t] = sum w W_down h
};

cudaError_t launch_mv_bf16(const MvArgs& a, bool dual, int num_sms, cudaStream_t stream);
cudaError_t launch_mv_int4(const MvArgs& a, int kind, bool zeros, int num_sms, cudaStream_t stream);
// bf16 src [R][K] -> codes and scales; and codes two to a byte [R][K / 2] with scales [R][groups]
// and zeros [R][groups] (or null) -> the layout above.
cudaError_t launch_int4_quantize(const uint16_t* src, int64_t R, int64_t K, int group, bool zeros, void* codes,
                                 void* scales, int num_sms, cudaStream_t stream);
cudaError_t launch_int4_pack(const uint8_t* q, const uint16_t* s, const uint8_t* z, int64_t R, int64_t K, int group,
                             void* codes, void* scales, int num_sms, cudaStream_t stream);

}  // namespace moe
