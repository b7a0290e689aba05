// ffn.cuh -- what the gated feed-forward block's kernels and their host side share.
//
// The block (the layer's W_shared term, or a dense layer's FFN; Mixture-of-Kittens layer equation):
//   u = x W_up^T,  g = x W_gate^T,  h = SiLU(u) (.) g,  out = h W_down^T
// and, for a loss L with dout = dL/dout,
//   dh = dout W_down,              s = 1 / (1 + exp(-u))
//   dg = dh (.) u s,               du = dh (.) g (.) s (1 + u (1 - s))
//   dx = du W_up + dg W_gate
//   dW_up = du^T x,  dW_gate = dg^T x,  dW_down = dout^T h
// Every one of these products is an instance of D[M][N] = sum_k A(m, k) B(n, k) with A and B each
// stored either with k contiguous ("K-major") or with m or n contiguous ("MN-major"), so that no
// operand is ever transposed in memory.
//
// Rounded to bf16, once each: h, du and dg, because they are operands of the next products and the tensor cores take
// their operands in 16 bits (tf32 would run at half the rate and twice the bytes; the layer's expert GEMMs round
// their h alike), u and g for the backward pass, and each bf16 result. Sums, splits' partials and the activation are in
// fp32. An output's error against 64 bits is then that of two roundings, 2.35e-3 of its norm, where one, of the result
// alone, gives 1.66e-3.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kFfnTileM = 256;   // rows of the MMA, and the most of an output tile (128 per CTA of a pair)
constexpr int kFfnMaxBN = 256;   // most columns of an output tile
constexpr int kFfnMaxProblems = 4;
constexpr int kFfnRaster = 8;    // m-tiles walked side by side, so that their B tiles stay in L2

// One product of a launch. A unit of work is (m-tile, n-tile, K split).
struct alignas(64) FfnProblem {
  CUtensorMap a[2], b[2];  // per K segment (dx has two: du W_up + dg W_gate); with b_by_rank,
                           // b[r] is what CTA r of the pair stages (W_up rows | W_gate rows)
  CUtensorMap out;         // bf16 or fp32 [M][N] (fp32 partials [splits * mpad][N] when splits > 1)
  int32_t mt, nt;          // tiles along M and N
  int32_t bn;              // columns per tile, a multiple of 16 in 64..256
  int32_t nrows, ncols;    // M, N (what lies past them is not stored)
  int32_t mrows;           // rows of a tile per CTA, at most 128: the MMA's other rows hold leftovers, not stored
  int32_t nkb, nseg;       // 64-wide K blocks per segment, segments
  int32_t a_mn, b_mn;      // 1: MN-major
  int32_t b_by_rank;
  int32_t splits, mpad;    // K splits; rows between two splits' partials (mt * 2 * mrows)
  int32_t unit0;           // first unit of this problem in the launch
  int32_t out_kind;        // 0 bf16, 1 fp32, 2 fp32 added to what is there
  int32_t gcol;            // partials of u | g: column of g's part
  uint32_t panel_inv;      // 2^32 / (kFfnRaster * nt), rounded up
};

struct FfnParams {
  FfnProblem p[kFfnMaxProblems];
  CUtensorMap out2, out3;  // up: u, g (save); dh: dg, h
  CUtensorMap in_u, in_g;  // dh: the saved pre-activations [M][N], boxes of {32 columns, 128 rows}
  int32_t nprob, units;
  int32_t save;            // up: also store u and g
  DeviceMeta* meta;
  int64_t timeout_ns;
};

// What an epilogue does with the accumulators of a tile.
enum FfnEpilogue : int {
  kFfnStore = 0,    // D -> out
  kFfnSwiglu = 1,   // columns [0, bn/2) are u, [bn/2, bn) the matching g: h -> out (u, g -> out2, out3)
  kFfnDSwiglu = 2,  // D is dh: du -> out, dg -> out2, h -> out3
};

cudaError_t launch_ffn_gemm(const FfnParams& p, int epilogue, int pairs, cudaStream_t stream);

// Sums K-split partials (fp32, `splits` of [mpad][ld]) in split order and applies an epilogue:
// store: out[M][N] in out_kind; swiglu: u at columns [0, N), g at [gcol, gcol + N); dswiglu.
struct FfnReduce {
  const float* parts;
  int64_t split_stride;  // elements between two splits
  int64_t ld;            // elements between two rows of a partial
  int32_t splits, rows, cols, gcol;
  int32_t out_kind;
  void* out;
  uint16_t* out2;
  uint16_t* out3;        // null: not stored
  const uint16_t* u;
  const uint16_t* g;
};
cudaError_t launch_ffn_reduce(const FfnReduce& r, int epilogue, int num_sms, cudaStream_t stream);

// ---- the activation, in fp32 -----------------------------------------------------------------
// exp through the fast-math intrinsic (a few units in fp32's last place, far below the bf16
// rounding of the results). exp(-u) overflows to infinity for u < -88: the quotient is then 0.
__device__ __forceinline__ float swiglu(float u, float g) { return __fdividef(u, 1.0f + __expf(-u)) * g; }

__device__ __forceinline__ void dswiglu(float dh, float u, float g, float& du, float& dg, float& h) {
  const float s = __fdividef(1.0f, 1.0f + __expf(-u));
  const float a = u * s;
  dg = dh * a;
  du = dh * g * (s * (1.0f + u * (1.0f - s)));
  h = a * g;
}

}  // namespace moe
