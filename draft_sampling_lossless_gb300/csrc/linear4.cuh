// What the kernels of the 4-bit products share.
#pragma once

#include "dspark.h"
#include "layer.cuh"
#include "sm100.cuh"

namespace dspark {

// silu(a) = a s(a); gelu's tanh form, 0.5 a (1 + tanh y) = a s(2 y), with s(v) = 1 / (1 +
// exp(-v)).  ex2.approx and the quick division are off by 2^-21 or so (2^-24 |v| in the exponent
// on top), far below the result's rounding.  exp(-v) past 2^126 gives 0.
__device__ __forceinline__ float activation(int act, float a) {
  float v = a;
  if (act != DSPARK_ACT_SILU) v = 1.5957691216057308f * fmaf(0.044715f * a * a, a, a);
  const float d = 1.f + sm100::ex2_approx(-1.4426950408889634f * v);
  return __fdividef(a, d);
}

// The kernel on the tensor cores (linear4_tile.cu), and how it cuts a product.
struct TileCut {
  int mats;      // row tiles of 128 (of W, or one each of two matrices) that share a block's x
  int tokens;    // rows of x a tile
  int wide;      // hi and lo of x as 2 * tokens columns of one MMA, else an MMA each
  int split;     // blocks that share a tile's K
  bool own;      // the blocks split x into hi and lo themselves (one tile each), no kernel before
  int64_t cycles;  // an estimate of its time but for what every call takes
};
size_t linear4_tile_workspace_bytes(int T, int K);
cudaError_t linear4_tile_cut(const Linear4Args& a, TileCut* cut);
cudaError_t launch_linear4_tile(const Linear4Args& a, const TileCut& cut, cudaStream_t st);

// The kernel of a few rows (linear4_rows.cu): up to 32, as many as fit in shared memory.
bool linear4_rows_fits(int T, int Kp);
int64_t linear4_rows_cycles(const Linear4Args& a);
cudaError_t launch_linear4_rows(const Linear4Args& a, cudaStream_t st);

}  // namespace dspark
