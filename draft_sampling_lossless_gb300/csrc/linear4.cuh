// What the kernels of the 4-bit products share.
#pragma once

#include "dspark.h"
#include "layer.cuh"

namespace dspark {

// silu, or gelu's tanh form.  exp and tanh in full fp32: their errors stay far below the
// result's rounding.
__device__ __forceinline__ float activation(int act, float a) {
  if (act == DSPARK_ACT_SILU) return a / (1.f + expf(-a));
  return 0.5f * a * (1.f + tanhf(0.7978845608028654f * fmaf(0.044715f * a * a, a, a)));
}

// The kernel on the tensor cores (linear4_tile.cu).
size_t linear4_tile_workspace_bytes(int T, int K);
cudaError_t launch_linear4_tile(const Linear4Args& a, cudaStream_t st);

// The kernel of a few rows (linear4_rows.cu): up to 16, as many as fit in shared memory.
bool linear4_rows_fits(int T, int Kp);
cudaError_t launch_linear4_rows(const Linear4Args& a, cudaStream_t st);

}  // namespace dspark
