// Products with 4-bit weights: which kernel runs.
#include "linear4.cuh"

namespace dspark {

size_t linear4_workspace_bytes(int T, int K) { return linear4_tile_workspace_bytes(T, K); }

cudaError_t launch_linear4(const Linear4Args& a, cudaStream_t st) {
  return linear4_rows_fits(a.T, a.w->Kp) ? launch_linear4_rows(a, st) : launch_linear4_tile(a, st);
}

}  // namespace dspark
