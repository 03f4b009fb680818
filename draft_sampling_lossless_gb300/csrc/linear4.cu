// Products with 4-bit weights: which kernel runs.
#include "linear4.cuh"

namespace dspark {

size_t linear4_workspace_bytes(int T, int K) { return linear4_tile_workspace_bytes(T, K); }

// The kernel of a few rows starts sooner (5000 cycles of a call to 7400: no tensor memory, no
// descriptors, no split of x), the tiles' takes far less a weight.
cudaError_t launch_linear4(const Linear4Args& a, cudaStream_t st) {
  const bool fits = linear4_rows_fits(a.T, a.w->Kp);
  const int64_t rows = fits ? linear4_rows_cycles(a) : 0;
  if (fits && rows <= 3000) return launch_linear4_rows(a, st);  // (whatever the tiles' cut)
  TileCut cut;
  const cudaError_t e = linear4_tile_cut(a, &cut);
  if (e != cudaSuccess) return e;
  if (fits && rows <= cut.cycles + 2400) return launch_linear4_rows(a, st);
  return launch_linear4_tile(a, cut, st);
}

}  // namespace dspark
