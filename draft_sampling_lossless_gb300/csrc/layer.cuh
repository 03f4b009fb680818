// The target's layers around its attention: the host description of 4-bit weights,
// what their kernels share, and the launchers.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace dspark {

// What the opaque words of a dspark_weights4 hold.  The store: tiles of 128 rows by 128 columns,
// [ceil(N / 128)][Kp / 128], Kp = K rounded up to 128, each its codes [128][64 bytes] and then
// its scales, one run of 8704 bytes.  (With codes in rows of K, 4100 rows of
// x gated by 2 x 10240 x 2560 took 2% longer, one by 6144 x 2560 3%.)
struct Weights4Desc {
  uint64_t magic;
  int N, K, Kp, pad;
  uint8_t* store;
  CUtensorMap tm;  // boxes of a tile's codes, spread to a byte each
};
constexpr uint64_t kWeights4Magic = 0x6473706b77347834ull;
constexpr int kTileCodes = 8192, kTileBytes = kTileCodes + 512;

__host__ __device__ constexpr int padded_k(int K) { return (K + 127) / 128 * 128; }
constexpr size_t weights4_bytes(int N, int K) {
  return (size_t)((N + 127) / 128) * (padded_k(K) / 128) * kTileBytes;
}
// The tile of row n, columns 32 g .. 32 g + 31; in it, their 16 bytes of codes, and their scale:
// [n % 32][n / 32 % 4][g % 4], as tcgen05.cp spreads 512 bytes over tensor memory's lanes (32 of
// them) and columns.
__host__ __device__ constexpr size_t tile_at(int n, int g, int Kp) {
  return ((size_t)(n >> 7) * (Kp >> 7) + (g >> 2)) * kTileBytes;
}
__host__ __device__ constexpr int code_in_tile(int n, int g) { return (n & 127) * 64 + (g & 3) * 16; }
__host__ __device__ constexpr int scale_in_tile(int n, int g) {
  return kTileCodes + (n & 31) * 16 + ((n >> 5) & 3) * 4 + (g & 3);
}

// out[t][n] = x[t] . W[n], or act(x[t] . G[n]) * (x[t] . U[n]).
struct Linear4Args {
  const Weights4Desc *w, *up;  // up: the second matrix of a gated product, else null
  int act;                     // DSPARK_ACT_*
  int T;
  const __nv_bfloat16* x;
  int64_t x_stride;
  __nv_bfloat16* out;
  int64_t out_stride;
  void* ws;
};
size_t linear4_workspace_bytes(int T, int K);
cudaError_t launch_linear4(const Linear4Args& a, cudaStream_t st);

cudaError_t launch_weights4_load(const Weights4Desc& d, const uint8_t* codes,
                                 const uint8_t* scales, cudaStream_t st);
cudaError_t launch_weights4_quantize(const Weights4Desc& d, const void* src, int dt,
                                     int64_t stride, cudaStream_t st);

struct NormArgs {
  int T, d, dt;
  float alpha, eps, inv_d;
  const void* x;
  int64_t x_stride;
  const __nv_bfloat16 *y, *gate;
  int64_t y_stride, gate_stride;
  const float *post, *pre;
  void* x_out;
  int64_t x_out_stride;
  __nv_bfloat16* h;
  int64_t h_stride;
};
cudaError_t launch_norm(const NormArgs& a, cudaStream_t st);

}  // namespace dspark
