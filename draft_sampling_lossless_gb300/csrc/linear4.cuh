// What the kernels of the 4-bit products share.
#pragma once

#include "dspark.h"
#include "layer.cuh"
#include "sm100.cuh"

namespace dspark {

// silu(a) = a s(a); gelu's tanh form, 0.5 a (1 + tanh y) = a s(2 y), with s(v) = g / (g + 1 / g),
// g = exp(v / 2): v / 2, so that s is right down to the subnormals, where silu(-88) lies (times a
// large second factor an ordinary number; 1 / (1 + exp(-v)) ends at exp(-v) = 2^126, for
// 18.9 us instead of 19.0 with 122 rows gated by 2 x 10240 x 2560).  Above 2 ln 2^120 s is 1.
// ex2.approx and rcp.approx are off by 2^-21 or so together (2^-24 |v| in the exponent on top),
// far below the result's rounding.  A NaN stays one by the factor a.
__device__ __forceinline__ float activation(int act, float a) {
  float v = a;
  if (act != DSPARK_ACT_SILU) v = 1.5957691216057308f * fmaf(0.044715f * a * a, a, a);
  const float t = fminf(0.72134752044448170f * v, 120.f);
  const float g = sm100::ex2_approx(t);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(g + sm100::ex2_approx(-t)));
  return a * (g * r);
}

// Codes p and p + 4 of a word as two bf16, 2^-126 of their values (0.5 is a subnormal).
template <int P>
__device__ __forceinline__ uint32_t pair_bits(uint32_t w) {
  const uint32_t u = P == 3 ? w : w << (12 - 4 * P);
  return (u & 0x80008000u) | ((u >> 6) & 0x01c001c0u);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 c = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&c);
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
