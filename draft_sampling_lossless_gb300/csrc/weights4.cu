// 4-bit weights laid out for the products: given codes and scales copied, or a bf16 or
// fp32 matrix quantised.  Once a matrix, so simple: HBM bounds both, and the scales' single
// bytes cost more than the copy.
#include "dspark.h"
#include "layer.cuh"

namespace dspark {

namespace {

constexpr int kThreads = 256;

// A thread a group of 32 columns (16 bytes of codes), rows padded to 128, columns to 128.
__global__ void __launch_bounds__(kThreads)
    load_kernel(const Weights4Desc d, const uint8_t* __restrict__ codes,
                const uint8_t* __restrict__ scales) {
  grid_dependency_wait();
  const int groups = d.Kp >> 5, used = d.K >> 5;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t n = i / groups;
  const int g = (int)(i - n * groups);
  if (n >= (d.N + 127) / 128 * 128) return;
  const bool in = n < d.N && g < used;
  uint4 c = make_uint4(0, 0, 0, 0);
  int b = 127;
  if (in) {
    c = __ldg(reinterpret_cast<const uint4*>(codes) + n * used + g);
    b = __ldg(scales + n * used + g);
  }
  uint8_t* tile = d.store + tile_at((int)n, g, d.Kp);
  *reinterpret_cast<uint4*>(tile + code_in_tile((int)n, g)) = c;
  tile[scale_in_tile((int)n, g)] = (uint8_t)min(max(b, 1), 252);
}

__device__ __forceinline__ float finite_abs(float v) {
  v = fabsf(v);
  return v < INFINITY ? v : 0.f;
}

// Four lanes a group, eight values each.  The smallest e with max |v| <= 6 * 2^e (6 = 1.5 *
// 2^2), so that nothing is cut off; codes to nearest, ties to the even code.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const Weights4Desc d, const T* __restrict__ src, int64_t stride) {
  grid_dependency_wait();
  const int groups = d.Kp >> 5;
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 2;
  const int q = threadIdx.x & 3;
  const int64_t n = i / groups;
  const int g = (int)(i - n * groups);
  const bool in = n < d.N && g < (d.K >> 5);
  float v[8] = {};
  if (in) {
    const T* p = src + n * stride + g * 32 + q * 8;
    uint4 raw[sizeof(T) / 2];
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) raw[j] = __ldg(reinterpret_cast<const uint4*>(p) + j);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = to_f32(reinterpret_cast<const T*>(raw)[j]);
  }
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, finite_abs(v[j]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const uint32_t b = __float_as_uint(amax);
  const int e =
      min(max((int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x400000u ? 2 : 1), -100), 125);
  const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = v[j] == v[j] ? v[j] * f : 0.f;
  uint32_t c;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(c)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  if (n >= (d.N + 127) / 128 * 128) return;
  uint8_t* tile = d.store + tile_at((int)n, g, d.Kp);
  *reinterpret_cast<uint32_t*>(tile + code_in_tile((int)n, g) + q * 4) = in ? c : 0u;
  if (q == 0) tile[scale_in_tile((int)n, g)] = (uint8_t)(in ? e + 127 : 127);
}

int64_t blocks_for(const Weights4Desc& d, int lanes) {
  const int64_t rows = (d.N + 127) / 128 * 128;
  return (rows * (d.Kp >> 5) * lanes + kThreads - 1) / kThreads;
}

}  // namespace

cudaError_t launch_weights4_load(const Weights4Desc& d, const uint8_t* codes,
                                 const uint8_t* scales, cudaStream_t st) {
  cudaError_t e;
  DSPARK_LAUNCH(kKindWeights4, st,
                e = launch_pdl(load_kernel, dim3((unsigned)blocks_for(d, 1)), dim3(kThreads), 0,
                               st, d, codes, scales));
  return e;
}

cudaError_t launch_weights4_quantize(const Weights4Desc& d, const void* src, int dt,
                                     int64_t stride, cudaStream_t st) {
  const dim3 grid((unsigned)blocks_for(d, 4));
  cudaError_t e;
  DSPARK_LAUNCH(kKindWeights4, st,
                e = dt == DSPARK_F32
                        ? launch_pdl(quantize_kernel<float>, grid, dim3(kThreads), 0, st, d,
                                     static_cast<const float*>(src), stride)
                        : launch_pdl(quantize_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st,
                                     d, static_cast<const __nv_bfloat16*>(src), stride));
  return e;
}

}  // namespace dspark
