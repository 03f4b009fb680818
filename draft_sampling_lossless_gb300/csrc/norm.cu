// The norms between two blocks of the target: the block's output through its own norm,
// gate and scale into the stream, and the next block's norm of the stream.
//
//   x' = x + alpha * gate * rms(y) * post,  h = rms(x') * pre
//
// Every value is read once and written once, and little is computed, so HBM bounds it:
// a row stays in the registers of its block between the two sums of squares.  h comes
// from x' before its rounding, so that each output is rounded once.
#include "dspark.h"
#include "layer.cuh"

namespace dspark {

namespace {

// Eight values of a row from `i` on.
__device__ __forceinline__ void load8(const float* p, int i, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p + i)[0];
  const float4 b = reinterpret_cast<const float4*>(p + i)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int i, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p + i);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, int i, const float (&v)[8]) {
  reinterpret_cast<float4*>(p + i)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p + i)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int i, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A block a row, V pieces of eight values a thread.
template <typename T, int V>
__global__ void __launch_bounds__(1024) norm_kernel(const NormArgs a) {
  __shared__ float sh[32];
  grid_dependency_wait();
  const int64_t t = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
  float v[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = (k * blockDim.x + threadIdx.x) * 8;
    if (i < a.d) {
      load8(x, i, v[k]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = 0.f;
    }
  }
  if (a.y != nullptr) {
    const __nv_bfloat16* y = a.y + t * a.y_stride;
    const __nv_bfloat16* gate = a.gate == nullptr ? nullptr : a.gate + t * a.gate_stride;
    float u[V][8], sum = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int i = (k * blockDim.x + threadIdx.x) * 8;
      if (i < a.d) {
        load8(y, i, u[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(u[k][j], u[k][j], sum);
      }
    }
    float r = 1.f;
    if (a.post != nullptr) r = 1.f / sqrtf(block_sum(sum, sh) / a.d + a.eps);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int i = (k * blockDim.x + threadIdx.x) * 8;
      if (i < a.d) {
        float g[8];
        if (a.post != nullptr) {
          load8(a.post, i, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[k][j] = u[k][j] * r * g[j];
        }
        if (gate != nullptr) {
          load8(gate, i, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[k][j] *= g[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = fmaf(a.alpha, u[k][j], v[k][j]);
        if (a.x_out != nullptr) store8(static_cast<T*>(a.x_out) + t * a.x_out_stride, i, v[k]);
      }
    }
  }
  if (a.h == nullptr) return;
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(v[k][j], v[k][j], sum);
  const float r = 1.f / sqrtf(block_sum(sum, sh) / a.d + a.eps);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = (k * blockDim.x + threadIdx.x) * 8;
    if (i < a.d) {
      float g[8];
      load8(a.pre, i, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * r * g[j];
      store8(a.h + t * a.h_stride, i, v[k]);
    }
  }
}

template <typename T>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
  const int pieces = a.d / 8;
  const int V = pieces <= 1024 ? 1 : pieces <= 2048 ? 2 : 4;
  const int threads = ((pieces + V - 1) / V + 31) / 32 * 32;
  auto kernel = V == 1 ? norm_kernel<T, 1> : V == 2 ? norm_kernel<T, 2> : norm_kernel<T, 4>;
  cudaError_t e;
  DSPARK_LAUNCH(kKindNorm, st, e = launch_pdl(kernel, dim3(a.T), dim3(threads), 0, st, a));
  return e;
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  return a.dt == DSPARK_F32 ? launch<float>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace dspark
