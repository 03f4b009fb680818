// The norms between two blocks of the target: the block's output through its own norm,
// gate and scale into the stream, and the next block's norm of the stream.
//
//   x' = x + alpha * gate * rms(y) * post,  h = rms(x') * pre
//
// Every value is read once and written once, and little is computed, so HBM bounds it:
// a row stays in the registers of its block between the two sums of squares, its loads
// issued together.  h comes from x' before its rounding, so that each output is rounded once.
//
// Measured: 16000 rows of 2560, fp32 stream, norms on both sides and one gate 72.2 us, 6.8
// TB/s (100% of the measured copy rate); 16000 of 7168, bf16 stream, a gate a row 191 us, 6.0
// TB/s; 300 of those 4.3 us; one row of 2560 1.9 us, latency (among calls in a graph).
#include <type_traits>

#include "dspark.h"
#include "layer.cuh"

namespace dspark {

namespace {

// Eight values of a row, as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
};
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The block's sum, in every thread and always in the same order; `sh` is used once.
__device__ __forceinline__ float row_sum(float v, float* sh) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < (int)(blockDim.x >> 5) ? sh[lane] : 0.f);
}

// rms(v) = (v * s) * q, from the sum of a row's squares.  Where that left fp32's range (values
// past 2^56 or so; where eps leaves it to them, below 2^-48) it is taken again of the values
// times s, a power of two; else s is 1.  Two factors, since their product may be past 2^128 (a
// row of subnormals); 2^100 times the largest of the small rows still has its square in range, and
// so has 2^100 times the smallest subnormal.  each(f) calls f for each of this thread's values.
struct Factor {
  float s, q;
};
template <class Each>
__device__ __forceinline__ Factor row_factor(float sum, float inv_d, float eps, float* sh,
                                             Each&& each) {
  if (sum <= 0x1p112f && (sum >= 0x1p-96f || eps >= 0x1p-80f))  // (the same in every thread)
    return {1.f, __frsqrt_rn(fmaf(sum, inv_d, eps))};
  const float s = sum < 1.f ? 0x1p100f : 0x1p-75f;
  float again = 0.f;
  each([&](float v) {
    v *= s;
    again = fmaf(v, v, again);
  });
  return {s, __frsqrt_rn(fmaf(row_sum(again, sh), inv_d, eps * s * s))};
}

// A block a row, V pieces of eight values a thread.  All of a row's loads are issued before
// the first sum.  (Up to 1024 threads with one piece, 512 with more; with two, 56 registers
// leave room for seven blocks of rows of 2560.)
template <typename T, int V>
__global__ void __maxnreg__(V == 1 ? 64 : V == 2 ? 56 : 128) norm_kernel(const NormArgs a) {
  __shared__ float sh[2][64];
  grid_dependency_wait();
  const int64_t t = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
  const __nv_bfloat16* y = a.y == nullptr ? nullptr : a.y + t * a.y_stride;
  const __nv_bfloat16* gate = a.gate == nullptr ? nullptr : a.gate + t * a.gate_stride;
  Raw8<T> rx[V];
  Raw8<__nv_bfloat16> ry[V], rg[V];
  const int i0 = threadIdx.x * 8, step = blockDim.x * 8;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = i0 + k * step;
    if (i < a.d) {
      rx[k].load(x + i);
      if (y != nullptr) ry[k].load(y + i);
      if (gate != nullptr) rg[k].load(gate + i);
    }
  }
  float v[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (i0 + k * step < a.d) {
      rx[k].get(v[k]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = 0.f;
    }
  }
  if (y != nullptr) {
    Factor r = {1.f, 1.f};
    if (a.post != nullptr) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (i0 + k * step < a.d) {
          float u[8];
          ry[k].get(u);
#pragma unroll
          for (int j = 0; j < 8; ++j) sum = fmaf(u[j], u[j], sum);
        }
      r = row_factor(row_sum(sum, sh[0]), a.inv_d, a.eps, sh[0] + 32, [&](auto&& f) {
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (i0 + k * step < a.d) {
            float u[8];
            ry[k].get(u);
#pragma unroll
            for (int j = 0; j < 8; ++j) f(u[j]);
          }
      });
    }
    // In the formula's order, so that what it has in range stays there: y normed before post,
    // alpha by the gate before either meets u.
    auto add = [&](auto scaled) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int i = i0 + k * step;
        if (i < a.d) {
          float u[8], g[8];
          ry[k].get(u);
          if (a.post != nullptr) {
            Raw8<float> w;
            w.load(a.post + i);
            w.get(g);
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = (scaled ? u[j] * r.s : u[j]) * r.q * g[j];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = 1.f;
          if (gate != nullptr) rg[k].get(g);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[k][j] = fmaf(a.alpha * g[j], u[j], v[k][j]);
          if (a.x_out != nullptr) store8(static_cast<T*>(a.x_out) + t * a.x_out_stride + i, v[k]);
        }
      }
    };
    // (A second copy of the loop saves a product: 2000 rows of 2560 7.45 us for 7.6.  With eight
    // pieces it costs registers: 1000 rows of 32768, fp32 stream, 107 us for 103, bf16 78 us both.)
    if (V < 8 && r.s == 1.f) add(std::false_type());
    else add(std::true_type());
  }
  if (a.h == nullptr) return;
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(v[k][j], v[k][j], sum);
  const Factor r = row_factor(row_sum(sum, sh[1]), a.inv_d, a.eps, sh[1] + 32, [&](auto&& f) {
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) f(v[k][j]);
  });
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = i0 + k * step;
    if (i < a.d) {
      Raw8<float> w;
      float g[8];
      w.load(a.pre + i);
      w.get(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * r.s * r.q * g[j];
      store8(a.h + t * a.h_stride + i, v[k]);
    }
  }
}

template <typename T>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
  const int pieces = a.d / 8;
  // One piece a thread is quickest for a few rows (one of 2560: 1.9 us, with two pieces 2.3),
  // two where rows fill the SMs more than once (16000 of 2560 in fp32 72.2 us, with one 75.6, with
  // four 78.1; 300 of 7168 4.3 us and 4.5); longer rows need more.
  const int V = pieces > 2048 ? 8 : pieces > 1024 ? 4 : a.T > sm_count() && pieces > 32 ? 2 : 1;
  const int threads = ((pieces + V - 1) / V + 31) / 32 * 32;
  auto kernel = V == 1   ? norm_kernel<T, 1>
                : V == 2 ? norm_kernel<T, 2>
                : V == 4 ? norm_kernel<T, 4>
                         : norm_kernel<T, 8>;
  cudaError_t e;
  DSPARK_LAUNCH(kKindNorm, st, e = launch_pdl(kernel, dim3(a.T), dim3(threads), 0, st, a));
  return e;
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  return a.dt == DSPARK_F32 ? launch<float>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace dspark
