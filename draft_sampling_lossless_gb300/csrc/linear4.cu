// Products with 4-bit weights: x W^T, and act(x G^T) * (x U^T).
#include "linear4.cuh"

namespace dspark {

namespace {

constexpr int kWarps = 4, kTokens = 4;

__device__ __forceinline__ float code_value(uint32_t c) {
  const uint32_t e = (c >> 1) & 3, f = c & 1;
  const float v = e == 0 ? 0.5f * f : (1.f + 0.5f * f) * (float)(1u << (e - 1));
  return c & 8 ? -v : v;
}

// A warp a feature and kTokens tokens, a lane a group of 32 columns.
__global__ void __launch_bounds__(kWarps * 32)
    linear4_simple(const Weights4Desc w, const Weights4Desc up, int mats, int act, int T,
                   const __nv_bfloat16* __restrict__ x, int64_t x_stride,
                   __nv_bfloat16* __restrict__ out, int64_t out_stride) {
  grid_dependency_wait();
  const int n = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int t0 = blockIdx.y * kTokens;
  if (n >= w.N) return;
  float sum[2][kTokens] = {};
  for (int m = 0; m < mats; ++m) {
    const Weights4Desc& d = m ? up : w;
    for (int g = lane; g < d.K / 32; g += 32) {
      const uint4 c4 = reinterpret_cast<const uint4*>(d.codes)[(int64_t)n * (d.Kp >> 5) + g];
      const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
      const float s = __uint_as_float((uint32_t)d.scales[scale_at(n, g, d.Kp)] << 23);
      for (int t = 0; t < kTokens && t0 + t < T; ++t) {
        const __nv_bfloat16* p = x + (t0 + t) * x_stride + g * 32;
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          a = fmaf(code_value(c[j / 8] >> (4 * (j % 8))), to_f32(p[j]), a);
        sum[m][t] = fmaf(a, s, sum[m][t]);
      }
    }
  }
  for (int t = 0; t < kTokens && t0 + t < T; ++t) {
    float a = warp_sum(sum[0][t]), b = warp_sum(sum[1][t]);
    if (mats == 2) a = activation(act, a) * b;
    if (lane == 0) out[(t0 + t) * out_stride + n] = __float2bfloat16(a);
  }
}

}  // namespace

size_t linear4_workspace_bytes(int T, int K) { return linear4_tile_workspace_bytes(T, K); }

cudaError_t launch_linear4(const Linear4Args& a, cudaStream_t st) {
  if (a.T > 16) return launch_linear4_tile(a, st);
  const int per = 65535 * kTokens;  // the grid's second dimension
  cudaError_t e = cudaSuccess;
  for (int t = 0; t < a.T && e == cudaSuccess; t += per) {
    const int T = a.T - t < per ? a.T - t : per;
    DSPARK_LAUNCH(kKindLinear4, st,
                  e = launch_pdl(linear4_simple,
                                 dim3((a.w->N + kWarps - 1) / kWarps, (T + kTokens - 1) / kTokens),
                                 dim3(kWarps * 32), 0, st, *a.w, a.up ? *a.up : *a.w,
                                 a.up ? 2 : 1, a.act, T, a.x + t * a.x_stride, a.x_stride,
                                 a.out + t * a.out_stride, a.out_stride));
  }
  return e;
}

}  // namespace dspark
