// Attention of packed rows over the paged cache.
//
// One warp a (row, query head): the lanes take 32 positions at a time for the
// scores, the running maximum and sum of the softmax, then a slice of D each
// for the weighted sum of the values.
#include "cache.cuh"

namespace dspark {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Params {
  CacheView c;
  int Hq, G, max_rows, causal, window;
  float scale;
  const __nv_bfloat16* q;
  int64_t q_stride;
  __nv_bfloat16* out;
  float* lse;
};

// Value d of a cached row (bf16, or an e4m3 code times 2^(byte - 127)).
template <bool E4M3>
__device__ __forceinline__ float cached(const void* pool, const uint8_t* ex, int64_t row, int D,
                                        int d) {
  if constexpr (E4M3) {
    const uint16_t w = static_cast<const uint8_t*>(pool)[row * D + d];
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
    return __half22float2(*reinterpret_cast<__half2*>(&h)).x *
           __uint_as_float((uint32_t)ex[row] << 23);
  } else {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(pool)[row * D + d]);
  }
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads) attend_kernel(const Params p) {
  __shared__ float s_q[kWarps][128];
  const CacheView& c = p.c;
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t job = (int64_t)blockIdx.x * kWarps + wid;
  if (job >= (int64_t)c.T * p.Hq) return;
  const int t = (int)(job / p.Hq), hq = (int)(job % p.Hq), h = hq / p.G;
  const int n = find_request(c.row_off, c.R, t);
  if (n < 0 || t >= c.row_off[n + 1]) return;
  const int j = t - c.row_off[n];
  int m = c.row_off[n + 1] - c.row_off[n];
  if (m > p.max_rows) {
    set_flag(c.status, kFlagRowRange);
    m = p.max_rows;
    if (j >= m) return;
  }
  const int64_t cap = (int64_t)c.max_pages << c.log_page;
  int64_t at = c.ctx[n];
  if (at > cap) at = cap;
  const int64_t pos = at + j;
  const int64_t hi = p.causal ? pos + 1 : at + m;
  const int64_t lo = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
  for (int d = lane; d < c.D; d += 32)
    s_q[wid][d] = __bfloat162float(p.q[(int64_t)t * p.q_stride + (int64_t)hq * c.D + d]);
  __syncwarp();
  float top = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t c0 = lo; c0 < hi; c0 += 32) {
    const int64_t pc = c0 + lane;
    float s = -INFINITY;
    int64_t row = -1;
    if (pc < hi) {
      const int64_t page = page_of(c, n, pc);
      s = 0.f;
      if (page >= 0) {
        row = ((page * c.Hkv + h) << c.log_page) + (pc & ((1 << c.log_page) - 1));
        for (int d = 0; d < c.D; ++d)
          s = fmaf(s_q[wid][d], cached<E4M3>(c.k, c.k_exp, row, c.D, d), s);
      }
      s *= p.scale;
    }
    float mx = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float nt = fmaxf(top, mx);
    const float keep = top == -INFINITY ? 0.f : expf(top - nt);
    top = nt;
    const float e = s == -INFINITY ? 0.f : expf(s - nt);
    float es = e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) es += __shfl_xor_sync(0xffffffffu, es, o);
    sum = sum * keep + es;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= keep;
    for (int l = 0; l < 32; ++l) {
      const float el = __shfl_sync(0xffffffffu, e, l);
      const int64_t rl = __shfl_sync(0xffffffffu, row, l);
      if (rl < 0) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < c.D)
          acc[i] = fmaf(el, cached<E4M3>(c.v, c.v_exp, rl, c.D, lane + 32 * i), acc[i]);
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < c.D)
      p.out[((int64_t)t * p.Hq + hq) * c.D + lane + 32 * i] = __float2bfloat16(acc[i] * inv);
  if (p.lse != nullptr && lane == 0)
    p.lse[(int64_t)t * p.Hq + hq] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st) {
  if (a.c.k_exp == nullptr) return launch_attend_tc(a, st);
  Params p;
  p.c = a.c;
  p.Hq = a.Hq;
  p.G = a.Hq / a.c.Hkv;
  p.max_rows = a.max_rows;
  p.causal = a.causal;
  p.window = a.window;
  p.scale = a.scale;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  const int64_t jobs = (int64_t)a.c.T * a.Hq;
  auto kernel = attend_kernel<true>;
  DSPARK_LAUNCH(kKindAttend, st,
                kernel<<<(unsigned)((jobs + kWarps - 1) / kWarps), kThreads, 0, st>>>(p));
  return cudaGetLastError();
}

}  // namespace dspark
