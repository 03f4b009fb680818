// The paged key/value cache's host description and the lookups its kernels
// share: which request a packed row belongs to, and where a position lives.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace dspark {

// What the opaque words of a dspark_cache hold.
struct CacheDesc {
  uint64_t magic;
  int format, Hkv, page, D;
  int64_t n_pages;
  void *k, *v;
  uint8_t *k_exp, *v_exp;
  CUtensorMap tm_k, tm_v;
};
constexpr uint64_t kCacheMagic = 0x6473706b63616368ull;

// The pools and the batch, as the kernels take them.
struct CacheView {
  int R, T, Hkv, D, log_page, max_pages;
  int64_t n_pages;
  void *k, *v;
  uint8_t *k_exp, *v_exp;
  const int32_t *row_off, *ctx, *pages;
  uint32_t* status;
};

// The request of packed row t: the largest n in [0, R) with row_off[n] <= t
// (row_off ascending), -1 if there is none.  Warp-collective.  A pass narrows the
// range 128-fold with four independent loads a lane, so one round trip to
// memory settles batches of up to 128 requests.
__device__ __forceinline__ int find_request(const int32_t* row_off, int R, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = R;
  for (;;) {
    const int step = (hi - lo + 127) / 128;
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = lo + (int64_t)(i * 32 + lane) * step;
      cnt += __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(row_off + at) <= t));
    }
    if (cnt == 0) return -1;
    lo += (cnt - 1) * step;
    hi = hi < lo + step ? hi : lo + step;
    if (step == 1) return lo;
  }
}

// Index of the (page, head 0, slot 0) row group of position p of request n, in
// pages; -1 (and the flag) where the table or the id does not cover it.
__device__ __forceinline__ int64_t page_of(const CacheView& c, int n, int64_t p) {
  const int64_t at = p >> c.log_page;
  if (at < c.max_pages) {
    const int id = __ldg(c.pages + (int64_t)n * c.max_pages + at);
    if (id >= 0 && id < c.n_pages) return id;
  }
  set_flag(c.status, kFlagPageRange);
  return -1;
}

// Two values rounded to e4m3 (to nearest even, to the largest past it; NaN stays).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// An exponent byte as it counts: 0, 254 and 255 are never written, and their powers of two
// are no normal floats of bf16's or fp32's (or leave no room for a code).
__device__ __forceinline__ uint32_t exponent_byte(uint32_t b) { return min(max(b, 1u), 253u); }

// The launchers: enqueue on `st`.
cudaError_t launch_cache_append(const CacheView& c, bool e4m3, const void* k, int64_t k_stride,
                                const void* v, int64_t v_stride, cudaStream_t st);
cudaError_t launch_cache_read(const CacheView& c, bool e4m3, void* k_out, void* v_out,
                              cudaStream_t st);

struct AttendArgs {
  CacheView c;
  const CacheDesc* desc;
  int Hq, max_rows, causal, window;
  float scale;
  const void* q;
  int64_t q_stride;
  void* out;
  float* lse;
  void* ws;
};
size_t attend_workspace_bytes(int T, int group, int D);
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st);

}  // namespace dspark
