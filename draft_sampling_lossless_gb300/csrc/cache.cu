// Paged key/value cache: the new rows written into their pages (bf16, or
// quantised to e4m3 with a power-of-two scale), and cached positions read back.
//
// Both move each byte once and compute next to nothing, so HBM bounds them:
// 2 * Hkv * (2 D read + 2 D or D + 1 written) bytes a row for the append, the
// reverse for the read.  One warp takes one row: it has four 16-byte
// loads a lane in flight, the append's issued before the request lookup that
// says where they go, so the lookup's round trips hide behind them.  More loads a
// lane leave room for fewer warps and are slower (eight, in blocks of eight warps:
// 79 us for 68 below).
//
// Measured (8 heads of 128): nine prompts of 1500 to 6000 rows written as e4m3 and read
// back 66 us, 5.4 TB/s (80% of the measured copy rate: the conversions and the exponents,
// single bytes, come on top); 24 prefixes of 500 to 8000 rows of bf16 read 118 us,
// 6.7 TB/s (99%); 64 requests' 1 to 8 rows of bf16 written 6.2 us, latency.
#include "cache.cuh"

namespace dspark {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMinExp = -100;  // smallest exponent kept for a row

// The smallest e >= kMinExp with amax <= 448 * 2^e (amax finite, >= 0).
// 448 = 1.75 * 2^8: amax = 1.f * 2^E gives E - 8 up to 1.75, E - 7 above.
__device__ __forceinline__ int row_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return e < kMinExp ? kMinExp : e;
}

// Two e4m3 codes (low and high byte of `w`) times f, as packed bf16.  Every
// code is a half, and its product with a power of two exact in bf16 as long as
// it is a normal number there.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t w, float f) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  const float2 x = __half22float2(*reinterpret_cast<__half2*>(&h));
  const __nv_bfloat162 y = __floats2bfloat162_rn(x.x * f, x.y * f);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// A warp's row in pieces of 16 bytes of bf16: unit u = (k or v, head), piece c
// of its D / 8.  A unit takes LP lanes (a power of two, for the reduction), so
// 32 / LP units a step.
template <int LP>
struct Piece {
  int u, c;
  bool ok;
  __device__ __forceinline__ Piece(const CacheView& v, int step) {
    const int lane = threadIdx.x & 31;
    u = step * (32 / LP) + lane / LP;
    c = lane % LP;
    ok = u < 2 * v.Hkv && c < (v.D >> 3);
  }
};

template <bool E4M3, int LP>
__global__ void __launch_bounds__(kThreads)
    cache_append_kernel(const CacheView c, const __nv_bfloat16* __restrict__ k, int64_t k_stride,
                        const __nv_bfloat16* __restrict__ v, int64_t v_stride) {
  constexpr int kBatch = 4;
  grid_dependency_wait();  // the rows, the tables, the pools
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= c.T) return;
  const int steps = (2 * c.Hkv * LP + 31) / 32;
  int64_t page = -1;
  int slot = 0;
  for (int s0 = 0; s0 < steps; s0 += kBatch) {
    uint4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const Piece<LP> p(c, s0 + i);
      x[i] = make_uint4(0, 0, 0, 0);
      if (p.ok) {
        const __nv_bfloat16* src =
            p.u < c.Hkv ? k + t * k_stride + (int64_t)p.u * c.D
                        : v + t * v_stride + (int64_t)(p.u - c.Hkv) * c.D;
        x[i] = __ldcs(reinterpret_cast<const uint4*>(src + p.c * 8));
      }
    }
    if (s0 == 0) {
      const int n = find_request(c.row_off, c.R, t);
      if (n < 0 || t >= __ldg(c.row_off + n + 1)) return;
      const int64_t pos = (int64_t)__ldg(c.ctx + n) + (t - __ldg(c.row_off + n));
      if (pos < 0) return;
      page = page_of(c, n, pos);
      if (page < 0) return;
      slot = (int)(pos & ((1 << c.log_page) - 1));
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (s0 + i >= steps) break;
      const Piece<LP> p(c, s0 + i);
      const bool is_k = p.u < c.Hkv;
      const int64_t row = ((page * c.Hkv + (is_k ? p.u : p.u - c.Hkv)) << c.log_page) + slot;
      if constexpr (!E4M3) {
        if (p.ok)
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_k ? c.k : c.v) + row * c.D +
                                    p.c * 8) = x[i];
      } else {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] = __uint_as_float(w[j] << 16);
          f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
        // the largest magnitude: bf16 without the sign are ordered as 16-bit integers
        constexpr uint32_t kMag = 0x7fff7fffu;
        uint32_t top = __vmaxu2(__vmaxu2(w[0] & kMag, w[1] & kMag),
                                __vmaxu2(w[2] & kMag, w[3] & kMag));
#pragma unroll
        for (int o = LP / 2; o > 0; o >>= 1)
          top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
        float amax = __uint_as_float(max(top >> 16, top & 0xffffu) << 16);
        bool finite = true;
        if (__any_sync(0xffffffffu, !(amax < INFINITY))) {  // of the finite values, then
          amax = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float a = fabsf(f[j]);
            const bool fin = a < INFINITY;
            finite &= fin;
            amax = fmaxf(amax, fin ? a : 0.f);
          }
#pragma unroll
          for (int o = LP / 2; o > 0; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        }
        const int e = row_exponent(amax);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t code[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) code[j] = e4m3x2(f[2 * j] * inv, f[2 * j + 1] * inv);
        if (p.ok) {
          if (!finite) set_flag(c.status, kFlagNonFinite);
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_k ? c.k : c.v) + row * c.D +
                                    p.c * 8) =
              make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
          if (p.c == 0) (is_k ? c.k_exp : c.v_exp)[row] = (uint8_t)(e + 127);
        }
      }
    }
  }
}

template <bool E4M3, int LP>
__global__ void __launch_bounds__(kThreads)
    cache_read_kernel(const CacheView c, __nv_bfloat16* __restrict__ k_out,
                      __nv_bfloat16* __restrict__ v_out) {
  constexpr int kBatch = 4;
  grid_dependency_wait();  // the rows, the tables, the pools
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= c.T) return;
  const int n = find_request(c.row_off, c.R, t);
  if (n < 0 || t >= __ldg(c.row_off + n + 1)) return;
  const int64_t pos = (int64_t)__ldg(c.ctx + n) + (t - __ldg(c.row_off + n));
  const int64_t page = pos < 0 ? -1 : page_of(c, n, pos);
  const int slot = (int)(pos & ((1 << c.log_page) - 1));
  const int steps = (2 * c.Hkv * LP + 31) / 32;
  for (int s0 = 0; s0 < steps; s0 += kBatch) {
    uint4 x[kBatch];
    int e[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const Piece<LP> p(c, s0 + i);
      x[i] = make_uint4(0, 0, 0, 0);
      e[i] = 127;
      if (p.ok && page >= 0) {
        const bool is_k = p.u < c.Hkv;
        const int64_t row = ((page * c.Hkv + (is_k ? p.u : p.u - c.Hkv)) << c.log_page) + slot;
        if constexpr (E4M3) {
          const uint2 y = __ldcs(reinterpret_cast<const uint2*>(
              static_cast<const uint8_t*>(is_k ? c.k : c.v) + row * c.D + p.c * 8));
          x[i].x = y.x;
          x[i].y = y.y;
          e[i] = (is_k ? c.k_exp : c.v_exp)[row];
        } else {
          x[i] = __ldcs(reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(is_k ? c.k : c.v) + row * c.D + p.c * 8));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const Piece<LP> p(c, s0 + i);
      if (!p.ok) continue;
      uint4 y = x[i];
      if constexpr (E4M3) {
        const float f = __uint_as_float(exponent_byte(e[i]) << 23);  // 2^(byte - 127)
        y = make_uint4(e4m3x2_to_bf16x2(x[i].x & 0xffffu, f), e4m3x2_to_bf16x2(x[i].x >> 16, f),
                       e4m3x2_to_bf16x2(x[i].y & 0xffffu, f), e4m3x2_to_bf16x2(x[i].y >> 16, f));
      }
      const bool is_k = p.u < c.Hkv;
      __nv_bfloat16* dst = (is_k ? k_out : v_out) +
                           ((int64_t)t * c.Hkv + (is_k ? p.u : p.u - c.Hkv)) * c.D + p.c * 8;
      __stcs(reinterpret_cast<uint4*>(dst), y);
    }
  }
}

}  // namespace

cudaError_t launch_cache_append(const CacheView& c, bool e4m3, const void* k, int64_t k_stride,
                                const void* v, int64_t v_stride, cudaStream_t st) {
  auto kernel = c.D > 64 ? (e4m3 ? cache_append_kernel<true, 16> : cache_append_kernel<false, 16>)
                         : (e4m3 ? cache_append_kernel<true, 8> : cache_append_kernel<false, 8>);
  cudaError_t e;
  DSPARK_LAUNCH(kKindCacheAppend, st,
                e = launch_pdl(kernel, dim3((c.T + kWarps - 1) / kWarps), dim3(kThreads), 0, st, c,
                               static_cast<const __nv_bfloat16*>(k), k_stride,
                               static_cast<const __nv_bfloat16*>(v), v_stride));
  return e;
}

cudaError_t launch_cache_read(const CacheView& c, bool e4m3, void* k_out, void* v_out,
                              cudaStream_t st) {
  auto kernel = c.D > 64 ? (e4m3 ? cache_read_kernel<true, 16> : cache_read_kernel<false, 16>)
                         : (e4m3 ? cache_read_kernel<true, 8> : cache_read_kernel<false, 8>);
  cudaError_t e;
  DSPARK_LAUNCH(kKindCacheRead, st,
                e = launch_pdl(kernel, dim3((c.T + kWarps - 1) / kWarps), dim3(kThreads), 0, st, c,
                               static_cast<__nv_bfloat16*>(k_out),
                               static_cast<__nv_bfloat16*>(v_out)));
  return e;
}

}  // namespace dspark
