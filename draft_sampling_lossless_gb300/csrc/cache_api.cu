// C ABI of the paged key/value cache and its attention: argument validation and
// launches (include/dspark.h has the contract).
#include <cudaTypedefs.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "cache.cuh"
#include "dspark.h"

using namespace dspark;

namespace {

static_assert(sizeof(CacheDesc) <= sizeof(dspark_cache), "dspark_cache holds a CacheDesc");

int fail(int code, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  set_error_text(msg);
  return code;
}

int cuda_fail(cudaError_t e, const char* where) {
  return fail(DSPARK_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

#define REQUIRE(p)                                                             \
  do {                                                                         \
    if ((p) == nullptr) return fail(DSPARK_ERR_INVALID_ARG, "%s is NULL", #p); \
  } while (0)
#define REQUIRE_16(p)                                                                        \
  do {                                                                                       \
    REQUIRE(p);                                                                              \
    if (((uintptr_t)(p) & 15) != 0)                                                          \
      return fail(DSPARK_ERR_INVALID_ARG, "%s must be 16-byte aligned", #p);                 \
  } while (0)

// The pools' rows of D values as a 2-D tensor; boxes of one page, or 128 of its
// rows, 128 bytes wide (64 values, or 128 codes) and swizzled as the MMA operands
// they land in.  Values past D read as zeros, rows past the last page too.
cudaError_t encode_pool(CUtensorMap* m, const CacheDesc& d, void* pool) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    return (PFN_cuTensorMapEncodeTiled_v12000) nullptr;
  }();
  if (fn == nullptr) return cudaErrorNotSupported;
  const bool e4m3 = d.k_exp != nullptr;
  const cuuint64_t size = e4m3 ? 1 : 2;
  cuuint64_t dims[2] = {(cuuint64_t)d.D, (cuuint64_t)d.n_pages * d.Hkv * d.page};
  cuuint64_t strides[1] = {(cuuint64_t)d.D * size};
  cuuint32_t box[2] = {e4m3 ? 128u : 64u, (cuuint32_t)(d.page < 128 ? d.page : 128)};
  cuuint32_t es[2] = {1, 1};
  return fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pool,
            dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

bool rows_ok(int R, int T) { return R >= 1 && R <= (1 << 20) && T >= 0 && T <= (1 << 24); }

// Checks what the three calls share and fills the kernels' view.
int view_of(const CacheDesc& d, int R, int T, const int32_t* row_off, const int32_t* ctx,
            const int32_t* pages, int max_pages, void* ws, size_t ws_bytes, size_t ws_need,
            CacheView& c) {
  if (!rows_ok(R, T))
    return fail(DSPARK_ERR_INVALID_ARG, "sizes out of range (R=%d T=%d; need 1<=R<=2^20, 0<=T<=2^24)",
                R, T);
  REQUIRE(row_off);
  REQUIRE(ctx);
  REQUIRE(pages);
  if (max_pages < 1 || (int64_t)max_pages * d.page >= (1 << 30))
    return fail(DSPARK_ERR_INVALID_ARG, "max_pages out of range (%d pages of %d)", max_pages, d.page);
  REQUIRE(ws);
  if (((uintptr_t)ws & 255) != 0) return fail(DSPARK_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  if (ws_bytes < ws_need)
    return fail(DSPARK_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, ws_need);
  c.R = R;
  c.T = T;
  c.Hkv = d.Hkv;
  c.D = d.D;
  c.log_page = 0;
  while ((1 << c.log_page) < d.page) ++c.log_page;
  c.max_pages = max_pages;
  c.n_pages = d.n_pages;
  c.k = d.k;
  c.v = d.v;
  c.k_exp = d.k_exp;
  c.v_exp = d.v_exp;
  c.row_off = row_off;
  c.ctx = ctx;
  c.pages = pages;
  c.status = static_cast<uint32_t*>(ws);
  return DSPARK_OK;
}

int load_desc(const dspark_cache* cache, CacheDesc& d) {
  REQUIRE(cache);
  memcpy(&d, cache, sizeof(d));
  if (d.magic != kCacheMagic)
    return fail(DSPARK_ERR_INVALID_ARG, "cache was not filled by dspark_cache_init");
  return DSPARK_OK;
}

}  // namespace

extern "C" {

int dspark_cache_init(dspark_cache* cache, int format, int64_t n_pages, int Hkv, int page, int D,
                      void* k, void* v, uint8_t* k_exp, uint8_t* v_exp) {
  REQUIRE(cache);
  memset(cache, 0, sizeof(*cache));
  if (format != DSPARK_CACHE_BF16 && format != DSPARK_CACHE_E4M3)
    return fail(DSPARK_ERR_INVALID_ARG, "format must be 0 (bf16) or 1 (e4m3)");
  if (D < 16 || D > 128 || D % 16 != 0)
    return fail(DSPARK_ERR_INVALID_ARG, "D must be a multiple of 16 in [16, 128] (got %d)", D);
  if (page < 16 || page > 1024 || (page & (page - 1)) != 0)
    return fail(DSPARK_ERR_INVALID_ARG, "page must be a power of two in [16, 1024] (got %d)", page);
  if (Hkv < 1 || Hkv > (1 << 16) || n_pages < 1 || n_pages >= (1ll << 31) ||
      n_pages * Hkv >= (1ll << 31) / page)
    return fail(DSPARK_ERR_INVALID_ARG, "n_pages * Hkv * page out of range (%lld, %d, %d)",
                (long long)n_pages, Hkv, page);
  REQUIRE_16(k);
  REQUIRE_16(v);
  if (format == DSPARK_CACHE_E4M3) {
    REQUIRE_16(k_exp);
    REQUIRE_16(v_exp);
  } else if (k_exp != nullptr || v_exp != nullptr) {
    return fail(DSPARK_ERR_INVALID_ARG, "a bf16 cache has no exponents");
  }
  CacheDesc d;
  memset(&d, 0, sizeof(d));
  d.format = format;
  d.Hkv = Hkv;
  d.page = page;
  d.D = D;
  d.n_pages = n_pages;
  d.k = k;
  d.v = v;
  d.k_exp = k_exp;
  d.v_exp = v_exp;
  cudaError_t e = encode_pool(&d.tm_k, d, k);
  if (e == cudaSuccess) e = encode_pool(&d.tm_v, d, v);
  if (e != cudaSuccess) return cuda_fail(e, "dspark_cache_init");
  d.magic = kCacheMagic;
  memcpy(cache, &d, sizeof(d));
  return DSPARK_OK;
}

size_t dspark_cache_workspace_bytes(const dspark_cache* cache, int R, int T, int Hq) {
  CacheDesc d;
  if (load_desc(cache, d) != DSPARK_OK || !rows_ok(R, T)) return 0;
  if (Hq < 1 || Hq % d.Hkv != 0 || Hq / d.Hkv > 128) return 0;
  return attend_workspace_bytes(T, Hq / d.Hkv, d.D);
}

int dspark_cache_append(const dspark_cache* cache, int R, int T, const void* k, int64_t k_stride,
                        const void* v, int64_t v_stride, const int32_t* row_off,
                        const int32_t* ctx, const int32_t* pages, int max_pages, void* ws,
                        size_t ws_bytes, void* stream) {
  CacheDesc d;
  CacheView c;
  int s = load_desc(cache, d);
  if (s) return s;
  if ((s = view_of(d, R, T, row_off, ctx, pages, max_pages, ws, ws_bytes, 256, c))) return s;
  if (T == 0) return DSPARK_OK;
  REQUIRE_16(k);
  REQUIRE_16(v);
  const int64_t row = (int64_t)d.Hkv * d.D;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return fail(DSPARK_ERR_INVALID_ARG,
                "row strides must be multiples of 8 and at least Hkv * D = %lld (got %lld, %lld)",
                (long long)row, (long long)k_stride, (long long)v_stride);
  const cudaError_t e = launch_cache_append(c, d.format == DSPARK_CACHE_E4M3, k, k_stride, v,
                                            v_stride, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "dspark_cache_append");
  return DSPARK_OK;
}

int dspark_cache_read(const dspark_cache* cache, int R, int T, const int32_t* row_off,
                      const int32_t* start, const int32_t* pages, int max_pages, void* k_out,
                      void* v_out, void* ws, size_t ws_bytes, void* stream) {
  CacheDesc d;
  CacheView c;
  int s = load_desc(cache, d);
  if (s) return s;
  if ((s = view_of(d, R, T, row_off, start, pages, max_pages, ws, ws_bytes, 256, c))) return s;
  if (T == 0) return DSPARK_OK;
  REQUIRE_16(k_out);
  REQUIRE_16(v_out);
  const cudaError_t e =
      launch_cache_read(c, d.format == DSPARK_CACHE_E4M3, k_out, v_out, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "dspark_cache_read");
  return DSPARK_OK;
}

int dspark_attend(const dspark_cache* cache, int R, int T, int Hq, int max_rows, float scale,
                  int causal, int window, const void* q, int64_t q_stride,
                  const int32_t* row_off, const int32_t* ctx, const int32_t* pages, int max_pages,
                  void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  CacheDesc d;
  AttendArgs a;
  int s = load_desc(cache, d);
  if (s) return s;
  if (!rows_ok(R, T))
    return fail(DSPARK_ERR_INVALID_ARG, "sizes out of range (R=%d T=%d; need 1<=R<=2^20, 0<=T<=2^24)",
                R, T);
  if (Hq < 1 || Hq % d.Hkv != 0 || Hq / d.Hkv > 128)
    return fail(DSPARK_ERR_INVALID_ARG,
                "Hq must be a multiple of Hkv, at most 128 times it (Hq=%d Hkv=%d)", Hq, d.Hkv);
  if ((int64_t)T * (Hq / d.Hkv) > (1 << 30))
    return fail(DSPARK_ERR_INVALID_ARG, "T * Hq / Hkv must be at most 2^30");
  if (max_rows < 0) return fail(DSPARK_ERR_INVALID_ARG, "max_rows must be >= 0 (got %d)", max_rows);
  if (!isfinite(scale) || !(scale > 0.0f))
    return fail(DSPARK_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (window < 0 || (window > 0 && !causal))
    return fail(DSPARK_ERR_INVALID_ARG, "window must be >= 0, and 0 when not causal (got %d)", window);
  if ((s = view_of(d, R, T, row_off, ctx, pages, max_pages, ws, ws_bytes,
                   attend_workspace_bytes(T, Hq / d.Hkv, d.D), a.c)))
    return s;
  if (T == 0) return DSPARK_OK;
  REQUIRE_16(q);
  REQUIRE_16(out);
  if (q_stride < (int64_t)Hq * d.D || q_stride % 8 != 0)
    return fail(DSPARK_ERR_INVALID_ARG,
                "q's row stride must be a multiple of 8 and at least Hq * D = %lld (got %lld)",
                (long long)Hq * d.D, (long long)q_stride);
  a.desc = &d;
  a.Hq = Hq;
  a.max_rows = max_rows == 0 || max_rows > T ? T : max_rows;
  a.causal = causal != 0;
  // No position reaches 2^30 + 2^24 (pages, then rows): a larger window is the same one, and
  // the kernels' 32-bit differences of positions and windows hold.
  constexpr int kWidest = (1 << 30) + (1 << 24);
  a.window = window < kWidest ? window : kWidest;
  a.scale = scale;
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.lse = lse;
  a.ws = ws;
  const cudaError_t e = launch_attend(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "dspark_attend");
  return DSPARK_OK;
}

}  // extern "C"
