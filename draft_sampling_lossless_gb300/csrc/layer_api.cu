// C ABI of the target's layers around its attention: argument validation and
// launches (include/dspark.h has the contract).
#include <cudaTypedefs.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "dspark.h"
#include "layer.cuh"

using namespace dspark;

namespace {

static_assert(sizeof(Weights4Desc) <= sizeof(dspark_weights4),
              "dspark_weights4 holds a Weights4Desc");

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
#define REQUIRE_ALIGNED(p, n)                                                             \
  do {                                                                                    \
    REQUIRE(p);                                                                           \
    if (((uintptr_t)(p) & ((n)-1)) != 0)                                                  \
      return fail(DSPARK_ERR_INVALID_ARG, "%s must be %d-byte aligned", #p, n);           \
  } while (0)

constexpr int kMaxN = 1 << 24, kMaxK = 1 << 16, kMaxT = 1 << 24, kMaxD = 1 << 15;

bool shape_ok(int N, int K) { return N >= 1 && N <= kMaxN && K >= 32 && K <= kMaxK && K % 32 == 0; }

// Row strides in elements: multiples of 8 (16 bytes of bf16) of at least a row.
int stride_ok(const char* what, int64_t stride, int64_t row) {
  if (stride < row || stride % 8 != 0 || stride > (1ll << 40))
    return fail(DSPARK_ERR_INVALID_ARG,
                "%s must be a multiple of 8 and at least a row of %lld (got %lld)", what,
                (long long)row, (long long)stride);
  return DSPARK_OK;
}

int load_desc(const char* what, const dspark_weights4* w, Weights4Desc& d) {
  if (w == nullptr) return fail(DSPARK_ERR_INVALID_ARG, "%s is NULL", what);
  memcpy(&d, w, sizeof(d));
  if (d.magic != kWeights4Magic)
    return fail(DSPARK_ERR_INVALID_ARG, "%s was not filled by dspark_weights4_init", what);
  return DSPARK_OK;
}

// Boxes of a tile's codes, 128 rows of 128, each code spread to a byte's place (16 codes in 8
// bytes, 8 bytes apart) and swizzled as the MMA operand that they land in; tiles past the last
// read as zeros.
cudaError_t encode_codes(Weights4Desc& d) {
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
  cuuint64_t dims[3] = {128, 128, (cuuint64_t)((d.N + 127) / 128) * (d.Kp / 128)};
  cuuint64_t strides[2] = {64, kTileBytes};
  cuuint32_t box[3] = {128, 128, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(&d.tm, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, d.store, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// What the two products check alike.
int run_linear4(const char* name, const Weights4Desc& w, const Weights4Desc* up, int act, int T,
                const void* x, int64_t x_stride, void* out, int64_t out_stride, void* ws,
                size_t ws_bytes, void* stream) {
  if (T < 0 || T > kMaxT)
    return fail(DSPARK_ERR_INVALID_ARG, "T out of range (%d; need 0 <= T <= 2^24)", T);
  if ((int64_t)T * w.N > (1ll << 38))
    return fail(DSPARK_ERR_INVALID_ARG, "T * N must be at most 2^38");
  REQUIRE_ALIGNED(ws, 256);
  const size_t need = linear4_workspace_bytes(T, w.K);
  if (ws_bytes < need)
    return fail(DSPARK_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  if (T == 0) return DSPARK_OK;
  REQUIRE_ALIGNED(x, 16);
  REQUIRE_ALIGNED(out, 2);
  int s;
  if ((s = stride_ok("x_stride", x_stride, w.K))) return s;
  if (out_stride < w.N || out_stride > (1ll << 40))
    return fail(DSPARK_ERR_INVALID_ARG, "out_stride must be at least N = %d (got %lld)", w.N,
                (long long)out_stride);
  Linear4Args a;
  a.w = &w;
  a.up = up;
  a.act = act;
  a.T = T;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.x_stride = x_stride;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.out_stride = out_stride;
  a.ws = ws;
  const cudaError_t e = launch_linear4(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, name);
  return DSPARK_OK;
}

}  // namespace

extern "C" {

size_t dspark_weights4_bytes(int N, int K) {
  return shape_ok(N, K) ? weights4_bytes(N, K) : 0;
}

int dspark_weights4_init(dspark_weights4* w, int N, int K, void* store) {
  REQUIRE(w);
  memset(w, 0, sizeof(*w));
  if (!shape_ok(N, K))
    return fail(DSPARK_ERR_INVALID_ARG,
                "need 1 <= N <= 2^24 and K a multiple of 32 in [32, 65536] (N=%d K=%d)", N, K);
  REQUIRE_ALIGNED(store, 256);
  Weights4Desc d;
  memset(&d, 0, sizeof(d));
  d.N = N;
  d.K = K;
  d.Kp = padded_k(K);
  d.store = static_cast<uint8_t*>(store);
  const cudaError_t e = encode_codes(d);
  if (e != cudaSuccess) return cuda_fail(e, "dspark_weights4_init");
  d.magic = kWeights4Magic;
  memcpy(w, &d, sizeof(d));
  return DSPARK_OK;
}

int dspark_weights4_load(const dspark_weights4* w, const uint8_t* codes, const uint8_t* scales,
                         void* stream) {
  Weights4Desc d;
  if (int s = load_desc("w", w, d)) return s;
  REQUIRE_ALIGNED(codes, 16);
  REQUIRE(scales);
  const cudaError_t e = launch_weights4_load(d, codes, scales, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "dspark_weights4_load");
  return DSPARK_OK;
}

int dspark_weights4_quantize(const dspark_weights4* w, const void* src, int dt, int64_t stride,
                             void* stream) {
  Weights4Desc d;
  int s = load_desc("w", w, d);
  if (s) return s;
  if (dt != DSPARK_BF16 && dt != DSPARK_F32)
    return fail(DSPARK_ERR_INVALID_ARG, "dt must be 0 (bf16) or 1 (f32)");
  REQUIRE_ALIGNED(src, 16);
  if ((s = stride_ok("stride", stride, d.K))) return s;
  const cudaError_t e = launch_weights4_quantize(d, src, dt, stride, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "dspark_weights4_quantize");
  return DSPARK_OK;
}

size_t dspark_linear4_workspace_bytes(int T, int K) {
  return T >= 0 && T <= kMaxT && shape_ok(1, K) ? linear4_workspace_bytes(T, K) : 0;
}

int dspark_linear4(const dspark_weights4* w, int T, const void* x, int64_t x_stride, void* out,
                   int64_t out_stride, void* ws, size_t ws_bytes, void* stream) {
  Weights4Desc d;
  if (int s = load_desc("w", w, d)) return s;
  return run_linear4("dspark_linear4", d, nullptr, 0, T, x, x_stride, out, out_stride, ws,
                     ws_bytes, stream);
}

int dspark_gated4(const dspark_weights4* gate, const dspark_weights4* up, int act, int T,
                  const void* x, int64_t x_stride, void* out, int64_t out_stride, void* ws,
                  size_t ws_bytes, void* stream) {
  Weights4Desc g, u;
  int s = load_desc("gate", gate, g);
  if (s || (s = load_desc("up", up, u))) return s;
  if (g.N != u.N || g.K != u.K)
    return fail(DSPARK_ERR_INVALID_ARG, "gate and up differ in shape ([%d, %d] and [%d, %d])", g.N,
                g.K, u.N, u.K);
  if (act != DSPARK_ACT_SILU && act != DSPARK_ACT_GELU)
    return fail(DSPARK_ERR_INVALID_ARG, "act must be 0 (silu) or 1 (gelu)");
  return run_linear4("dspark_gated4", g, &u, act, T, x, x_stride, out, out_stride, ws, ws_bytes,
                     stream);
}

int dspark_norm(int T, int d, int dt, const void* x, int64_t x_stride, const void* y,
                int64_t y_stride, const float* post, const void* gate, int64_t gate_stride,
                float alpha, const float* pre, float eps, void* x_out, int64_t x_out_stride,
                void* h, int64_t h_stride, void* stream) {
  if (T < 0 || T > kMaxT || d < 8 || d > kMaxD || d % 8 != 0)
    return fail(DSPARK_ERR_INVALID_ARG,
                "need 0 <= T <= 2^24 and d a multiple of 8 in [8, 32768] (T=%d d=%d)", T, d);
  if (dt != DSPARK_BF16 && dt != DSPARK_F32)
    return fail(DSPARK_ERR_INVALID_ARG, "dt must be 0 (bf16) or 1 (f32)");
  if (!isfinite(eps) || eps < 0.0f || !isfinite(alpha))
    return fail(DSPARK_ERR_INVALID_ARG, "eps must be finite and >= 0, alpha finite");
  if (T == 0) return DSPARK_OK;
  int s;
  REQUIRE_ALIGNED(x, 16);
  if ((s = stride_ok("x_stride", x_stride, d))) return s;
  if (h == nullptr && x_out == nullptr)
    return fail(DSPARK_ERR_INVALID_ARG, "h and x_out are both NULL");
  if (y != nullptr) {
    REQUIRE_ALIGNED(y, 16);
    if ((s = stride_ok("y_stride", y_stride, d))) return s;
    if (gate != nullptr) {
      REQUIRE_ALIGNED(gate, 16);
      if (gate_stride != 0 && (s = stride_ok("gate_stride", gate_stride, d))) return s;
    }
    if (post != nullptr) REQUIRE_ALIGNED(post, 16);
  } else if (post != nullptr || gate != nullptr || x_out != nullptr) {
    return fail(DSPARK_ERR_INVALID_ARG, "post, gate and x_out need y");
  }
  if (h != nullptr) {
    REQUIRE_ALIGNED(h, 16);
    REQUIRE_ALIGNED(pre, 16);
    if ((s = stride_ok("h_stride", h_stride, d))) return s;
  } else if (pre != nullptr) {
    return fail(DSPARK_ERR_INVALID_ARG, "pre needs h");
  }
  if (x_out != nullptr) {
    REQUIRE_ALIGNED(x_out, 16);
    if ((s = stride_ok("x_out_stride", x_out_stride, d))) return s;
  }
  NormArgs a;
  a.T = T;
  a.d = d;
  a.dt = dt;
  a.alpha = alpha;
  a.eps = eps;
  a.inv_d = 1.f / (float)d;
  a.x = x;
  a.x_stride = x_stride;
  a.y = static_cast<const __nv_bfloat16*>(y);
  a.y_stride = y_stride;
  a.gate = static_cast<const __nv_bfloat16*>(gate);
  a.gate_stride = gate_stride;
  a.post = post;
  a.pre = pre;
  a.x_out = x_out;
  a.x_out_stride = x_out_stride;
  a.h = static_cast<__nv_bfloat16*>(h);
  a.h_stride = h_stride;
  const cudaError_t e = launch_norm(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "dspark_norm");
  return DSPARK_OK;
}

}  // extern "C"
