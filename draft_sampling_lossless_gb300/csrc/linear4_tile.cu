// Products with 4-bit weights on the tensor cores: x W^T, and act(x G^T) * (x U^T).
//
// Block-scaled MMAs (kind mxf8f6f4) take the codes and scales of W as they are stored, so
// nothing is unpacked: A is 128 rows of W, a code in each byte (the TMA load spreads
// them), its scales beside the accumulators in tensor memory.  B is the rows of x.  Its
// e4m3 has 4 significant bits, bf16 has 8: x is two e4m3 terms, exactly,
//
//   x = 2^e (hi + 2^-4 lo),  |hi| <= 448,  e for each row and 32 columns,
//
// but for what lies below 2^-22 of a group's largest (lo ends at 2^-9 of its scale), so
// each step of K runs two MMAs, on hi and on lo, into one accumulator.  That is the rate of
// bf16 MMAs, for a quarter of the weights' bytes and no conversions.  Rows where that is more than
// a few small values among larger ones are found as x is split and computed again from x itself.
//
// A first kernel writes hi, lo and their exponents in tiles that one bulk copy brings in,
// swizzled as the MMA reads them; the second starts under it and already loads weights.  Blocks
// that have one tile only may split x themselves, as long as that keeps up.
//
// What bounds it: with many rows the MMAs (an A of 128 x 32 takes 62 cycles from shared memory,
// so N = 160 to 192 columns run at 90 to 95% of their rate and 64 at half of it); with a few
// the issuing thread, 390 to 500 cycles a step of 128 columns (waits, copies of scales and
// commits 210, an MMA 45) where A's reads take some 300, on as many SMs as there are tiles;
// with a large vocabulary HBM beside the MMAs.  Measured among calls in a graph: 4100 rows gated by 2 x
// 10240 x 2560 237 us, 1.81 PFLOP/s (97% of cuBLAS's measured bf16 rate), tensor pipe 78%
// busy at 2100 rows; 4100 rows by 6144 x 2560 84 us, 1.54 PFLOP/s, 10 of them the first kernel; 64
// rows by 151936 x 2560 47.3 us, 4.8 TB/s; 122 rows by 2560 x 4096 11.0 us, gated by 2 x 10240 x
// 2560 19.4 us (80 tiles on 152 SMs, or 240 in two rounds); one row gated by the same 10.5 us.
#include "linear4.cuh"
#include "sm100.cuh"

namespace dspark {

using namespace sm100;

namespace {

constexpr int kMaxTokens = 192;   // rows of x a tile
constexpr int kOutWarps = 16;     // warps of results, a quarter of them for 32 lanes each
constexpr int kTurns = kOutWarps / 4;
constexpr int kThreads = 64 + kOutWarps * 32;  // one that loads, one that issues MMAs, results
constexpr int kMaxSmem = 232448;
constexpr int kSfCol = 480;       // tensor memory: accumulators below, scales above
constexpr int kMaxSlots = 8;
constexpr int kMaxSplit = 8;
constexpr uint32_t kStatusBytes = 1024;
constexpr uint32_t kWaitNs = 2000000000u;

using Cut = TileCut;

// The tile of `tokens` rows and 128 columns of x: hi, lo, their exponents in blocks of 512
// bytes for 128 MMA columns, as tcgen05.cp takes them (hi's then lo's).
__host__ __device__ constexpr uint32_t exp_blocks(int tokens, int wide) {
  return wide ? (2 * tokens + 127) / 128 : 2 * ((tokens + 127) / 128);
}
__host__ __device__ constexpr uint32_t tile_bytes(int tokens, int wide) {
  return (uint32_t)tokens * 256 + exp_blocks(tokens, wide) * 512;
}

// A workspace: the status word; a byte for 512 columns of a row, whether they lost bits,
// [ceil(Kp / 512)][T rounded up to 8]; tiles of x.
__host__ __device__ constexpr int lossy_stride(int T) { return (T + 7) & ~7; }
__host__ __device__ constexpr size_t lossy_bytes(int T, int Kp) {
  return ((size_t)lossy_stride(T) * ((Kp + 511) / 512) + 255) & ~(size_t)255;
}

// ---------------------------------------------------------------- x in two terms

// The smallest e >= -118 with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ int group_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return max(e, -118);
}
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// The largest finite magnitude of eight values, as bf16 bits (magnitudes order as whole numbers,
// past 0x7f80 a NaN).  What is not finite becomes NaN in v: its row's results are not finite.
__device__ __forceinline__ uint32_t top_of8(uint4 raw, float (&v)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                          __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
  top = max(top & 0xffffu, top >> 16);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
  if (top >= 0x7f80u) {
    top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(v[j]);
      if (a < INFINITY) top = max(top, __float_as_uint(a) >> 16);
      else v[j] = NAN;
    }
  }
  return top;
}
// Their codes of hi and lo for the group's factor f = 2^-e.
__device__ __forceinline__ void codes_of8(const float (&v)[8], float f, uint2& hi, uint2& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = v[2 * j] * f, b = v[2 * j + 1] * f;
    h[j] = to_e4m3x2(a, b);
    const float2 c = from_e4m3x2(h[j]);
    l[j] = to_e4m3x2((a - c.x) * 16.f, (b - c.y) * 16.f);
  }
  hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}
// The two terms hold all 8 bits of values from 2^-6 of the scale up (2^-14 of a group's largest);
// below, bits go.  A group counts as lossy where half of its nonzero values lie there: beside one
// channel far above its neighbours, whose weight may be zero (with the neighbours at 2^-14 of it
// the group's sum is then off by 2^-9 of itself, at 2^-16 by 2^-7).  Rows with such a group are
// computed again by exact_rows below.  In normal and gated activations a value or two of a group
// are that small, beside a channel of 2^10 a few, of 2^12 a fifth: what those lose is below
// 2^-22 of the largest, and most of the others are there at full length.
//
// The bits 7 of four codes of hi that are above 2^-6: no more than the whole values among them,
// so that the counting is left out for nearly all.
__device__ __forceinline__ uint32_t whole_codes(uint32_t hi) {
  return ((hi & 0x7f7f7f7fu) + 0x77777777u) & 0x80808080u;
}
// How many of eight nonzero values are below 2^-6 of exponent e's scale, and in the second byte how
// many are not zero.
__device__ __forceinline__ uint32_t small_of8(uint4 raw, int e) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  const uint32_t add = (0x8000u - ((uint32_t)(e + 121) << 7)) * 0x00010001u;
  uint32_t nonzero = 0, big = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // (no sum of two halves passes 0xffff)
    const uint32_t m = w[j] & 0x7fff7fffu;
    nonzero = nonzero >> 1 | ((m + 0x7fff7fffu) & 0x80008000u);
    big = big >> 1 | ((m + add) & 0x80008000u);
  }
  return (uint32_t)(__popc(nonzero) - __popc(big)) | (uint32_t)__popc(nonzero) << 8;
}
__device__ __forceinline__ bool lossy_group(uint32_t counts) {
  const uint32_t small = counts & 0xffu, nonzero = counts >> 8;
  return small > 0 && 2 * small >= nonzero;
}

// A row's exponents go to the place of its MMA column n: lane n % 32 of tensor memory, column
// n / 32; hi's and lo's (`term` 0 and 1).
__device__ __forceinline__ void put_exps(uint8_t* dst, int tokens, int wide, int r, int term,
                                         uint32_t exps) {
  const int n = term == 0 ? r : wide ? tokens + r : (tokens + 127) / 128 * 128 + r;
  *reinterpret_cast<uint32_t*>(dst + tokens * 256 + (n >> 7) * 512 + (n & 31) * 16 +
                               ((n >> 5) & 3) * 4) = exps - term * 0x04040404u;
}

// Eight values of a row's 128 columns by each of 16 lanes, into row r of the tile at `dst`; e:
// the group's exponent; whether to count its small values.
__device__ __forceinline__ bool split8(uint4 raw, uint8_t* dst, int tokens, int wide, int r,
                                       int& e) {
  const int lane = threadIdx.x & 15;
  float v[8];
  uint32_t top = top_of8(raw, v);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  e = group_exponent(__uint_as_float(top << 16));
  uint2 hi, lo;
  codes_of8(v, __uint_as_float((uint32_t)(127 - e) << 23), hi, lo);
  uint32_t exps = 0;
#pragma unroll
  for (int g = 0; g < 4; ++g)
    exps |= (uint32_t)(__shfl_sync(0xffffffffu, e, (threadIdx.x & 16) + g * 4) + 127) << (8 * g);
  const uint32_t at = r * 128 + (((lane >> 1) ^ (r & 7)) << 4) + (lane & 1) * 8;
  *reinterpret_cast<uint2*>(dst + at) = hi;
  *reinterpret_cast<uint2*>(dst + tokens * 128 + at) = lo;
  if (lane < 2) put_exps(dst, tokens, wide, r, lane, exps);
  return top != 0 && (whole_codes(hi.x) & whole_codes(hi.y)) != 0x80808080u;
}

// A warp a row's four tiles of 128 columns, 16 values a lane.  Rows past T stay as they are:
// they reach only columns of the product that are not stored.
constexpr int kSplitWarps = 8;

__global__ void __launch_bounds__(kSplitWarps * 32, 8)
    split_kernel(const __nv_bfloat16* __restrict__ x, int64_t x_stride, int T, int K, int KB,
                 int tokens, int wide, uint8_t* __restrict__ out, uint8_t* __restrict__ lossy) {
  grid_dependency_wait();
  asm volatile("griddepcontrol.launch_dependents;");
  const int t = blockIdx.x * kSplitWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int kb = blockIdx.y * 4 + (lane >> 3), l8 = lane & 7, col = kb * 128 + l8 * 16;
  if (t >= T) {  // (whole warps)
    if (lane == 0) lossy[(size_t)blockIdx.y * lossy_stride(T) + t] = 0;
    return;
  }
  const int tile = t / tokens, r = t - tile * tokens;
  uint4 raw[2] = {};
  if (col < K) {  // K is a multiple of 32
    const uint4* p = reinterpret_cast<const uint4*>(x + t * x_stride + col);
    raw[0] = __ldg(p);
    raw[1] = __ldg(p + 1);
  }
  float v[2][8];
  uint32_t top = max(top_of8(raw[0], v[0]), top_of8(raw[1], v[1]));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  const int e = group_exponent(__uint_as_float(top << 16));
  const float f = __uint_as_float((uint32_t)(127 - e) << 23);
  uint2 hi[2], lo[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) codes_of8(v[i], f, hi[i], lo[i]);
  uint32_t exps = (uint32_t)(e + 127) << (4 * (l8 & 6));  // of the lane's group, then of four
  exps |= __shfl_xor_sync(0xffffffffu, exps, 2);
  exps |= __shfl_xor_sync(0xffffffffu, exps, 4);
  uint32_t any = 0;
  int whole = __popc(whole_codes(hi[0].x) | whole_codes(hi[0].y) >> 1 | whole_codes(hi[1].x) >> 2 |
                     whole_codes(hi[1].y) >> 3);
  whole += __shfl_xor_sync(0xffffffffu, whole, 1);
  // (with more than 16 whole ones the small ones are fewer than half)
  if (__builtin_expect(__any_sync(0xffffffffu, top != 0 && whole <= 16), 0)) {
    uint32_t counts = 0;
    if (col < K) {  // (read again: kept, the values cost registers)
      const uint4* p = reinterpret_cast<const uint4*>(x + t * x_stride + col);
      counts = small_of8(__ldg(p), e) + small_of8(__ldg(p + 1), e);
    }
    counts += __shfl_xor_sync(0xffffffffu, counts, 1);
    any = __any_sync(0xffffffffu, lossy_group(counts));
  }
  if (lane == 0) lossy[(size_t)blockIdx.y * lossy_stride(T) + t] = any ? 1 : 0;
  if (kb >= KB) return;
  uint8_t* dst = out + ((size_t)tile * KB + kb) * tile_bytes(tokens, wide);
  const uint32_t at = r * 128 + ((l8 ^ (r & 7)) << 4);
  *reinterpret_cast<uint4*>(dst + at) = make_uint4(hi[0].x, hi[0].y, hi[1].x, hi[1].y);
  *reinterpret_cast<uint4*>(dst + tokens * 128 + at) =
      make_uint4(lo[0].x, lo[0].y, lo[1].x, lo[1].y);
  if (l8 < 2) put_exps(dst, tokens, wide, r, l8, exps);
}

// ---------------------------------------------------------------- the product

struct Params {
  const uint8_t *w, *u;    // the matrices' tiles
  const uint8_t* xq;       // tiles of x, or null: the blocks make their own
  const uint8_t* lossy;    // with xq: which rows lost bits
  const __nv_bfloat16* x;
  int64_t x_stride;
  int N, T, K, KB, row_blocks, tokens, wide, feature_tiles, tiles, split, stages, slots, act;
  bool vector;  // rows of out are 16-byte aligned
  __nv_bfloat16* out;
  int64_t out_stride;
  uint32_t* status;
};

struct Small {  // at the end of shared memory
  uint64_t full[12], empty[12], acc_full[kMaxSlots], acc_empty[kMaxSlots], drain;
  uint32_t lossy[kMaxSplit][kMaxTokens / 32];  // rows that the blocks split and that lost bits
  int again;  // there are rows for exact_rows
  uint32_t tmem;
  int abort_flag, issued;
};

// kind mxf8f6f4: A e2m1 (5), B e4m3 (0), scales powers of two, both K-major, M = 128, the
// first byte of the scales' columns (byte j: j << 4 for B's, j << 29 for A's).
__device__ __forceinline__ uint32_t idesc_mx(int N) {
  return (5u << 7) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (8u << 24);
}
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t sa, uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}
// 512 bytes (32 rows of 16) over the 32 lanes and 4 columns at `taddr`, in each quarter of the
// lanes; in order with this thread's MMAs.
__device__ __forceinline__ uint64_t desc_scales(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(128 >> 4) << 16;
  d |= static_cast<uint64_t>(128 >> 4) << 32;  // from 8 rows to the next 8
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t d) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d)
               : "memory");
}
// Untiled copy, 16-byte aligned, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t addr, int rank, const float (&v)[4]) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.v4.f32 [a], {%2, %3, %4, %5};\n\t}" ::"r"(addr),
      "r"(rank), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
      : "memory");
}

// What the kernel before wrote of rows t .. t + 7 and 512 columns.
__device__ __forceinline__ uint64_t lossy_bytes8(const Params& p, int i, int t) {
  return *reinterpret_cast<const uint64_t*>(p.lossy + (size_t)i * lossy_stride(p.T) + t);
}
// Which of these rows lost bits.
__device__ __forceinline__ uint32_t lossy_rows(const Params& p, int t) {
  uint64_t any = 0;
  for (int i = threadIdx.x & 31; i < (p.KB + 3) >> 2; i += 32) any |= lossy_bytes8(p, i, t);
  const uint32_t lo = __reduce_or_sync(0xffffffffu, (uint32_t)any);
  const uint32_t hi = __reduce_or_sync(0xffffffffu, (uint32_t)(any >> 32));
  return (lo * 0x10204080u >> 28) | (hi * 0x10204080u >> 28) << 4;  // (bytes of 0 or 1 to bits)
}
__device__ __forceinline__ void store_cluster(uint32_t addr, int rank, uint32_t v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.u32 [a], %2;\n\t}" ::"r"(addr),
      "r"(rank), "r"(v)
      : "memory");
}

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_wait_or_abort(bar, parity, abort_flag, kWaitNs);
}

// Eight rows of x of an accumulator at `taddr`, hi's and lo's sums added.
__device__ __forceinline__ void load_sums(uint32_t taddr, const Params& p, float (&v)[8]) {
  uint32_t a[8], b[8];
  tmem_ld_32x32b_x8(taddr, a);
  if (p.wide) {
    tmem_ld_32x32b_x8(taddr + p.tokens, b);
    tmem_wait_ld_regs(a, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(a[i]) + __uint_as_float(b[i]);
  } else {
    tmem_wait_ld_regs(a);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(a[i]);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// A warp's 8 rows of x by 32 features, a feature a lane (v[0..3]: pairs of rows in bf16), turned
// in three exchanges so that a lane has 8 neighbouring features of a row: one 16-byte store
// for 8 of two bytes.  `out`: the first row and feature.
__device__ __forceinline__ void store_rows(const uint32_t* v, const Params& p,
                                           __nv_bfloat16* out, int rows, int features) {
  const uint32_t lane = threadIdx.x & 31;
  const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
  uint32_t x[4];  // rows 2 j and 2 j + 1, then row 2 j + b0 of two features
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = v[j];
  const uint32_t give = b0 ? 0x5410u : 0x7632u;
  const uint32_t first = b0 ? 0x3254u : 0x5410u, second = b0 ? 0x3276u : 0x7610u;
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const uint32_t r = __shfl_xor_sync(0xffffffffu, __byte_perm(x[j], x[j + 1], give), 1);
    x[j] = __byte_perm(x[j], r, first);
    x[j + 1] = __byte_perm(x[j + 1], r, second);
  }
  uint2 y[2];  // row 4 i + 2 b1 + b0 of four features
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t keep = b1 ? x[2 * i + 1] : x[2 * i];
    const uint32_t r = __shfl_xor_sync(0xffffffffu, b1 ? x[2 * i] : x[2 * i + 1], 2);
    y[i] = b1 ? make_uint2(r, keep) : make_uint2(keep, r);
  }
  const uint2 keep = b2 ? y[1] : y[0], send = b2 ? y[0] : y[1];
  uint2 r;
  r.x = __shfl_xor_sync(0xffffffffu, send.x, 4);
  r.y = __shfl_xor_sync(0xffffffffu, send.y, 4);
  const uint4 z = b2 ? make_uint4(r.x, r.y, keep.x, keep.y) : make_uint4(keep.x, keep.y, r.x, r.y);
  const int row = lane & 7, f = lane & ~7u;
  if (row >= rows || f >= features) return;
  __nv_bfloat16* dst = out + row * p.out_stride + f;
  if (p.vector && f + 8 <= features) {
    *reinterpret_cast<uint4*>(dst) = z;
  } else {
    const uint32_t w[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (f + i < features)
        reinterpret_cast<uint16_t*>(dst)[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}

// The rows of a tile (of r0 .. r0 + n - 1) that lost bits, computed again from x itself: bf16 MMAs
// of 16 features by 8 rows, the codes as they are loaded, as in linear4_rows.cu.  A warp has 16 of
// the block's features and all of K (half of it with one row tile).  This runs after everything
// else in the block: calls without such rows take 0 to 0.4 us more than without all of this (122
// rows by 2560 x 4096 10.98 us for 10.7, 4100 by 6144 x 2560 83.7 for 83.1).  A few rows take some
// 16 us, all of 4100 some twenty times as long as the rest (1.6 ms for 84 us).
template <int MATS, bool GATED>
__device__ __forceinline__ void exact_rows(const Params& p, Small* ms, uint8_t* smem, int tile,
                                           int r0, int n) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  float4(*red)[32] = reinterpret_cast<float4(*)[32]>(smem);  // [16 warps][32]
  int* count = reinterpret_cast<int*>(smem + 8192);
  int* list = count + 1;
  const int tt = tile / p.feature_tiles, ft = tile - tt * p.feature_tiles;
  const int t0 = tt * p.tokens, end = min(r0 + n, p.T - t0);
  __syncthreads();  // (the last tile's results have been read)
  if (tid == 0) *count = 0;
  __syncthreads();
  for (int c = (r0 & ~7) + warp * 8; c < end; c += kThreads / 4) {
    uint32_t mask = 0;
    if (p.xq) {
      mask = lossy_rows(p, t0 + c);
    } else {
      for (int i = 0; i < p.split; ++i) mask |= ms->lossy[i][c >> 5] >> (c & 31);
    }
    const int r = c + lane;
    if (lane < 8 && (mask >> lane & 1) && r >= r0 && r < end) list[atomicAdd(count, 1)] = r;
  }
  __syncthreads();
  const int rows = *count;
  for (int b = 0; b < rows; b += 8) {
    if (warp < 16) {
      const int m = MATS == 2 ? warp >> 3 : 0, half = MATS == 2 ? 0 : warp >> 3;
      const int f = (warp & 7) * 16 + g;
      const int k0 = MATS == 2 ? 0 : p.KB * half / 2, k1 = MATS == 2 || half ? p.KB : p.KB / 2;
      const int block = min(GATED || MATS == 1 ? ft : ft * 2 + m, p.row_blocks - 1);
      const uint8_t* w = (GATED && m ? p.u : p.w) + (size_t)block * p.KB * kTileBytes;
      const int row = t0 + list[min(b + g, rows - 1)];
      const __nv_bfloat16* x = p.x + (int64_t)row * p.x_stride + t * 32;
      float d[4] = {};
#pragma unroll 2
      for (int k = k0; k < k1; ++k) {
        const uint8_t* at = w + (size_t)k * kTileBytes;
        const uint4 c0 = __ldg(reinterpret_cast<const uint4*>(at + code_in_tile(f, t)));
        const uint4 c1 = __ldg(reinterpret_cast<const uint4*>(at + code_in_tile(f + 8, t)));
        const uint32_t s0 = __ldg(at + scale_in_tile(f, t));
        const uint32_t s1 = __ldg(at + scale_in_tile(f + 8, t));
        // a group's power of two, times 2^126 for the codes' bits, in two factors
        const uint32_t f0 = min(s0 + 126u, 254u) * 0x00800080u;
        const uint32_t f1 = min(s1 + 126u, 254u) * 0x00800080u;
        const uint32_t h0 = (max(s0, 128u) - 1u) * 0x00800080u;
        const uint32_t h1 = (max(s1, 128u) - 1u) * 0x00800080u;
        const bool in = k * 128 + t * 32 < p.K;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (in) v = __ldg(reinterpret_cast<const uint4*>(x + k * 128) + i);
          const uint32_t w0 = i == 0 ? c0.x : i == 1 ? c0.y : i == 2 ? c0.z : c0.w;
          const uint32_t w1 = i == 0 ? c1.x : i == 1 ? c1.y : i == 2 ? c1.z : c1.w;
          auto value = [](uint32_t bits, uint32_t f, uint32_t h) {
            return mul_bf16x2(mul_bf16x2(bits, f), h);
          };
          const uint32_t lo[4] = {value(pair_bits<0>(w0), f0, h0), value(pair_bits<0>(w1), f1, h1),
                                  value(pair_bits<1>(w0), f0, h0), value(pair_bits<1>(w1), f1, h1)};
          const uint32_t hi[4] = {value(pair_bits<2>(w0), f0, h0), value(pair_bits<2>(w1), f1, h1),
                                  value(pair_bits<3>(w0), f0, h0), value(pair_bits<3>(w1), f1, h1)};
          mma_16816(d, lo, __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632));
          mma_16816(d, hi, __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        }
      }
      red[warp][lane] = make_float4(d[0], d[1], d[2], d[3]);
    }
    __syncthreads();
    for (int i = tid; i < (GATED ? 1 : MATS) * 1024; i += kThreads) {
      const int c = i & 127, j = i >> 7 & 7, m = i >> 10;  // feature, row, row tile
      const int l = (c & 7) * 4 + (j >> 1), e = (c >> 3 & 1) * 2 + (j & 1);
      float o = reinterpret_cast<const float*>(&red[m * 8 + (c >> 4)][l])[e];
      if (MATS == 1 || GATED) {
        const float o1 = reinterpret_cast<const float*>(&red[8 + (c >> 4)][l])[e];
        o = GATED ? activation(p.act, o) * o1 : o + o1;
      }
      const int feature = (GATED ? ft : ft * MATS + m) * 128 + c;
      if (b + j < rows && feature < p.N)
        p.out[(int64_t)(t0 + list[b + j]) * p.out_stride + feature] = __float2bfloat16(o);
    }
    __syncthreads();
  }
}

// MATS row tiles of 128 share a block's x: two of one matrix, or (GATED) one of each.
template <int MATS, bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_u,
                const Params p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t x_bytes = tile_bytes(p.tokens, p.wide);
  // a stage: codes (16 KB a matrix), x's tile, the codes' scales (512 bytes a matrix)
  const uint32_t stage_bytes = (MATS * (16384 + 512) + x_bytes + 1023) & ~1023u;
  const uint32_t s0 = smem_u32(smem);
  Small* ms = reinterpret_cast<Small*>(smem + (size_t)p.stages * stage_bytes);
  const uint32_t b_full = smem_u32(ms->full), b_empty = smem_u32(ms->empty);
  const uint32_t b_accFull = smem_u32(ms->acc_full), b_accEmpty = smem_u32(ms->acc_empty);
  const uint32_t b_drain = smem_u32(&ms->drain);
  volatile int* s_abort = &ms->abort_flag;

  if (tid >= 64 && tid < 64 + kMaxSplit * (kMaxTokens / 32)) ms->lossy[0][tid - 64] = 0;
  if (warp == 1) {
    tmem_alloc(smem_u32(&ms->tmem), 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    const int t0 = blockIdx.x / p.split / p.feature_tiles * p.tokens;
    const int quads = (min(p.tokens, p.T - t0) + 3) >> 2;  // arrivals of who splits x
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(b_full + 8 * i, p.xq ? 1 : 1 + quads);
      mbar_init(b_empty + 8 * i, 1);
    }
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(b_accFull + 8 * i, 1);
      mbar_init(b_accEmpty + 8 * i, kOutWarps);
    }
    mbar_init(b_drain, 1);
    fence_mbar_init();
    ms->abort_flag = 0;
    ms->issued = 0;
    ms->again = 0;
    tma_prefetch(&tm_w);
    if (GATED) tma_prefetch(&tm_u);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem;

  // Tiles: `split` blocks (a cluster) share one, each a range of K; or a block takes every
  // gridDim.x-th.
  const int rank = p.split > 1 ? (int)(blockIdx.x % p.split) : 0;
  const int first = blockIdx.x / p.split, step = gridDim.x / p.split;
  const int k0 = (int)((int64_t)p.KB * rank / p.split);
  const int k1 = (int)((int64_t)p.KB * (rank + 1) / p.split);

  // Places in the ring of stages and phases are counted, not divided out: a division by a
  // number that only the launch knows costs the one issuing thread 200 cycles a step.
  if (warp == 0) {
    if (elect_one()) {
      const uint32_t tx = MATS * (8192 + 512) + (p.xq ? x_bytes : 0);
      const int tt_step = step / p.feature_tiles, ft_step = step - tt_step * p.feature_tiles;
      int tt = first / p.feature_tiles, ft = first - tt * p.feature_tiles;
      auto load_w = [&](uint32_t bar, uint32_t dst, int kb) {
        mbar_arrive_expect_tx(bar, tx);
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          const int row = GATED || MATS == 1 ? ft : ft * 2 + m;  // in blocks of 128
          tma_load_3d(dst + m * 16384, GATED && m ? &tm_u : &tm_w, bar, 0, 0, row * p.KB + kb);
          // (the second tile of an odd number reads zeros, with the last tile's scales)
          const int in = GATED || MATS == 1 ? row : min(row, p.row_blocks - 1);
          bulk_load(dst + MATS * 16384 + x_bytes + m * 512,
                    (GATED && m ? p.u : p.w) + ((size_t)in * p.KB + kb) * kTileBytes + kTileCodes,
                    512, bar);
        }
      };
      auto load_x = [&](uint32_t bar, uint32_t dst, int kb) {
        if (p.xq)
          bulk_load(dst + MATS * 16384, p.xq + ((size_t)tt * p.KB + kb) * x_bytes, x_bytes, bar);
      };
      // the first stages' weights, before the kernel that writes x's tiles has ended (without
      // that, the kernel before this one may have written the weights)
      if (!p.xq) grid_dependency_wait();
      const int here = min(p.stages, k1 - k0);
      for (int i = 0; i < here; ++i) load_w(b_full + 8 * i, s0 + i * stage_bytes, k0 + i);
      grid_dependency_wait();
      for (int i = 0; i < here; ++i) load_x(b_full + 8 * i, s0 + i * stage_bytes, k0 + i);
      int issued = here, s = here, kb = k0 + here;
      uint32_t free_parity = 1;  // of the ring's round: the first finds every stage free
      bool ok = true;
      for (int tile = first; ok;) {
        for (; kb < k1; ++kb, ++s, ++issued) {
          if (s == p.stages) {
            s = 0;
            free_parity ^= 1;
          }
          ok = wait_bar(b_empty + 8 * s, free_parity, s_abort);
          if (!ok) break;
          load_w(b_full + 8 * s, s0 + s * stage_bytes, kb);
          load_x(b_full + 8 * s, s0 + s * stage_bytes, kb);
        }
        tile += step;
        if (tile >= p.tiles) break;
        kb = k0;
        tt += tt_step;
        ft += ft_step;
        if (ft >= p.feature_tiles) {
          ft -= p.feature_tiles;
          ++tt;
        }
      }
      ms->issued = issued;
    }
  } else if (warp == 1) {
    grid_dependency_wait();  // so that the waits' limits do not count what ran before
    if (elect_one()) {
      const uint32_t nb = exp_blocks(p.tokens, p.wide), acc_cols = p.tokens << p.wide;
      const uint32_t id0 = idesc_mx(acc_cols);
      const uint32_t stage_desc = stage_bytes >> 4;
      const uint64_t d_w0 = desc_kmajor_sw128(s0);
      const uint64_t d_x0 = d_w0 + MATS * (16384 >> 4);
      const uint64_t d_e0 = desc_scales(s0 + MATS * 16384 + p.tokens * 256);
      const uint64_t d_s0 = desc_scales(s0 + MATS * 16384 + x_bytes);
      const uint32_t lo_off = p.tokens * 128 >> 4;
      // Accumulators are a ring of `slots`, MATS of them a tile: three slots for two matrices let
      // the next tile start when the first matrix's sums have left.
      int s = 0, slot = 0;
      uint32_t full_parity = 0, acc_parity = 1, at = 0;
      bool ok = true;
      for (int tile = first; tile < p.tiles && ok; tile += step) {
        uint32_t acc[MATS], b_done[MATS];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          ok = ok && wait_bar(b_accEmpty + 8 * slot, acc_parity, s_abort);
          acc[m] = tmem + slot * acc_cols;
          b_done[m] = b_accFull + 8 * slot;
          if (++slot == p.slots) {
            slot = 0;
            acc_parity ^= 1;
          }
        }
        tc_fence_after();
        uint32_t add = 0;
        for (int kb = k0; kb < k1 && ok; ++kb) {
          ok = wait_bar(b_full + 8 * s, full_parity, s_abort);
          if (!ok) break;
          tc_fence_after();
          // the scales' columns: W (4 a tile), hi's, lo's (copies and MMAs run in order)
          const uint32_t t_w = tmem + kSfCol, t_x = t_w + 4 * MATS;
#pragma unroll
          for (int m = 0; m < MATS; ++m) scales_to_tmem(t_w + 4 * m, d_s0 + at + 32 * m);
          scales_to_tmem(t_x, d_e0 + at);
          if (nb > 1) scales_to_tmem(t_x + 4, d_e0 + at + 32);
          if (nb > 2) {
            scales_to_tmem(t_x + 8, d_e0 + at + 64);
            scales_to_tmem(t_x + 12, d_e0 + at + 96);
          }
          if (p.wide) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
              for (int m = 0; m < MATS; ++m)
                mma_mx(acc[m], d_w0 + at + m * (16384 >> 4) + 2 * j, d_x0 + at + 2 * j,
                       id0 + j * ((1u << 4) + (1u << 29)), t_w + 4 * m, t_x, j > 0 ? 1 : add);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
              for (int m = 0; m < MATS; ++m) {
                const uint32_t id = id0 + j * ((1u << 4) + (1u << 29));
                const uint64_t d_a = d_w0 + at + m * (16384 >> 4) + 2 * j;
                const uint64_t d_b = d_x0 + at + 2 * j;
                mma_mx(acc[m], d_a, d_b, id, t_w + 4 * m, t_x, j > 0 ? 1 : add);
                mma_mx(acc[m], d_a, d_b + lo_off, id, t_w + 4 * m, t_x + 2 * nb, 1);
              }
            }
          }
          mma_commit(b_empty + 8 * s);
          add = 1;
          at += stage_desc;
          if (++s == p.stages) {
            s = 0;
            at = 0;
            full_parity ^= 1;
          }
        }
#pragma unroll
        for (int m = 0; m < MATS; ++m) mma_commit(b_done[m]);
      }
      if (*s_abort) {  // what was issued ends before tensor memory goes
        mma_commit(b_drain);
        mbar_wait(b_drain, 0);
      }
    }
  } else {
    // ------------------------------------------------------------ results
    // Each of the warps that share a quarter of the lanes takes 8 rows of x in turn.
    grid_dependency_wait();
    const int quad = warp & 3, turn = (warp - 2) >> 2;
    const uint32_t acc_cols = p.tokens << p.wide;
    const uint32_t t_lane = static_cast<uint32_t>(quad * 32) << 16;
    int slot = 0;
    uint32_t acc_parity = 0;
    bool ok = true;
    if (!p.xq) {
      // x's tiles first.  A task is four rows of 128 columns, 16 lanes a row; it takes a warp some
      // 1000 cycles from end to end, so the warps take tasks in turn, several tiles at a time.
      const int t0 = first / p.feature_tiles * p.tokens, rows = min(p.tokens, p.T - t0);
      const int quads = (rows + 3) >> 2, l16 = lane & 15;
      // (No more warps than tasks of a ring of stages: then the tile one round before a warp's
      // next has been waited for, and a phase's parity tells the two rounds apart.)
      const int takers = min(kOutWarps, p.stages * quads);
      const int kb_step = takers / quads, q_step = takers - kb_step * quads;
      int kb = warp - 2 < takers ? k0 + (warp - 2) / quads : k1, q = (warp - 2) % quads;
      const __nv_bfloat16* x = p.x + (int64_t)t0 * p.x_stride + l16 * 8;
      auto fetch = [&](uint4 (&v)[2], int kb, int q) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = q * 4 + i * 2 + (lane >> 4);
          v[i] = make_uint4(0, 0, 0, 0);
          if (kb < k1 && r < rows && kb * 128 + l16 * 8 < p.K)
            v[i] = __ldg(reinterpret_cast<const uint4*>(x + (int64_t)r * p.x_stride + kb * 128));
        }
      };
      uint4 next[2];
      fetch(next, kb, q);
      int s = kb - k0;  // its place in the ring of stages
      uint32_t free_parity = 1;
      while (kb < k1) {
        for (; s >= p.stages; s -= p.stages) free_parity ^= 1;
        const uint4 now[2] = {next[0], next[1]};
        const int q_now = q, s_now = s;
        kb += kb_step;
        s += kb_step;
        q += q_step;
        if (q >= quads) {
          q -= quads;
          ++kb;
          ++s;
        }
        fetch(next, kb, q);
        ok = wait_bar(b_empty + 8 * s_now, free_parity, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* dst = smem + (size_t)s_now * stage_bytes + MATS * 16384;
        bool small = false;
        int e[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)  // (the tile has a multiple of 16 rows)
          small |= split8(now[i], dst, p.tokens, p.wide, q_now * 4 + i * 2 + (lane >> 4), e[i]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_full + 8 * s_now);
        if (__any_sync(0xffffffffu, small)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = q_now * 4 + i * 2 + (lane >> 4);
            uint32_t counts = small_of8(now[i], e[i]);
            counts += __shfl_xor_sync(0xffffffffu, counts, 1);
            counts += __shfl_xor_sync(0xffffffffu, counts, 2);
            if (lossy_group(counts)) {
              atomicOr(&ms->lossy[rank][r >> 5], 1u << (r & 31));
              ms->again = 1;
            }
          }
        }
      }
    }
    auto wait_slot = [&]() {
      ok = wait_bar(b_accFull + 8 * slot, acc_parity, s_abort);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      return tmem + t_lane + slot * acc_cols;
    };
    auto free_slot = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_accEmpty + 8 * slot);
      if (++slot == p.slots) {
        slot = 0;
        acc_parity ^= 1;
      }
    };
    for (int tile = first; tile < p.tiles; tile += step) {
      const int tt = tile / p.feature_tiles, ft = tile - tt * p.feature_tiles;
      const int t0 = tt * p.tokens, rows = min(p.tokens, p.T - t0);
      const int f0 = ft * (GATED ? 128 : 128 * MATS) + quad * 32;
      if (p.xq) {  // rows that lost bits?  (512 columns and 8 rows a lane)
        uint64_t lossy = 0;
        for (int c = ((lane >> 3) * kTurns + turn) * 8; c < rows; c += 4 * kTurns * 8)
          for (int i = lane & 7; i < (p.KB + 3) >> 2; i += 8) lossy |= lossy_bytes8(p, i, t0 + c);
        if (lossy != 0) ms->again = 1;
      }
      // The sums leave tensor memory before the activation and the stores (which go out at some 2
      // TB/s where all blocks store at once): the first matrix's in fp32 where the second
      // belongs to it, else rounded.
      constexpr int kRounds = (MATS == 2 ? 160 : 192) / (8 * kTurns);
      uint32_t v[kRounds][GATED ? 8 : 4 * MATS];
#pragma unroll
      for (int m = 0; m < (GATED ? 1 : MATS); ++m) {
        const uint32_t acc = wait_slot();
        if (!ok || p.split > 1) break;
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
          const int c = (i * kTurns + turn) * 8;
          if (c < rows) {
            float a[8];
            load_sums(acc + c, p, a);
#pragma unroll
            for (int j = 0; j < (GATED ? 8 : 4); ++j)
              v[i][4 * m + j] = GATED ? __float_as_uint(a[j]) : pack_bf16(a[2 * j & 7], a[2 * j + 1 & 7]);
          }
        }
        free_slot();
      }
      if (!ok || p.split > 1) break;
      uint32_t acc = 0;
      if (GATED) {
        acc = wait_slot();
        if (!ok) break;
      }
      __nv_bfloat16* out = p.out + (int64_t)(t0 + turn * 8) * p.out_stride + f0;
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int c = (i * kTurns + turn) * 8;
        if (c < rows) {
          if (GATED) {
            float b[8];
            load_sums(acc + c, p, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] *= activation(p.act, __uint_as_float(v[i][j]));
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = pack_bf16(b[2 * j], b[2 * j + 1]);
            store_rows(o, p, out, rows - c, p.N - f0);
          } else {
#pragma unroll
            for (int m = 0; m < MATS; ++m)
              store_rows(&v[i][4 * m], p, out + m * 128, rows - c, p.N - f0 - m * 128);
          }
        }
        out += (int64_t)kTurns * 8 * p.out_stride;
      }
      if (GATED) free_slot();
    }
  }

  if (p.split > 1) {
    // Each block of the cluster sums some columns (rows of x) of the tile over all of them, in
    // the order of their ranges of K.  The partial sums go to their block's shared memory,
    // where the stages were: no MMA of the cluster reads them any more.
    __syncthreads();
    __syncwarp();
    cluster_sync_all();
    const int cols = p.tokens / p.split;  // a multiple of 4
    float4* part = reinterpret_cast<float4*>(smem);  // [split][MATS][cols / 4][128]
    constexpr int kWords = kMaxTokens / 32;
    if (!p.xq && tid < p.split * kWords) {  // the rows that lost bits in this block's range, to all
      const uint32_t mask = ms->lossy[rank][tid % kWords];
      if (mask != 0) {
        store_cluster(smem_u32(&ms->lossy[rank][tid % kWords]), tid / kWords, mask);
        store_cluster(smem_u32(&ms->again), tid / kWords, 1u);
      }
    }
    if (warp >= 2) {
      tc_fence_after();
      const int quad = warp & 3, turn = (warp - 2) >> 2, f = quad * 32 + lane;
      const uint32_t acc_cols = p.tokens << p.wide;
#pragma unroll 1
      for (int m = 0; m < MATS; ++m) {
        const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + m * acc_cols;
#pragma unroll 1
        for (int c = turn * 8; c < p.tokens; c += kTurns * 8) {
          float a[8];
          load_sums(acc + c, p, a);
          int to = c / cols, at = (c - to * cols) >> 2;
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            const float v[4] = {a[i], a[i + 1], a[i + 2], a[i + 3]};
            store_cluster(smem_u32(part + ((rank * MATS + m) * (cols >> 2) + at) * 128 + f), to, v);
            if (++at == cols >> 2) at = 0, ++to;
          }
        }
      }
      tc_fence_before();
    }
    __syncthreads();
    __syncwarp();
    cluster_sync_all();
    const int tt = first / p.feature_tiles, ft = first - tt * p.feature_tiles;
    const int t0 = tt * p.tokens + rank * cols;
    for (int i = tid; i < cols * 32; i += kThreads) {  // four rows of x, one feature
      const int c = i >> 7, f = i & 127;
      float4 v[MATS];
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        v[m] = part[(m * (cols >> 2) + c) * 128 + f];
        for (int r = 1; r < p.split; ++r) {
          const float4 x = part[((r * MATS + m) * (cols >> 2) + c) * 128 + f];
          v[m].x += x.x;
          v[m].y += x.y;
          v[m].z += x.z;
          v[m].w += x.w;
        }
      }
#pragma unroll
      for (int m = 0; m < (GATED ? 1 : MATS); ++m) {
        const int n = ft * (GATED ? 128 : 128 * MATS) + m * 128 + f;
        if (n >= p.N) continue;
        float o[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
        if (GATED) {
          const float4 u = v[MATS - 1];
          o[0] = activation(p.act, o[0]) * u.x;
          o[1] = activation(p.act, o[1]) * u.y;
          o[2] = activation(p.act, o[2]) * u.z;
          o[3] = activation(p.act, o[3]) * u.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (t0 + c * 4 + j < p.T)
            p.out[(int64_t)(t0 + c * 4 + j) * p.out_stride + n] = __float2bfloat16(o[j]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (__builtin_expect(ms->again && !*s_abort, 0)) {
    const int per = p.tokens / p.split;
    for (int tile = first; tile < p.tiles; tile += step)
      exact_rows<MATS, GATED>(p, ms, smem, tile, rank * per, per);
  }
  if (tid == 0 && *s_abort) {
    set_flag(p.status, kFlagWaitTimeout);
    // the copies in flight land before the block's shared memory goes
    const int n = ms->issued;
    // (a wait that runs out, where x's part never came, has been long enough for all of them)
    for (int i = max(0, n - p.stages); i < n; ++i)
      if (!mbar_wait(b_full + 8 * (i % p.stages), (i / p.stages) & 1)) break;
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr uint32_t stage_bytes_of(const Cut& c) {
  return (c.mats * (16384 + 512) + tile_bytes(c.tokens, c.wide) + 1023) & ~1023u;
}
int stages_of(const Cut& c) {
  const int n = (int)((kMaxSmem - 1024 - sizeof(Small)) / stage_bytes_of(c));
  return n < 12 ? n : 12;
}
int slots_of(const Cut& c) {
  const int n = kSfCol / (c.tokens << c.wide);
  return n < kMaxSlots ? n : kMaxSlots;
}

const void* kernel_of(bool gated, int mats) {
  return gated ? (const void*)tile_kernel<2, true>
               : mats == 2 ? (const void*)tile_kernel<2, false> : (const void*)tile_kernel<1, false>;
}

// Cycles of a step of 128 columns.  An MMA of 128 x N x 32 was measured to take 70 (N = 96; A's
// 4 KB from shared memory), 76 (128), 80 (144), 86 (160), 101 (192); the issuing thread takes 45
// an MMA and 210 a step; a stage's bytes come at some 80 a cycle.
int64_t step_cycles(const Cut& c) {
  const int n = c.tokens << c.wide, by_n = n / 2 + 5, by_a = 58 + n / 8;
  const int count = (c.wide ? 4 : 8) * c.mats;
  const int64_t mma = count * (by_n > by_a ? by_n : by_a) + 20;
  const int64_t fill = (8704 * c.mats + (int64_t)tile_bytes(c.tokens, c.wide)) / 80;
  const int64_t issue = 210 + 45 * count;
  return mma > fill ? (mma > issue ? mma : issue) : (fill > issue ? fill : issue);
}

// The cut with the least time of the busiest block, in cycles.  Between two tiles the MMAs
// pause, the longer the fewer accumulators there are; blocks that share a tile exchange sums in
// some 3000 to 6000; a row of x that a block splits takes it 43 a step, a kernel before it 3000, most of
// that the host's (one token by 10240 x 2560 gated: 10.3 us own, 10.6 us with a kernel before;
// 16 rows 11.7 and 10.7 us; 10 us of the host's time instead of 6).
Cut choose(int N, int T, int KB, bool gated) {
  const int sms = sm_count(), blocks = (N + 127) / 128;
  Cut best = {gated ? 2 : 1, 16, 1, 1, false, 0};
  int64_t least = INT64_MAX;
  Cut c;
  for (c.mats = gated ? 2 : 1; c.mats <= 2; ++c.mats)
    for (c.wide = 0; c.wide < 2; ++c.wide)
      for (c.tokens = 16; c.tokens <= (c.wide ? kMaxTokens / 2 : kMaxTokens); c.tokens += 16) {
        if (stages_of(c) < 3 || c.tokens > (c.mats == 2 ? 160 : 192)) break;
        if (c.tokens - 16 >= T) break;
        const int64_t ft = gated ? blocks : (blocks + c.mats - 1) / c.mats;
        const int64_t tiles = ft * ((T + c.tokens - 1) / c.tokens);
        const int64_t step = step_cycles(c);
        const int64_t split_x = 43 * (int64_t)(c.tokens < T ? c.tokens : T);
        const int slots = slots_of(c);
        const int64_t pause = slots >= 2 * c.mats ? 350 : slots > c.mats ? 1500 : gated ? 4000 : 2000;
        const int64_t out = 500 + (gated ? 40 : 24 * c.mats) * c.tokens;
        for (c.split = 1; c.split <= kMaxSplit; c.split *= 2) {
          if (c.split > 1 &&
              (tiles * c.split > sms || KB < 2 * c.split || c.tokens % (4 * c.split) != 0))
            break;
          const int64_t waves = c.split > 1 ? 1 : (tiles + sms - 1) / sms;
          const int64_t steps = (KB + c.split - 1) / c.split;
          for (int own = 0; own < 2; ++own) {
            c.own = own;
            if (own && waves > 1) break;
            const int64_t time = waves * (steps * (own && split_x > step ? split_x : step) + pause) +
                                 (c.split > 1 ? 1500 + 600 * c.split + 14 * c.mats * c.tokens : out) +
                                 (own ? 0 : 3000);
            if (time >= least) continue;
            // (fewer clusters fit than blocks: those of a GPC)
            if (c.split > 1 && tiles > resident_clusters(kernel_of(gated, c.mats), kThreads,
                                                         kMaxSmem, c.split))
              continue;
            least = time;
            best = c;
          }
        }
      }
  best.cycles = least;
  return best;
}

template <int MATS, bool GATED>
cudaError_t launch(const Linear4Args& a, const Cut& cut, cudaStream_t st) {
  auto kernel = tile_kernel<MATS, GATED>;
  Params p;
  p.w = a.w->store;
  p.u = a.up ? a.up->store : nullptr;
  p.lossy = static_cast<const uint8_t*>(a.ws) + kStatusBytes;
  p.xq = cut.own ? nullptr : p.lossy + lossy_bytes(a.T, a.w->Kp);
  p.x = a.x;
  p.x_stride = a.x_stride;
  p.K = a.w->K;
  p.N = a.w->N;
  p.T = a.T;
  p.KB = a.w->Kp / 128;
  p.row_blocks = (p.N + 127) / 128;
  p.tokens = cut.tokens;
  p.wide = cut.wide;
  p.feature_tiles = GATED ? p.row_blocks : (p.row_blocks + MATS - 1) / MATS;
  p.tiles = p.feature_tiles * ((a.T + cut.tokens - 1) / cut.tokens);
  p.split = cut.split;
  p.act = a.act;
  p.out = a.out;
  p.out_stride = a.out_stride;
  p.status = static_cast<uint32_t*>(a.ws);
  p.vector = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && a.out_stride % 8 == 0;
  p.stages = stages_of(cut);
  p.slots = slots_of(cut);
  cudaError_t e;
  const int sms = sm_count();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cut.split > 1 ? p.tiles * cut.split : p.tiles < sms ? p.tiles : sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kMaxSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cut.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cut.split > 1 ? 2 : 1;
  DSPARK_LAUNCH(kKindLinear4, st,
                e = cudaLaunchKernelEx(&cfg, kernel, a.w->tm, a.up ? a.up->tm : a.w->tm, p));
  return e;
}

}  // namespace

size_t linear4_tile_workspace_bytes(int T, int K) {
  size_t most = 0;
  for (int wide = 0; wide < 2; ++wide)
    for (int tokens = 16; tokens <= kMaxTokens; tokens += 16) {
      const size_t n = (size_t)((T + tokens - 1) / tokens) * tile_bytes(tokens, wide);
      if (n > most) most = n;
    }
  return kStatusBytes + lossy_bytes(T, padded_k(K)) + most * (padded_k(K) / 128);
}

cudaError_t launch_linear4_tile(const Linear4Args& a, const TileCut& cut, cudaStream_t st) {
  const int KB = a.w->Kp / 128;
  uint8_t* lossy = static_cast<uint8_t*>(a.ws) + kStatusBytes;
  cudaError_t e;
  if (!cut.own) {
    DSPARK_LAUNCH(kKindLinear4, st,
                  e = launch_pdl(split_kernel,
                                 dim3((a.T + kSplitWarps - 1) / kSplitWarps, (KB + 3) / 4),
                                 dim3(kSplitWarps * 32), 0, st, a.x, a.x_stride, a.T, a.w->K, KB,
                                 cut.tokens, cut.wide,
                                 lossy + lossy_bytes(a.T, a.w->Kp), lossy));
    if (e != cudaSuccess) return e;
  }
  return a.up            ? launch<2, true>(a, cut, st)
         : cut.mats == 2 ? launch<2, false>(a, cut, st)
                         : launch<1, false>(a, cut, st);
}

cudaError_t linear4_tile_cut(const Linear4Args& a, TileCut* t) {
  for (int mats = a.up ? 2 : 1; mats <= 2; ++mats) {
    const cudaError_t e = ensure_smem_attr(kernel_of(a.up != nullptr, mats), kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  *t = choose(a.w->N, a.T, a.w->Kp / 128, a.up != nullptr);
  return cudaSuccess;
}

}  // namespace dspark
