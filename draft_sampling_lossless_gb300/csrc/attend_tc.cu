// Attention of packed rows over the paged cache on the tensor cores.
//
// For each request and key/value head h, the rows of all G = Hq / Hkv query heads
// that share h are packed, r = j * G + g, so a tile of keys and values is read
// once for all of them.  With S = Q K^T over a tile of 128 positions, and a
// reference m of each row's running maximum:
//
//   P = 2^(c S - c m),  l = l + sum P,  O = O + P V      (c = scale * log2 e)
//
// and out = O / l, lse = (c m + log2 l) ln 2 at the end.  m moves only when the
// maximum has grown by more than 8 powers of two (O and l are then rescaled):
// any reference gives the same quotient, and fp32 has the range.  P enters its
// product as two bf16 terms, its rounding and the rounding of the rest (16
// significant bits in all): a row that a few positions dominate would otherwise
// carry their 2^-9 straight into the result.
//
// Q K^T and P V are tcgen05 MMAs (M = 128 rows).  Two streams, each a warpgroup
// with its own S, P and O in tensor memory, alternate on the tensor core: one's
// softmax runs under the other's products.
//   more than 128 packed rows: the streams take 128 rows each of up to 256, both over
//     every tile (a tile in shared memory feeds 256 rows: the L2 reads of K and
//     V stay half the tensor core's time);
//   up to 128 rows: the same rows, every other tile each.  With 64 or 32 rows the
//     128 MMA rows hold them 2 or 4 times, and each copy keeps to its own half or
//     quarter of the tile's positions (its P is zero elsewhere): softmax work
//     shrinks with the rows, and no warp waits for another's maximum.  The copies
//     and the two streams are joined once, at the end.
//
// Work is split evenly by tiles over the SMs, in the order (request, row tile, head,
// position tile); a block that gets part of an item leaves its O, m, l in the
// workspace, and the last of the item's blocks to finish joins them in block order
// (results do not depend on which one that is).  The lengths are read on
// the device: every block finds its own range with a scan over the requests.
//
// Roles: warps 0-7 the two softmax warpgroups (they also load Q and store), warp 8
// issues the MMAs, warp 9 the TMA loads (10 and 11 complete its warpgroup).  Every
// wait is bounded; a timeout sets DSPARK_DEVFLAG_TIMEOUT and ends the kernel.
#include "cache.cuh"
#include "f32x2.cuh"
#include "sm100.cuh"

namespace dspark {

namespace {

using namespace sm100;

constexpr int kBN = 128;                     // positions a tile
constexpr int kThreads = 384;  // three warpgroups: setmaxnreg moves registers between them
constexpr int kSoftThreads = 256;
constexpr int kWarpMma = 8;
constexpr int kWarpTma = 9;
constexpr int kSegDepth = 4;
constexpr int kMaxCtas = 160;
constexpr uint32_t kHalf = kBN * 128;        // bytes of 128 rows of 64 values
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;              // S at 0 and 128, O at 256 and 256 + DP
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.0f;                // log2 growth of a maximum that moves the reference
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint32_t kCounterOffset = 256;     // workspace: status word, counters, partials
constexpr uint32_t kPartOffset = 4096;
constexpr int kMinTiles = 2;

// n / d for 0 <= n < 2^31 by a multiplication (d fixed for the launch): with
// 2^(s-1) < d <= 2^s and mul = floor(2^32 (2^s - d) / d) + 1, n / d is
// (mulhi(n, mul) + n) >> s (Granlund and Montgomery 1994).
struct Divider {
  uint32_t mul, shift;
  __device__ __forceinline__ int operator()(int n) const {
    return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
  }
};
Divider divider(int d) {
  Divider v;
  v.shift = 0;
  while ((1ll << v.shift) < d) ++v.shift;
  v.mul = (uint32_t)(((1ull << 32) * ((1ull << v.shift) - d)) / d + 1);
  return v;
}

struct Params {
  CacheView c;
  int Hq, G, max_rows, causal, window;
  Divider by_G;
  float scale;
  const __nv_bfloat16* q;
  int64_t q_stride;
  __nv_bfloat16* out;
  float* lse;
  unsigned* counters;  // [kMaxCtas], zero between calls
  float* part;         // [kMaxCtas][2] records of O [DP / 4][rows][4], (m, l) [rows]
};

// The number of 128- or 256-row tiles that one item holds.
template <bool WIDE>
struct Shape {
  static constexpr int kRows = WIDE ? 256 : 128;
};
template <int DP, bool WIDE>
struct Smem {
  static constexpr uint32_t kTile = kHalf * (DP / 64);  // a K, V or Q tile
  static constexpr uint32_t kQBytes =
      kTile * (WIDE ? 2 : 1) > 32768 ? kTile * (WIDE ? 2 : 1) : 32768;  // also the join's buffer
  static constexpr int kFit = (int)((232448 - 4096 - kQBytes + 1024) / kTile);
  static constexpr int kSlots = kFit > 12 ? 12 : kFit;
  static constexpr uint32_t kXchOffset = kQBytes + kSlots * kTile;
  static constexpr uint32_t kSegOffset = kXchOffset + kSoftThreads * 8;
  static constexpr uint32_t kBarOffset = kSegOffset + kSegDepth * 64;
  static constexpr int kBars = 2 * kSlots + 2 * kSegDepth + 1 + 2 + 2 + 2 + 1;
  static constexpr uint32_t kTotal = kBarOffset + kBars * 8 + 16 + 32;
  static_assert(kTotal <= 232448, "shared memory");
};
template <int DP>
__host__ __device__ constexpr size_t record_floats(int rows) {
  return (size_t)rows * DP + (size_t)rows * 2;
}

struct Req {
  int row0, m, ctx;
};

// Request n's rows and context, clamped so that whatever the tables hold no
// address is out of range and no loop is long.
__device__ __forceinline__ Req load_req(const Params& p, int n) {
  int a = __ldg(p.c.row_off + n), b = __ldg(p.c.row_off + n + 1), ctx = __ldg(p.c.ctx + n);
  a = min(max(a, 0), p.c.T);
  b = min(max(b, a), p.c.T);
  const int cap = p.c.max_pages << p.c.log_page;
  Req r;
  r.row0 = a;
  r.m = min(b - a, p.max_rows);
  r.ctx = min(max(ctx, -(1 << 29)), cap);
  return r;
}

// The rows and positions of one item.
struct Item {
  int r0, nrows, lo, hi, tile0, ntiles;
};
template <int ROWS>
__device__ __forceinline__ Item item_of(const Params& p, const Req& q, int qt) {
  Item it;
  const int M = q.m * p.G;
  it.r0 = qt * ROWS;
  it.nrows = min(ROWS, M - it.r0);
  const int j0 = p.by_G(it.r0), j1 = p.by_G(it.r0 + it.nrows - 1);
  it.hi = max(p.causal ? q.ctx + j1 + 1 : q.ctx + q.m, 0);
  it.lo = p.window > 0 ? min(max(q.ctx + j0 - p.window + 1, 0), it.hi) : 0;
  it.tile0 = it.lo / kBN;
  it.ntiles = max(1, (it.hi + kBN - 1) / kBN - it.tile0);
  return it;
}
template <int ROWS>
__device__ __forceinline__ int row_tiles(const Params& p, int m) {
  return (m * p.G + ROWS - 1) / ROWS;
}

struct Segment {  // part of an item that this block computes
  int row0, m, ctx, h, r0, nrows, lo, hi, tile0, ntiles;
  int split;  // 0: the whole item, 1 / 2: its partial result goes to record 0 / 1
  int first, last;  // the item's blocks
  int pad[3];
};
static_assert(sizeof(Segment) == 64, "a segment's words");

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         uint32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait_sleep(bar, parity, 1000)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitNs) {
      *abort_flag = 1;
      set_flag(status, kFlagWaitTimeout);
      return false;
    }
  }
}

// Registers a thread after the roles part: 256 x 200 + 128 x 104 = 384 x 168.
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Barrier of the softmax warpgroups.
__device__ __forceinline__ void soft_sync() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(kSoftThreads) : "memory");
}
// The same; every thread learns whether any of them brought `v`.
__device__ __forceinline__ bool soft_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(kSoftThreads)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Blocks 0 .. ctas-1 take `each` tiles, the first `extra` of them one more.
struct Range {
  int64_t each, u0, u1;  // u0 .. u1 - 1: this block's tiles
  int ctas, extra;
  int n;                 // the request of tile u0
  int64_t before;        // tiles of the requests before n
  Req q;                 // request n

  __device__ __forceinline__ int block_of(int64_t u) const {
    const int64_t wide = extra * (each + 1);
    return u < wide ? (int)(u / (each + 1)) : extra + (int)((u - wide) / each);
  }
};

struct Found {  // the request of a block's first tile, from the thread that finds it
  int64_t before;
  int n;
  Req q;
};

// Tiles of request n over all row tiles and heads.
template <int ROWS>
__device__ __forceinline__ int64_t req_tiles(const Params& p, const Req& q, int first, int step) {
  int64_t u = 0;
  const int qts = row_tiles<ROWS>(p, q.m);
  for (int qt = first; qt < qts; qt += step) u += item_of<ROWS>(p, q, qt).ntiles;
  return u * p.c.Hkv;
}

// Every block's range of tiles, from a scan over the requests (all threads).
template <int ROWS>
__device__ __forceinline__ Range plan(const Params& p, int64_t* s_sum, Found* s_found) {
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const int per = (p.c.R + kThreads - 1) / kThreads;
  int64_t local = 0;
  Req q = {0, 0, 0};
  for (int i = 0; i < per; ++i) {
    const int n = tid * per + i;
    q = {0, 0, 0};
    if (n < p.c.R) q = load_req(p, n);
    const bool many = row_tiles<ROWS>(p, q.m) > 4;
    if (!many) local += req_tiles<ROWS>(p, q, 0, 1);
    // requests of many row tiles: the warp together
    for (uint32_t left = __ballot_sync(0xffffffffu, many); left != 0; left &= left - 1) {
      const int src = __ffs(left) - 1;
      Req o;
      o.row0 = 0;
      o.m = __shfl_sync(0xffffffffu, q.m, src);
      o.ctx = __shfl_sync(0xffffffffu, q.ctx, src);
      int64_t u = req_tiles<ROWS>(p, o, lane, 32);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) u += __shfl_xor_sync(0xffffffffu, u, d);
      if (lane == src) local += u;
    }
  }
  int64_t incl = local;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) s_sum[wid] = incl;
  __syncthreads();
  int64_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < wid) base += s_sum[w];
    total += s_sum[w];
  }
  Range r;
  // few tiles: fewer blocks, kMinTiles each, rather than more partial results
  r.ctas = (int)min((int64_t)gridDim.x, (total + kMinTiles - 1) / kMinTiles);
  r.u0 = r.u1 = 0;
  if ((int)blockIdx.x >= r.ctas) return r;
  r.each = total < (1ll << 31) ? (int64_t)((uint32_t)total / (uint32_t)r.ctas) : total / r.ctas;
  r.extra = (int)(total - r.each * r.ctas);
  r.u0 = r.each * blockIdx.x + min((int)blockIdx.x, r.extra);
  r.u1 = r.u0 + r.each + ((int)blockIdx.x < r.extra);
  int64_t at = base + incl - local;
  if (at <= r.u0 && r.u0 < at + local) {
    for (int i = 0; i < per; ++i) {
      const int n = tid * per + i;
      if (n >= p.c.R) break;
      if (per > 1) q = load_req(p, n);
      const int64_t u = per == 1 ? local : req_tiles<ROWS>(p, q, 0, 1);
      if (r.u0 < at + u) {
        s_found->n = n;
        s_found->before = at;
        s_found->q = q;
        break;
      }
      at += u;
    }
  }
  __syncthreads();
  r.n = s_found->n;
  r.before = s_found->before;
  r.q = s_found->q;
  return r;
}

__device__ __forceinline__ void mask_chunk(uint32_t (&v)[32], int col, int lo, int hi) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (col + i < lo || col + i >= hi) v[i] = 0xff800000u;
}

__device__ __forceinline__ float max_chunk(const uint32_t (&v)[32], float top) {
  float m[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 32; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m[k] = fmaxf(m[k], fmaxf(__uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1])));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// P of 32 positions in place of their scores: its bf16 rounding in the first 16
// columns, the bf16 rounding of the rest in the other 16.
__device__ __forceinline__ void exp_chunk(const uint32_t (&v)[32], uint32_t t_at, float c2,
                                          float mc, unsigned long long (&sum)[2]) {
  uint32_t out[32];
  const unsigned long long cc = pack2(c2, c2), mm = pack2(-mc, -mc);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a, b;
    unpack2(fma2(pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), cc, mm), a, b);
    a = ex2_approx(a);
    b = ex2_approx(b);
    const unsigned long long e = pack2(a, b);
    sum[i & 1] = add2(sum[i & 1], e);
    out[i] = pack_bf16(a, b);
    unpack2(sub2(e, pack2(__uint_as_float(out[i] << 16), __uint_as_float(out[i] & 0xffff0000u))),
            a, b);
    out[16 + i] = pack_bf16(a, b);
  }
  tmem_st_32x32b_x32(t_at, out);
}

// One tile's P for a warp: its rows' scores of NC * 32 positions from column col0
// of S on, the running reference and sum, and P over S's columns (zero outside
// the warp's own positions).  128 positions are read twice, for the maximum and
// for the exponentials: tensor memory has the bandwidth, registers would spill.
template <int NC, int DP>
__device__ __forceinline__ void softmax_tile(uint32_t t_s, uint32_t t_o, int col0, bool mask,
                                             int rel_lo, int rel_hi, float c2, bool first,
                                             float& m_ref, float& l) {
  constexpr int kHeld = NC < 2 ? 1 : 2;
  uint32_t v[kHeld][32];
  float top = -INFINITY;
#pragma unroll
  for (int k0 = 0; k0 < NC; k0 += kHeld) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k) tmem_ld_32x32b_x32(t_s + col0 + 32 * (k0 + k), v[k]);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
#pragma unroll
      for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[k][i]));
      if (mask) mask_chunk(v[k], col0 + 32 * (k0 + k), rel_lo, rel_hi);
      top = max_chunk(v[k], top);
    }
  }
  if (NC > kHeld) tmem_ld_32x32b_x32(t_s + col0, v[0]);
  if (first) {
    m_ref = top;
  } else if (__any_sync(0xffffffffu, (top - m_ref) * c2 > kGrow)) {
    float f = 1.f;
    if (top > m_ref) {
      f = ex2_approx((m_ref - top) * c2);
      m_ref = top;
    }
    l *= f;
    if (NC > kHeld) tmem_wait_ld_regs(v[0]);
#pragma unroll 1
    for (int ch = 0; ch < DP; ch += 32) {
      uint32_t o[32];
      tmem_ld_32x32b_x32(t_o + ch, o);
      tmem_wait_ld_regs(o);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
      tmem_st_32x32b_x32(t_o + ch, o);
    }
  }
  const float mc = m_ref == -INFINITY ? 0.f : m_ref * c2;
  unsigned long long sum[2] = {0, 0};  // two packed zeros each
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    if (NC > kHeld) {
      // the next chunk's load is in flight under this one's exponentials
      tmem_wait_ld_regs(v[k & 1]);
      if (k + 1 < NC) tmem_ld_32x32b_x32(t_s + col0 + 32 * (k + 1), v[(k + 1) & 1]);
      if (mask) mask_chunk(v[k & 1], col0 + 32 * k, rel_lo, rel_hi);
    }
    exp_chunk(v[k & (kHeld - 1)], t_s + col0 + 32 * k, c2, mc, sum);
  }
  if (NC < 4) {
    uint32_t z[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) z[i] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < col0 / 32 || k >= col0 / 32 + NC) tmem_st_32x32b_x32(t_s + 32 * k, z);
  }
  float a, b;
  unpack2(add2(sum[0], sum[1]), a, b);
  l += a + b;
}

// Zeroes the rows of a V tile that no row of the item sees: whatever is stored
// there, 0 * NaN must not reach a sum.
template <int DP>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int to, int tid) {
  for (int r = from + tid; r < to; r += 128)
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
      *reinterpret_cast<uint4*>(tile + (i >> 3) * kHalf + r * 128 + (i & 7) * 16) =
          make_uint4(0, 0, 0, 0);
}

// Joins the partial results of an item's blocks (all softmax threads of the last
// one to finish).  `buf`, 32 KB of shared memory: the blocks' (m, l) of a
// group of rows, then their weights 2^(m - M) / L; the sums run over the blocks in
// order, eight values a thread with lanes along the rows.
template <int DP, int ROWS>
__device__ __forceinline__ void join(const Params& p, const Segment& sg, float2* buf) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int np = sg.last - sg.first + 1;
  const size_t rec = record_floats<DP>(ROWS);
  const float* rec0 = p.part + ((size_t)sg.first * 2 + 1) * rec;  // the first block's, then
  const float* recs = p.part + ((size_t)sg.first * 2 + 2) * rec;  // two records a block on
  auto part = [&](int i) { return i == 0 ? rec0 : recs + (size_t)(i - 1) * 2 * rec; };
  const int group = min(sg.nrows, 4096 / np);
  for (int r0 = 0; r0 < sg.nrows; r0 += group) {
    const int g = min(group, sg.nrows - r0);
    for (int i = tid; i < np * g; i += kSoftThreads) {
      const int b = i / g, row = i - b * g;
      buf[i] = __ldcg(reinterpret_cast<const float2*>(part(b) + (size_t)ROWS * DP) + r0 + row);
    }
    soft_sync();
    for (int row = warp; row < g; row += kSoftThreads / 32) {
      float M = -INFINITY, L = 0.f;
      for (int b = lane; b < np; b += 32) M = fmaxf(M, buf[b * g + row].x);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
      for (int b = lane; b < np; b += 32) {
        const float2 ml = buf[b * g + row];
        L = fmaf(ml.y, ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M), L);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
      const float inv = L == 0.f ? 0.f : 1.f / L;
      for (int b = lane; b < np; b += 32) {
        const float m = buf[b * g + row].x;
        buf[b * g + row].x = m == -INFINITY ? 0.f : ex2_approx(m - M) * inv;
      }
      if (lane == 0 && p.lse != nullptr) {
        const int r = sg.r0 + r0 + row, j = p.by_G(r);
        p.lse[(int64_t)(sg.row0 + j) * p.Hq + (int64_t)sg.h * p.G + (r - j * p.G)] =
            L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
      }
    }
    soft_sync();
    for (int task = tid; task < g * (DP / 8); task += kSoftThreads) {
      const int d8 = task / g, row = task - d8 * g;
      if (d8 * 8 >= p.c.D) break;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 4
      for (int b = 0; b < np; ++b) {
        const float4* r = reinterpret_cast<const float4*>(part(b)) + (size_t)d8 * 2 * ROWS + r0 + row;
        const float4 u = __ldcg(r), v = __ldcg(r + ROWS);
        const float f = buf[b * g + row].x;
        x.x = fmaf(u.x, f, x.x);
        x.y = fmaf(u.y, f, x.y);
        x.z = fmaf(u.z, f, x.z);
        x.w = fmaf(u.w, f, x.w);
        y.x = fmaf(v.x, f, y.x);
        y.y = fmaf(v.y, f, y.y);
        y.z = fmaf(v.z, f, y.z);
        y.w = fmaf(v.w, f, y.w);
      }
      const int r = sg.r0 + r0 + row, j = p.by_G(r);
      const int64_t at = (int64_t)(sg.row0 + j) * p.Hq + (int64_t)sg.h * p.G + (r - j * p.G);
      *reinterpret_cast<uint4*>(p.out + at * p.c.D + d8 * 8) =
          make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y),
                     pack_bf16(y.z, y.w));
    }
    soft_sync();
  }
}

template <int DP, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  using S = Smem<DP, WIDE>;
  constexpr int kRows = Shape<WIDE>::kRows;
  constexpr int NS = S::kSlots;
  constexpr int NH = DP / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* s_q = smem;
  uint8_t* s_kv = smem + S::kQBytes;
  float2* s_xch = reinterpret_cast<float2*>(smem + S::kXchOffset);
  Segment* s_seg = reinterpret_cast<Segment*>(smem + S::kSegOffset);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBarOffset);
  const uint32_t b_full = smem_u32(bars), b_empty = b_full + 8 * NS;
  const uint32_t b_segFull = b_empty + 8 * NS, b_segEmpty = b_segFull + 8 * kSegDepth;
  const uint32_t b_q = b_segEmpty + 8 * kSegDepth;
  const uint32_t b_s = b_q + 8, b_p = b_s + 16, b_o = b_p + 16, b_drain = b_o + 16;
  volatile int* s_abort = reinterpret_cast<volatile int*>(bars + S::kBars);
  volatile int* s_last = s_abort + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + S::kBars) + 2;
  Found* s_found = reinterpret_cast<Found*>(bars + S::kBars + 2);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* status = p.c.status;

  if (tid == 0) {
    *s_abort = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(b_full + 8 * i, 1);
      mbar_init(b_empty + 8 * i, 1);
    }
    for (int i = 0; i < kSegDepth; ++i) {
      mbar_init(b_segFull + 8 * i, 1);
      mbar_init(b_segEmpty + 8 * i, 9);  // the MMA thread and eight softmax warps
    }
    mbar_init(b_q, kSoftThreads);
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_s + 8 * i, 1);
      mbar_init(b_p + 8 * i, 128);
      mbar_init(b_o + 8 * i, 1);
    }
    mbar_init(b_drain, 1);
    fence_mbar_init();
  }
  const Range rg = plan<kRows>(p, reinterpret_cast<int64_t*>(s_xch), s_found);
  if (rg.u0 >= rg.u1) return;       // no tiles for this block
  if (smem_u32(smem) & 1023) return;  // never: the declared alignment, which the swizzle needs
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(s_tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp >= 8) {
    reg_dec<104>();
    if (warp == kWarpTma) {
      // ------------------------------------------------------------ loads
      const int log_page = p.c.log_page, page = 1 << log_page;
      const int box_rows = min(page, kBN);
      const int n_boxes = kBN / box_rows;  // of each half; lane b looks box b up
      const int none = (int)(p.c.n_pages * p.c.Hkv) << log_page;  // past the pool: zeros
      if (lane == 0) {
        tma_prefetch(&tm_k);
        tma_prefetch(&tm_v);
      }
      int n = rg.n;
      Req q = rg.q;
      int64_t u = rg.u0;
      int qts = row_tiles<kRows>(p, q.m), qt = 0, h, off;
      {
        // the row tile, head and position tile of u0 within its request
        int64_t v = u - rg.before;
        for (;;) {
          const int64_t mine =
              qt + lane < qts ? (int64_t)item_of<kRows>(p, q, qt + lane).ntiles * p.c.Hkv : 0;
          int64_t incl = mine;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
          }
          const uint32_t past = __ballot_sync(0xffffffffu, v < incl);
          if (past != 0 || qt + 32 >= qts) {
            const int src = past != 0 ? __ffs(past) - 1 : 0;
            v -= __shfl_sync(0xffffffffu, incl - mine, src);
            qt += src;
            break;
          }
          v -= __shfl_sync(0xffffffffu, incl, 31);
          qt += 32;
        }
        const int nt = item_of<kRows>(p, q, qt).ntiles;
        h = v < (1ll << 31) ? (int)((uint32_t)v / (uint32_t)nt) : (int)(v / nt);
        off = (int)(v - (int64_t)h * nt);
      }
      int64_t seq = 0;  // tiles loaded; K is ring entry 2 seq, V 2 seq + 1
      bool ok = true;
      for (int sn = 0;; ++sn) {
        const int ss = sn % kSegDepth;
        ok = wait_bar(b_segEmpty + 8 * ss, ((sn / kSegDepth) & 1) ^ 1, s_abort, status);
        if (!__all_sync(0xffffffffu, ok)) break;
        Segment sg;
        const Item it = item_of<kRows>(p, q, qt);
        const bool end = u >= rg.u1;
        sg.row0 = q.row0;
        sg.m = q.m;
        sg.ctx = q.ctx;
        sg.h = h;
        sg.r0 = it.r0;
        sg.nrows = it.nrows;
        sg.lo = it.lo;
        sg.hi = it.hi;
        sg.tile0 = it.tile0 + off;
        sg.ntiles = end ? 0 : (int)min((int64_t)(it.ntiles - off), rg.u1 - u);
        sg.split = sg.first = sg.last = 0;
        if (off != 0 || sg.ntiles != it.ntiles) {
          sg.first = rg.block_of(u - off);
          sg.last = rg.block_of(u - off + it.ntiles - 1);
          sg.split = (int)blockIdx.x == sg.first ? 2 : 1;
        }
        if (lane == 0) {
          s_seg[ss] = sg;
          mbar_arrive(b_segFull + 8 * ss);
        }
        if (end) break;
        if (lane == 0 && __ldg(p.c.row_off + n + 1) - __ldg(p.c.row_off + n) > p.max_rows)
          set_flag(status, kFlagRowRange);
        // this lane's box of a tile: its row of the pool, or `none`
        auto lookup = [&](int tile) {
          if (lane >= n_boxes) return none;
          const int pos = tile * kBN + lane * box_rows;
          if (pos >= sg.hi || pos + box_rows <= sg.lo) return none;
          const int64_t id = page_of(p.c, n, pos);
          if (id < 0) return none;
          return (int)((id * p.c.Hkv + h) << log_page) + (pos & (page - 1));
        };
        int next = lookup(sg.tile0);
        for (int i = 0; i < sg.ntiles; ++i, ++seq) {
          int y[8];
#pragma unroll
          for (int b = 0; b < 8; ++b) y[b] = __shfl_sync(0xffffffffu, next, b);
          if (i + 1 < sg.ntiles) next = lookup(sg.tile0 + i + 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int64_t e = 2 * seq + kv;
            const int slot = (int)(e % NS);
            ok = wait_bar(b_empty + 8 * slot, (uint32_t)((e / NS) & 1) ^ 1, s_abort, status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (elect_one()) {
              const uint32_t full = b_full + 8 * slot;
              const uint32_t dst = smem_u32(s_kv) + slot * S::kTile;
              mbar_arrive_expect_tx(full, S::kTile);
#pragma unroll
              for (int b = 0; b < 8; ++b)
                if (b < n_boxes)
#pragma unroll
                  for (int half = 0; half < NH; ++half)
                    tma_load_2d(dst + half * kHalf + b * box_rows * 128, kv ? &tm_v : &tm_k, full,
                                half * 64, y[b]);
            }
            __syncwarp();
          }
          if (!ok) break;
        }
        if (!ok) break;
        u += sg.ntiles;
        off = 0;
        if (sg.tile0 + sg.ntiles == it.tile0 + it.ntiles && ++h == p.c.Hkv) {
          h = 0;
          if (++qt == qts) {
            qt = 0;
            while (u < rg.u1 && ++n < p.c.R) {
              q = load_req(p, n);
              qts = row_tiles<kRows>(p, q.m);
              if (qts > 0) break;
            }
          }
        }
      }
      if (*s_abort) {
        // the copies in flight land before the block's shared memory goes
        for (int64_t e = max((int64_t)0, 2 * seq - NS); e < 2 * seq; ++e)
          mbar_wait(b_full + 8 * (int)(e % NS), (uint32_t)((e / NS) & 1));
      }
    } else if (warp == kWarpMma) {
      // ------------------------------------------------------------ products
      if (elect_one()) {
        constexpr uint32_t kIdS = idesc_bf16_f32(128, kBN);
        constexpr uint32_t kIdO = idesc_bf16_f32(128, DP) | kIdescTransposeB;
        const int ksteps = (p.c.D + 15) / 16;
        const uint32_t q_at = smem_u32(s_q), kv_at = smem_u32(s_kv);
        int64_t base = 0;  // tiles of the segments before
        uint32_t ph_q = 0, ph_p = 0;
        bool ok = true;
        auto need = [&](int64_t e) {
          ok = ok && wait_bar(b_full + 8 * (int)(e % NS), (uint32_t)((e / NS) & 1), s_abort, status);
          tc_fence_after();
        };
        auto need_p = [&](int s) {
          ok = ok && wait_bar(b_p + 8 * s, (ph_p >> s) & 1, s_abort, status);
          ph_p ^= 1u << s;
          tc_fence_after();
        };
        auto scores = [&](int s, int qtile, int64_t e) {
          const uint32_t a = q_at + qtile * S::kTile, b = kv_at + (uint32_t)(e % NS) * S::kTile;
          for (int k = 0; k < ksteps; ++k) {
            const uint32_t at = (k >> 2) * kHalf + (k & 3) * 32;
            mma_bf16(tmem + s * kBN, desc_kmajor_sw128(a + at), desc_kmajor_sw128(b + at), kIdS,
                     k > 0);
          }
          mma_commit(b_s + 8 * s);
        };
        auto values = [&](int s, int64_t e, bool acc) {
          // 16 positions a step: 2048 bytes on (the sum stays within the 14 address bits)
          const uint64_t v = desc_mnmajor_sw128(kv_at + (uint32_t)(e % NS) * S::kTile, kHalf);
#pragma unroll 1
          for (int k = 0; k < kBN / 16; ++k) {
            const uint32_t a = tmem + s * kBN + (k >> 1) * 32 + (k & 1) * 8;
            mma_bf16_ts(tmem + kColO + s * DP, a, v + k * (2048 >> 4), kIdO, acc || k > 0);
            mma_bf16_ts(tmem + kColO + s * DP, a + 16, v + k * (2048 >> 4), kIdO, 1);
          }
        };
        auto release = [&](int64_t e) { mma_commit(b_empty + 8 * (int)(e % NS)); };
        for (int sn = 0; ok; ++sn) {
          const int ss = sn % kSegDepth;
          ok = wait_bar(b_segFull + 8 * ss, (sn / kSegDepth) & 1, s_abort, status);
          if (!ok) break;
          const int nt = s_seg[ss].ntiles;
          const bool two = s_seg[ss].nrows > 128;
          mbar_arrive(b_segEmpty + 8 * ss);
          if (nt == 0) break;
          ok = wait_bar(b_q, ph_q, s_abort, status);
          if (!ok) break;
          ph_q ^= 1;
          tc_fence_after();
          const int64_t e0 = 2 * base;  // K of tile i: e0 + 2 i, V: one more
          if (two) {
            need(e0);
            if (!ok) break;
            scores(0, 0, e0);
            scores(1, 1, e0);
            release(e0);
            for (int i = 0; i < nt && ok; ++i) {
              const int64_t ev = e0 + 2 * i + 1, ek = ev + 1;
              const bool more = i + 1 < nt;
              need(ev);
              if (more) need(ek);
              need_p(0);
              if (!ok) break;
              values(0, ev, i > 0);
              if (more) scores(0, 0, ek);
              else mma_commit(b_o);
              need_p(1);
              if (!ok) break;
              values(1, ev, i > 0);
              release(ev);
              if (more) {
                scores(1, 1, ek);
                release(ek);
              } else {
                mma_commit(b_o + 8);
              }
            }
          } else {
            for (int i = 0; i < 2 && i < nt && ok; ++i) {
              need(e0 + 2 * i);
              if (!ok) break;
              scores(i, 0, e0 + 2 * i);
              release(e0 + 2 * i);
            }
            for (int i = 0; i < nt && ok; ++i) {
              const int s = i & 1;
              const int64_t ev = e0 + 2 * i + 1;
              need(ev);
              need_p(s);
              if (!ok) break;
              values(s, ev, i >= 2);
              release(ev);
              if (i + 2 < nt) {
                need(ev + 3);
                if (!ok) break;
                scores(s, 0, ev + 3);
                release(ev + 3);
              } else {
                mma_commit(b_o + 8 * s);
              }
            }
          }
          base += nt;
        }
        if (!ok) {
          mma_commit(b_drain);
          mbar_wait(b_drain, 0);
        }
      }
      __syncwarp();
    }
  } else {
    reg_inc<200>();
    // ------------------------------------------------------------ softmax
    const int s = warp >> 2;  // the stream
    const int lrow = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + s * kBN, t_o = tmem + lanes + kColO + s * DP;
    const float c2 = p.scale * kLog2e;
    uint32_t ph_s = 0, ph_o = 0;
    int64_t base = 0;
    for (int sn = 0;; ++sn) {
      const int ss = sn % kSegDepth;
      const bool got = wait_bar(b_segFull + 8 * ss, (sn / kSegDepth) & 1, s_abort, status);
      // all leave together; the barrier also ends the previous segment's use of s_q
      if (soft_any(!got)) break;
      const Segment sg = s_seg[ss];
      __syncwarp();
      if (lane == 0) mbar_arrive(b_segEmpty + 8 * ss);
      if (sg.ntiles == 0) break;
      const bool two = sg.nrows > 128;
      const int rep = two || sg.nrows > 64 ? 1 : sg.nrows > 32 ? 2 : 4;
      const int rp = 128 / rep;  // rows of a copy

      // Q: rows past the item's are zero
      {
        uint8_t* dst = s_q + (two ? s * S::kTile : 0);
        const int r_first = sg.r0 + (two ? s * 128 : 0);
        const int threads = two ? 128 : 256, t0 = two ? lrow : tid;
        for (int i = t0; i < 128 * (DP / 8); i += threads) {
          const int row = i / (DP / 8), ch = i % (DP / 8);
          const int r = r_first + row % rp;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (r < sg.r0 + sg.nrows && ch * 8 < p.c.D) {
            const int j = p.by_G(r);
            x = __ldg(reinterpret_cast<const uint4*>(
                p.q + (int64_t)(sg.row0 + j) * p.q_stride +
                ((int64_t)sg.h * p.G + (r - j * p.G)) * p.c.D + ch * 8));
          }
          *reinterpret_cast<uint4*>(dst + (ch >> 3) * kHalf + row * 128 +
                                    (((ch & 7) ^ (row & 7)) << 4)) = x;
        }
        fence_proxy_async_smem();
        mbar_arrive(b_q);
      }

      // this thread's row and the positions it sees
      const int my = (two ? s * 128 : 0) + lrow % rp;
      const bool live = my < sg.nrows;
      const int pos = sg.ctx + p.by_G(sg.r0 + my);
      const int row_hi = !live ? 0x7fffffff : p.causal ? pos + 1 : sg.ctx + sg.m;
      const int row_lo = !live || p.window == 0 ? 0 : pos - p.window + 1;
      const int first_r = sg.r0 + (two ? s * 128 : 0);
      const int last_r = sg.r0 + min(sg.nrows, first_r - sg.r0 + 128) - 1;
      const int min_hi = p.causal ? sg.ctx + p.by_G(first_r) + 1 : sg.ctx + sg.m;
      const int max_lo = p.window == 0 ? 0 : sg.ctx + p.by_G(last_r) - p.window + 1;
      const int nc = 4 / rep, col0 = two ? 0 : (lrow / rp) * (kBN / rep);

      float m_ref = -INFINITY, l = 0.f;
      const int step = two ? 1 : 2, i0 = two ? 0 : s;
      for (int i = i0; i < sg.ntiles; i += step) {
        const int t0 = (sg.tile0 + i) * kBN;
        const int64_t e = 2 * (base + i) + 1;
        wait_bar(b_s + 8 * s, ph_s, s_abort, status);
        __syncwarp();
        ph_s ^= 1;
        tc_fence_after();
        const bool mask = t0 < max_lo || t0 + kBN > min_hi;
        const bool first = i == i0;
        const int rel_lo = row_lo - t0, rel_hi = row_hi - t0;
        if (nc == 4)
          softmax_tile<4, DP>(t_s, t_o, col0, mask, rel_lo, rel_hi, c2, first, m_ref, l);
        else if (nc == 2)
          softmax_tile<2, DP>(t_s, t_o, col0, mask, rel_lo, rel_hi, c2, first, m_ref, l);
        else
          softmax_tile<1, DP>(t_s, t_o, col0, mask, rel_lo, rel_hi, c2, first, m_ref, l);
        if ((!two || s == 0) && (t0 < sg.lo || t0 + kBN > sg.hi)) {
          const int slot = (int)(e % NS);
          wait_bar(b_full + 8 * slot, (uint32_t)((e / NS) & 1), s_abort, status);
          uint8_t* tile = s_kv + (size_t)slot * S::kTile;
          zero_rows<DP>(tile, 0, sg.lo - t0, lrow);
          zero_rows<DP>(tile, max(sg.hi - t0, 0), kBN, lrow);
          fence_proxy_async_smem();
          __syncwarp();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(b_p + 8 * s);
      }
      const bool has = i0 < sg.ntiles;
      if (has) {
        wait_bar(b_o + 8 * s, ph_o, s_abort, status);
        __syncwarp();
        ph_o ^= 1;
        tc_fence_after();
      }
      base += sg.ntiles;

      float* rec = p.part +
                   ((size_t)blockIdx.x * 2 + (sg.split == 2 ? 1 : 0)) * record_floats<DP>(kRows);
      const float mine = m_ref == -INFINITY ? -INFINITY : m_ref * c2;
      if (two) {
        const int r = sg.r0 + my, j = p.by_G(r);
        const int64_t at = (int64_t)(sg.row0 + j) * p.Hq + (int64_t)sg.h * p.G + (r - j * p.G);
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int ch = 0; ch < DP; ch += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(t_o + ch, o);
          tmem_wait_ld_regs(o);
          if (live && sg.split == 0) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              if (ch + i < p.c.D) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  w[k] = pack_bf16(__uint_as_float(o[i + 2 * k]) * inv,
                                   __uint_as_float(o[i + 2 * k + 1]) * inv);
                *reinterpret_cast<uint4*>(p.out + at * p.c.D + ch + i) =
                    make_uint4(w[0], w[1], w[2], w[3]);
              }
          } else if (live) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              __stcg(reinterpret_cast<uint4*>(rec) + (size_t)((ch + i) / 4) * kRows + my,
                     make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]));
          }
          __syncwarp();
        }
        if (live) {
          if (sg.split != 0)
            __stcg(reinterpret_cast<float2*>(rec + (size_t)kRows * DP) + my, make_float2(mine, l));
          else if (p.lse != nullptr)
            p.lse[at] = l == 0.f ? -INFINITY : (mine + log2f(l)) * kLn2;
        }
      } else {
        // the copies of a row in the streams: a common reference first
        const int parts = sg.ntiles > 1 ? 2 * rep : rep;
        s_xch[tid] = make_float2(mine, l);
        soft_sync();
        const int rr = lrow % rp;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int a = 0; a < 8; ++a)
          if (a < parts) M = fmaxf(M, s_xch[a * rp + rr].x);
#pragma unroll
        for (int a = 0; a < 8; ++a)
          if (a < parts) {
            const float2 ml = s_xch[a * rp + rr];
            L = fmaf(ml.y, ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M), L);
          }
        const float w = mine == -INFINITY ? 0.f : ex2_approx(mine - M);
        soft_sync();
        if (tid < rp) s_xch[tid] = make_float2(M, L);
        // then their sums through shared memory (Q is no longer read): as many
        // columns a round as 32 KB hold for the rows there are
        float* buf = reinterpret_cast<float*>(s_q);
        const int brows = sg.nrows <= 8 ? 8 : sg.nrows <= 16 ? 16 : rp;
        const int cw = min(DP, 8192 / (2 * rep * brows)), log_c4 = 31 - __clz(cw >> 2);
        const int brow = (tid / rp) * brows + rr;
#pragma unroll 1
        for (int ch = 0; ch < DP; ch += cw) {
          __syncwarp();
          if (has) {
#pragma unroll 1
            for (int c = 0; c < cw; c += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(t_o + ch + c, o);
              tmem_wait_ld_regs(o);
              if (rr < brows) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  *reinterpret_cast<float4*>(buf + brow * cw + c + ((i ^ (brow & 7)) << 2)) =
                      make_float4(__uint_as_float(o[4 * i]) * w, __uint_as_float(o[4 * i + 1]) * w,
                                  __uint_as_float(o[4 * i + 2]) * w,
                                  __uint_as_float(o[4 * i + 3]) * w);
              }
              __syncwarp();
            }
          }
          soft_sync();
          for (int task = tid; task < brows << log_c4; task += kSoftThreads) {
            const int row = task >> log_c4, d4 = task & ((1 << log_c4) - 1);
            if (row >= sg.nrows) break;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int a = 0; a < 8; ++a)
              if (a < parts) {
                const int src = a * brows + row;
                const float4 y =
                    *reinterpret_cast<const float4*>(buf + src * cw + ((d4 ^ (src & 7)) << 2));
                x.x += y.x;
                x.y += y.y;
                x.z += y.z;
                x.w += y.w;
              }
            if (sg.split != 0) {
              __stcg(reinterpret_cast<float4*>(rec) + (size_t)(ch / 4 + d4) * kRows + row, x);
            } else if (ch + d4 * 4 < p.c.D) {
              const float Lr = s_xch[row].y;
              const float inv = Lr == 0.f ? 0.f : 1.f / Lr;
              const int r = sg.r0 + row, j = p.by_G(r);
              const int64_t at =
                  (int64_t)(sg.row0 + j) * p.Hq + (int64_t)sg.h * p.G + (r - j * p.G);
              *reinterpret_cast<uint2*>(p.out + at * p.c.D + ch + d4 * 4) =
                  make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
            }
          }
          soft_sync();
        }
        if (tid < sg.nrows) {
          if (sg.split != 0) {
            __stcg(reinterpret_cast<float2*>(rec + (size_t)kRows * DP) + tid, make_float2(M, L));
          } else if (p.lse != nullptr) {
            const int r = sg.r0 + tid, j = p.by_G(r);
            p.lse[(int64_t)(sg.row0 + j) * p.Hq + (int64_t)sg.h * p.G + (r - j * p.G)] =
                L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
          }
        }
      }
      if (sg.split != 0) {
        __threadfence();
        soft_sync();
        if (tid == 0) {
          const unsigned want = (unsigned)(sg.last - sg.first);
          const unsigned old = atomicAdd(p.counters + sg.first, 1u);
          *s_last = old == want;
          if (old == want) p.counters[sg.first] = 0;
        }
        soft_sync();
        if (*s_last) {
          __threadfence();
          join<DP, kRows>(p, sg, reinterpret_cast<float2*>(s_q));
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int DP, bool WIDE>
cudaError_t launch_one(const AttendArgs& a, const Params& p, cudaStream_t st) {
  auto kernel = attend_tc_kernel<DP, WIDE>;
  constexpr uint32_t bytes = Smem<DP, WIDE>::kTotal;
  cudaError_t e = ensure_smem_attr((const void*)kernel, bytes);
  if (e != cudaSuccess) return e;
  const int grid = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
  DSPARK_LAUNCH(kKindAttend, st,
                kernel<<<grid, kThreads, bytes, st>>>(a.desc->tm_k, a.desc->tm_v, p));
  return cudaGetLastError();
}

}  // namespace

// Row tiles of 128 packed rows while no request has more, else of 256.
static bool wide(int max_rows, int group) { return (int64_t)max_rows * group > 128; }

size_t attend_workspace_bytes(int T, int group, int D) {
  const int rows = wide(T, group) ? 256 : 128;
  const size_t rec = D > 64 ? record_floats<128>(rows) : record_floats<64>(rows);
  return kPartOffset + (size_t)kMaxCtas * 2 * rec * sizeof(float);
}

cudaError_t launch_attend_tc(const AttendArgs& a, cudaStream_t st) {
  Params p;
  p.c = a.c;
  p.Hq = a.Hq;
  p.G = a.Hq / a.c.Hkv;
  p.by_G = divider(p.G);
  p.max_rows = a.max_rows;
  p.causal = a.causal;
  p.window = a.window;
  p.scale = a.scale;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.counters = reinterpret_cast<unsigned*>(static_cast<char*>(a.ws) + kCounterOffset);
  p.part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + kPartOffset);
  const bool w = wide(p.max_rows, p.G);
  if (a.c.D > 64) return w ? launch_one<128, true>(a, p, st) : launch_one<128, false>(a, p, st);
  return w ? launch_one<64, true>(a, p, st) : launch_one<64, false>(a, p, st);
}

}  // namespace dspark
