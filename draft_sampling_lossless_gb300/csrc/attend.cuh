// What the attention kernels share (attend_few.cu, attend_many.cu): the split of
// the work over the blocks, the load of the pages, and the join of partial results.
//
// For each request and key/value head h, the rows of all G = Hq / Hkv query heads
// that share h are packed, r = j * G + g, and cut into row tiles; an item is one row
// tile of one head of one request, its work the tiles of 128 positions that its
// rows see.  The items, in the order (request, row tile, head), are split evenly over
// the blocks, an item counting its tiles and kItemCost more for what it costs besides.
// A block that gets part of an item leaves its O, m, l in the workspace, and the last
// of the item's blocks to finish joins them in block order (results do not depend on
// which one that is).  A join takes as long as a few tiles, so a cut that falls
// within kSnap tiles of an item's end moves there.  The lengths are read on the
// device: every block finds its own range with a scan over the requests (2 us).  One
// warp walks the range, loads K, and hands the others their parts of items through a
// short queue of segments.
#pragma once

#include "cache.cuh"
#include "f32x2.cuh"
#include "sm100.cuh"

namespace dspark {
namespace attend {

using namespace sm100;

constexpr int kBN = 128;               // positions a tile
constexpr int kSegDepth = 4;
constexpr int kMaxCtas = 160;
constexpr int kMaxSmem = 232448;
constexpr uint32_t kHalf = kBN * 128;  // bytes of 128 rows of 128 bytes
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A role may wait for another's whole part of an item, longer than the library's usual
// second in the largest calls.
constexpr uint32_t kWaitLimitNs = 4000000000u;
constexpr uint32_t kCounterOffset = 256;  // workspace: status word, counters, partials
constexpr uint32_t kPartOffset = 4096;
constexpr int kItemCost = 2;  // in tiles: Q, the final sums and the store of an item
constexpr int kSnap = 3;
constexpr int kMinUnits = 6;  // fewer blocks rather than less work for each

// n / d for 0 <= n < 2^31 by a multiplication (d fixed for the launch): with
// 2^(s-1) < d <= 2^s and mul = floor(2^32 (2^s - d) / d) + 1, n / d is
// (mulhi(n, mul) + n) >> s (Granlund and Montgomery 1994).
struct Divider {
  uint32_t mul, shift;
  __device__ __forceinline__ int operator()(int n) const {
    return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
  }
};
inline Divider divider(int d) {
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
  float* part;         // [kMaxCtas][2] records: O, then (m, l) [rows]
};

__host__ __device__ constexpr size_t record_floats(int rows, int DP) {
  return (size_t)rows * DP + (size_t)rows * 2;
}

struct Req {
  int row0, m, ctx;
  int tiles, rows;  // row tiles, and the packed rows of each (the last may have fewer)
};

// Request n's rows and context, clamped so that whatever the tables hold no
// address is out of range and no loop is long.
template <int ROWS>
__device__ __forceinline__ Req load_req(const Params& p, int n) {
  int a = __ldg(p.c.row_off + n), b = __ldg(p.c.row_off + n + 1), ctx = __ldg(p.c.ctx + n);
  a = min(max(a, 0), p.c.T);
  b = min(max(b, a), p.c.T);
  const int cap = p.c.max_pages << p.c.log_page;
  Req r;
  r.row0 = a;
  r.m = min(b - a, p.max_rows);
  r.ctx = min(max(ctx, -(1 << 29)), cap);
  // as few tiles as hold the rows, all of one size: the tile count measures the work
  const int M = r.m * p.G;
  r.tiles = (M + ROWS - 1) / ROWS;
  r.rows = r.tiles > 1 ? (M + r.tiles - 1) / r.tiles : M;
  return r;
}

// The rows and positions of one item.
struct Item {
  int r0, nrows, lo, hi, tile0, ntiles;
};
__device__ __forceinline__ Item item_of(const Params& p, const Req& q, int qt) {
  Item it;
  it.r0 = qt * q.rows;
  it.nrows = min(q.rows, q.m * p.G - it.r0);
  const int j0 = p.by_G(it.r0), j1 = p.by_G(it.r0 + it.nrows - 1);
  it.hi = max(p.causal ? q.ctx + j1 + 1 : q.ctx + q.m, 0);
  it.lo = p.window > 0 ? min(max(q.ctx + j0 - p.window + 1, 0), it.hi) : 0;
  it.tile0 = it.lo / kBN;
  it.ntiles = max(1, (it.hi + kBN - 1) / kBN - it.tile0);
  return it;
}

// Where packed row r of head h goes: its index in [T][Hq].
__device__ __forceinline__ int64_t out_row(const Params& p, int row0, int h, int r) {
  const int j = p.by_G(r);
  return (int64_t)(row0 + j) * p.Hq + (int64_t)h * p.G + (r - j * p.G);
}
// Its query: 8 values from d on (zeros past D).
__device__ __forceinline__ uint4 load_q(const Params& p, int row0, int h, int r, int d) {
  if (d >= p.c.D) return make_uint4(0, 0, 0, 0);
  const int j = p.by_G(r);
  return __ldg(reinterpret_cast<const uint4*>(p.q + (int64_t)(row0 + j) * p.q_stride +
                                              ((int64_t)h * p.G + (r - j * p.G)) * p.c.D + d));
}

struct Segment {  // part of an item that this block computes
  int row0, m, ctx, h, r0, nrows, lo, hi, tile0, ntiles;
  int split;        // 0: the whole item, 1 / 2: its partial result goes to record 0 / 1
  int first, last;  // the item's blocks
  int n;            // its request
  int pad[2];
};
static_assert(sizeof(Segment) == 64, "a segment's words");

// A wait that has run out shows in the block's flag; the block reports it at its end.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_wait_or_abort(bar, parity, abort_flag, kWaitLimitNs);
}

// Registers a thread after the roles part.
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Barrier `id` of n threads; the second form tells each whether any brought `v`.
__device__ __forceinline__ void group_sync(int id, int n) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ bool group_any(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 16 e4m3 codes as packed bf16 times 2^(byte - 127), exact but for what falls below
// bf16's range.  Code s eeee mmm moved to s 0000eeee mmm0000 is its value times 2^-120: the
// factor 2^(byte - 7) makes up for that, in two steps where it passes bf16's range.
__device__ __forceinline__ void codes_to_bf16(const uint32_t (&w)[4], uint32_t byte,
                                              uint32_t (&out)[8]) {
  byte = exponent_byte(byte);
  const uint32_t e = min(byte + 120u, 254u), f = (e << 7) | (e << 23);
  uint32_t nan = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    nan |= (w[j] & 0x7f7f7f7fu) + 0x01010101u;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t u;  // two codes with their signs over the bytes above, four bits up
      asm("prmt.b32 %0, %1, 0, %2;" : "=r"(u) : "r"(w[j]), "r"(k ? 0xb3a2 : 0x9180));
      u = (u << 4) & 0x87f087f0u;
      const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                       *reinterpret_cast<const __nv_bfloat162*>(&f));
      out[2 * j + k] = *reinterpret_cast<const uint32_t*>(&x);
    }
  }
  if (byte > 134u) {
    const uint32_t g = (byte - 7u) * 0x00800080u;  // 2^(byte - 134), both halves
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(out + j),
                                       *reinterpret_cast<const __nv_bfloat162*>(&g));
      out[j] = *reinterpret_cast<const uint32_t*>(&x);
    }
  }
  if (nan & 0x80808080u) {  // a code without a value
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t t = (w[j] & 0x7f7f7f7fu) + 0x01010101u;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t u;  // the bytes' top bits over two bytes each
        asm("prmt.b32 %0, %1, 0, %2;" : "=r"(u) : "r"(t), "r"(k ? 0xbbaa : 0x9988));
        out[2 * j + k] |= u & 0x7fff7fffu;
      }
    }
  }
}

// Turns tiles of codes (128 bytes a row, as the TMA swizzles them) into bf16 tiles.  Eight
// lanes that access shared memory together take four chunks of 16 codes of two rows, r and
// r ^ 5 of a group of eight: their reads, and the even and the odd halves of their writes,
// fall in different banks.
template <int DP, int WARPS>
struct Converter {
  static constexpr int kStep = (DP > 64 ? 4 : 8) * WARPS;  // rows a step
  int row;            // of the first step
  uint32_t from, to;  // its codes, its first 8 values (the others 16 bytes ^ on)
  __device__ __forceinline__ Converter(int warp, int lane) {
    const int c = ((lane >> 1) & 3) | (DP > 64 ? (lane >> 1) & 4 : 0);
    const int p = DP > 64 ? (lane >> 4) | ((warp & 1) << 1) : lane >> 3;
    const int r = lane & 1 ? p ^ 5 : p;
    row = (DP > 64 ? warp >> 1 : warp) * 8 + r;
    from = row * 128 + ((c ^ r) << 4);
    to = (c >> 2) * kHalf + row * 128 + ((((c & 3) * 2) ^ r) << 4);
  }
  // `lo`, `hi`: rows outside become zeros (0 * NaN must not reach a sum).
  __device__ __forceinline__ void operator()(const uint8_t* src, const uint8_t* exps,
                                             uint8_t* dst, int lo, int hi) const {
    const bool edge = lo > 0 || hi < kBN;
    src += from;
    exps += row;
    uint4 next = *reinterpret_cast<const uint4*>(src);
    uint32_t byte = *exps;
#pragma unroll 1
    for (int k = 0; k < kBN / kStep; ++k) {
      uint32_t w[4] = {next.x, next.y, next.z, next.w}, h[8];
      const uint32_t b = byte;
      src += kStep * 128;
      exps += kStep;
      if (k + 1 < kBN / kStep) {
        next = *reinterpret_cast<const uint4*>(src);
        byte = *exps;
      }
      const int r = row + k * kStep;
      if (edge && (r < lo || r >= hi)) w[0] = w[1] = w[2] = w[3] = 0;
      codes_to_bf16(w, b, h);
      *reinterpret_cast<uint4*>(dst + to) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(dst + (to ^ 16)) = make_uint4(h[4], h[5], h[6], h[7]);
      dst += kStep * 128;
    }
  }
};

// Blocks 0 .. ctas-1 take `each` units (tiles and items' costs), the first `extra` of
// them one more.
struct Found {  // the request that holds a unit, from the thread that finds it
  int64_t before;  // units of the requests before it
  int n;
  Req q;
};
struct Range {
  int64_t each, u0, u1;  // u0 .. u1 - 1: this block's units
  int ctas, extra;
  bool last;             // u1 is the end of all work

  __device__ __forceinline__ int block_of(int64_t u) const {
    const int64_t wide = extra * (each + 1), d = u < wide ? each + 1 : each;
    const int64_t n = u < wide ? u : u - wide;
    const int q = n < (1ll << 31) && d < (1ll << 31) ? (int)((uint32_t)n / (uint32_t)d)
                                                     : (int)(n / d);
    return u < wide ? q : extra + q;
  }
};

// Units of a request over all heads and every step-th row tile from `first` on.
__device__ __forceinline__ int64_t req_units(const Params& p, const Req& q, int first, int step) {
  int64_t u = 0;
#pragma unroll 1
  for (int qt = first; qt < q.tiles; qt += step) u += item_of(p, q, qt).ntiles + kItemCost;
  return u * p.c.Hkv;
}

// Every block's range of units, from a scan over the requests (all threads);
// s_found[0] and [1] get the requests of u0 and u1.
template <int ROWS, int THREADS>
__device__ __forceinline__ Range plan(const Params& p, int64_t* s_sum, Found* s_found) {
  const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
  const int per = (p.c.R + THREADS - 1) / THREADS;
  int64_t local = 0;
  Req q = {};
#pragma unroll 1
  for (int i = 0; i < per; ++i) {
    const int n = tid * per + i;
    q = Req{};
    if (n < p.c.R) q = load_req<ROWS>(p, n);
    const bool many = q.tiles > 4;
    if (!many) local += req_units(p, q, 0, 1);
    // requests of many row tiles: the warp together
    for (uint32_t left = __ballot_sync(0xffffffffu, many); left != 0; left &= left - 1) {
      const int src = __ffs(left) - 1;
      Req o;
      o.row0 = 0;
      o.m = __shfl_sync(0xffffffffu, q.m, src);
      o.ctx = __shfl_sync(0xffffffffu, q.ctx, src);
      o.tiles = __shfl_sync(0xffffffffu, q.tiles, src);
      o.rows = __shfl_sync(0xffffffffu, q.rows, src);
      int64_t u = req_units(p, o, lane, 32);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) u += __shfl_xor_sync(0xffffffffu, u, d);
      if (lane == src) local += u;
    }
  }
  int64_t incl = local;
#pragma unroll 1
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) s_sum[wid] = incl;
  __syncthreads();
  int64_t sums = lane < THREADS / 32 ? s_sum[lane] : 0;
#pragma unroll 1
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, sums, d);
    if (lane >= d) sums += o;
  }
  const int64_t total = __shfl_sync(0xffffffffu, sums, 31);
  const int64_t base = __shfl_sync(0xffffffffu, sums, wid) - __shfl_sync(0xffffffffu, incl, 31);
  Range r;
  r.ctas = (int)min((int64_t)gridDim.x, (total + kMinUnits - 1) / kMinUnits);
  r.u0 = r.u1 = 0;
  if ((int)blockIdx.x >= r.ctas) return r;
  r.each = total < (1ll << 31) ? (int64_t)((uint32_t)total / (uint32_t)r.ctas) : total / r.ctas;
  r.extra = (int)(total - r.each * r.ctas);
  r.u0 = r.each * blockIdx.x + min((int)blockIdx.x, r.extra);
  r.u1 = r.u0 + r.each + ((int)blockIdx.x < r.extra);
  r.last = r.u1 == total;
  int64_t at = base + incl - local;
  if (at < r.u1 + 1 && r.u0 < at + local) {
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
      const int n = tid * per + i;
      if (n >= p.c.R) break;
      if (per > 1) q = load_req<ROWS>(p, n);
      const int64_t u = per == 1 ? local : req_units(p, q, 0, 1);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int64_t x = k ? r.u1 : r.u0;
        if (at <= x && x < at + u) {
          s_found[k].n = n;
          s_found[k].before = at;
          s_found[k].q = q;
        }
      }
      at += u;
    }
  }
  __syncthreads();
  return r;
}

// A place in the order of items: `tile` of the nt of head h of row tile qt of request
// n; n = R is the end.
struct Place {
  Req q;
  int64_t a;  // units before the item
  int n, qt, h, tile, nt;
};

// What a cut does to an item of nt tiles: up to `low` tiles in, it moves to the
// item's start, from nt - high on to its end.
__device__ __forceinline__ int snap_low(int nt) { return min(kSnap, nt >> 1); }
__device__ __forceinline__ int snap_high(int nt) { return min(kSnap, nt - snap_low(nt) - 1); }

// The first tile of the next item (whose nt is not known yet).
template <int ROWS>
__device__ __forceinline__ void next_item(const Params& p, Place& w) {
  w.a += w.nt + kItemCost;
  w.tile = 0;
  w.nt = 1;
  if (++w.h < p.c.Hkv) return;
  w.h = 0;
  if (++w.qt < w.q.tiles) return;
  w.qt = 0;
#pragma unroll 1
  while (++w.n < p.c.R) {
    w.q = load_req<ROWS>(p, w.n);
    if (w.q.tiles > 0) break;
  }
}

// The place of unit u, a cut between two blocks (warp-collective).
template <int ROWS>
__device__ __forceinline__ Place locate(const Params& p, const Found& f, int64_t u) {
  const int lane = threadIdx.x & 31;
  Place w;
  w.q = f.q;
  w.n = f.n;
  w.qt = 0;
  int64_t v = u - f.before;
#pragma unroll 1
  while (w.q.tiles > 1) {
    const int64_t mine =
        w.qt + lane < w.q.tiles
            ? (int64_t)(item_of(p, w.q, w.qt + lane).ntiles + kItemCost) * p.c.Hkv
            : 0;
    int64_t incl = mine;
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, v < incl);
    if (past != 0 || w.qt + 32 >= w.q.tiles) {
      const int src = past != 0 ? __ffs(past) - 1 : 0;
      v -= __shfl_sync(0xffffffffu, incl - mine, src);
      w.qt += src;
      break;
    }
    v -= __shfl_sync(0xffffffffu, incl, 31);
    w.qt += 32;
  }
  w.nt = item_of(p, w.q, w.qt).ntiles;
  const int units = w.nt + kItemCost;
  w.h = v < (1ll << 31) ? (int)((uint32_t)v / (uint32_t)units) : (int)(v / units);
  const int off = (int)(v - (int64_t)w.h * units);
  w.a = u - off;
  const int t = off - kItemCost;
  w.tile = t <= snap_low(w.nt) ? 0 : t >= w.nt - snap_high(w.nt) ? w.nt : t;
  return w;
}

// A loading warp: the one that leads walks the block's range and queues its segments (an
// empty one at the end); each loads the tiles of every segment.  `issue(rows, box, none)`
// loads a tile: lane box + b's `rows` is the pool's row of the first position of its box b, or
// `none` (past the pool, so that the box reads as zeros) where no row of the item sees
// the box; false when it failed.  flush() after each segment.
template <int ROWS, class Issue, class Flush>
__device__ __forceinline__ void load_all(const Params& p, const Range& rg, bool lead,
                                         const Found* s_found, Segment* s_seg,
                                         uint32_t b_segFull, uint32_t b_segEmpty,
                                         volatile int* s_abort, Issue&& issue, Flush&& flush) {
  const int lane = threadIdx.x & 31;
  const int log_page = p.c.log_page, page = 1 << log_page;
  const int box_rows = min(page, kBN), n_boxes = kBN / box_rows;
  const int none = (int)(p.c.n_pages * p.c.Hkv) << log_page;
  Place w = {}, e = {};
  if (lead) {
#pragma unroll 1
    for (int k = 1; k >= 0; --k) {
      if (k == 1) {
        e.n = p.c.R;
        if (rg.last) continue;
      }
      w = locate<ROWS>(p, s_found[k], k ? rg.u1 : rg.u0);
      if (k == 1) e = w;
    }
  }
#pragma unroll 1
  for (int sn = 0;; ++sn) {
    const int ss = sn % kSegDepth;
    const uint32_t parity = (sn / kSegDepth) & 1;
    const bool ok = wait_bar((lead ? b_segEmpty : b_segFull) + 8 * ss, lead ? parity ^ 1 : parity,
                             s_abort);
    if (!__all_sync(0xffffffffu, ok)) return;
    Segment sg;
    if (lead) {
      auto at_e = [&]() { return w.n == e.n && w.qt == e.qt && w.h == e.h; };
      bool end = w.n >= p.c.R || (at_e() && w.tile >= e.tile);
      if (!end && w.tile >= w.nt) {
        next_item<ROWS>(p, w);
        end = w.n >= p.c.R || (at_e() && w.tile >= e.tile);
      }
      if (end) {
        sg.ntiles = 0;
      } else {
        const Item it = item_of(p, w.q, w.qt);
        const int nt = it.ntiles, stop = at_e() ? e.tile : nt;
        sg.n = w.n;
        sg.row0 = w.q.row0;
        sg.m = w.q.m;
        sg.ctx = w.q.ctx;
        sg.h = w.h;
        sg.r0 = it.r0;
        sg.nrows = it.nrows;
        sg.lo = it.lo;
        sg.hi = it.hi;
        sg.tile0 = it.tile0 + w.tile;
        sg.ntiles = stop - w.tile;
        sg.split = sg.first = sg.last = 0;
        if (sg.ntiles != nt) {
          sg.first = rg.block_of(w.a + kItemCost + snap_low(nt));
          sg.last = rg.block_of(w.a + kItemCost + nt - snap_high(nt) - 1);
          sg.split = (int)blockIdx.x == sg.first ? 2 : 1;
        }
        w.tile = stop;
        w.nt = nt;
      }
      if (lane == 0) {
        s_seg[ss] = sg;
        mbar_arrive(b_segFull + 8 * ss);
        if (sg.ntiles != 0 &&
            __ldg(p.c.row_off + sg.n + 1) - __ldg(p.c.row_off + sg.n) > p.max_rows)
          set_flag(p.c.status, kFlagRowRange);
      }
    } else {
      sg = s_seg[ss];
      __syncwarp();
      if (lane == 0) mbar_arrive(b_segEmpty + 8 * ss);
    }
    if (sg.ntiles == 0) return;
    // 32 boxes' rows a time, a box a lane; the next 32 in flight under the loads of these
    auto lookup = [&](int i) {
      const int pos = (sg.tile0 + i) * kBN + lane * box_rows;
      if (i + lane / n_boxes >= sg.ntiles || pos >= sg.hi || pos + box_rows <= sg.lo) return none;
      const int64_t id = page_of(p.c, sg.n, pos);
      return id < 0 ? none : (int)((id * p.c.Hkv + sg.h) << log_page) + (pos & (page - 1));
    };
    int rows = lookup(0), next = none;
#pragma unroll 1
    for (int i = 0, box = 0; i < sg.ntiles; ++i, box += n_boxes) {
      if (box == 32) {
        rows = next;
        box = 0;
      }
      if (box == 0 && i + 32 / n_boxes < sg.ntiles) next = lookup(i + 32 / n_boxes);
      if (!issue(rows, box, none)) return;
    }
    flush();
  }
}

// Joins the partial results of an item's blocks (the THREADS softmax threads, warps 0
// on, of the last one to finish).  `buf`, 32 KB of shared memory: the blocks' (m, l) of a
// group of rows, then their weights 2^(m - M) / L; the sums run over the blocks in
// order, eight values a thread.  About 3000 cycles for 32 rows of two or three blocks.
// kLanesOnRows: records hold O as [DP / 4][ROWS][4], else [ROWS][DP]; a warp's loads are
// contiguous either way.
template <int DP, int ROWS, int THREADS, bool kLanesOnRows>
__device__ __forceinline__ void join(const Params& p, const Segment& sg, float2* buf) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int np = sg.last - sg.first + 1;
  constexpr size_t rec = record_floats(ROWS, DP);
  const float* rec0 = p.part + ((size_t)sg.first * 2 + 1) * rec;  // the first block's, then
  const float* recs = p.part + ((size_t)sg.first * 2 + 2) * rec;  // two records a block on
  auto part = [&](int i) { return i == 0 ? rec0 : recs + (size_t)(i - 1) * 2 * rec; };
  const int group = min(sg.nrows, 4096 / np);
#pragma unroll 1
  for (int r0 = 0; r0 < sg.nrows; r0 += group) {
    const int g = min(group, sg.nrows - r0);
#pragma unroll 1
    for (int i = tid; i < np * g; i += THREADS) {
      const int b = i / g, row = i - b * g;
      buf[i] = __ldcg(reinterpret_cast<const float2*>(part(b) + (size_t)ROWS * DP) + r0 + row);
    }
    group_sync(1, THREADS);
#pragma unroll 1
    for (int row = warp; row < g; row += THREADS / 32) {
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
      if (lane == 0 && p.lse != nullptr)
        p.lse[out_row(p, sg.row0, sg.h, sg.r0 + r0 + row)] =
            L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
    group_sync(1, THREADS);
#pragma unroll 1
    for (int task = tid; task < g * (DP / 8); task += THREADS) {
      const int d8 = kLanesOnRows ? task / g : task % (DP / 8);
      const int row = kLanesOnRows ? task - d8 * g : task / (DP / 8);
      if (d8 * 8 >= p.c.D) continue;
      const size_t at = kLanesOnRows ? (size_t)d8 * 2 * ROWS + r0 + row
                                     : (size_t)(r0 + row) * (DP / 4) + d8 * 2;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 1
      for (int b0 = 0; b0 < np; b0 += 4) {
        float4 u[4], v[4];  // four blocks' loads in flight
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (b0 + i < np) {
            const float4* r = reinterpret_cast<const float4*>(part(b0 + i)) + at;
            u[i] = __ldcg(r);
            v[i] = __ldcg(r + (kLanesOnRows ? ROWS : 1));
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (b0 + i < np) {
            const float f = buf[(b0 + i) * g + row].x;
            x.x = fmaf(u[i].x, f, x.x);
            x.y = fmaf(u[i].y, f, x.y);
            x.z = fmaf(u[i].z, f, x.z);
            x.w = fmaf(u[i].w, f, x.w);
            y.x = fmaf(v[i].x, f, y.x);
            y.y = fmaf(v[i].y, f, y.y);
            y.z = fmaf(v[i].z, f, y.z);
            y.w = fmaf(v[i].w, f, y.w);
          }
      }
      *reinterpret_cast<uint4*>(p.out + out_row(p, sg.row0, sg.h, sg.r0 + r0 + row) * p.c.D +
                                d8 * 8) =
          make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y),
                     pack_bf16(y.z, y.w));
    }
    group_sync(1, THREADS);
  }
}

// After a block wrote its part of a split item (all softmax threads): the last of
// the item's blocks joins.  s_last is a word of shared memory, buf 32 KB.
template <int DP, int ROWS, int THREADS, bool kLanesOnRows>
__device__ __forceinline__ void finish_split(const Params& p, const Segment& sg,
                                             volatile int* s_last, float2* buf) {
  __threadfence();
  group_sync(1, THREADS);
  if (threadIdx.x == 0) {
    const unsigned want = (unsigned)(sg.last - sg.first);
    const unsigned old = atomicAdd(p.counters + sg.first, 1u);
    *s_last = old == want;
    if (old == want) p.counters[sg.first] = 0;
  }
  group_sync(1, THREADS);
  if (*s_last) {
    __threadfence();
    join<DP, ROWS, THREADS, kLanesOnRows>(p, sg, buf);
  }
}

}  // namespace attend

// The kernels' launchers (attend_few.cu, attend_many.cu).
cudaError_t launch_attend_few(const AttendArgs& a, const attend::Params& p, cudaStream_t st);
cudaError_t launch_attend_many(const AttendArgs& a, const attend::Params& p, cudaStream_t st);

}  // namespace dspark
