// Attention of many packed rows a head (prompt chunks, large groups) over the paged
// cache.
//
// With S = Q K^T over a tile of 128 positions, and a reference m of each row's
// running maximum:
//
//   P = 2^(c S - c m),  l = l + sum P,  O = O + P V      (c = scale * log2 e)
//
// and out = O / l, lse = (c m + log2 l) ln 2 at the end.  m moves only when the
// maximum has grown by more than 8 powers of two (O and l are then rescaled):
// any reference gives the same quotient, and fp32 has the range.  P enters its
// product as two bf16 terms, its rounding and the rounding of the rest (16
// significant bits in all): a row that a few positions dominate would otherwise
// carry their rounding straight into the result.
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
// e4m3 caches: eight more warps turn the codes into bf16 tiles, scaled (exact: the
// scales are powers of two), between the loads and the products.
//
// Roles: warps 0-7 the two softmax warpgroups (they also load Q and store), warp 8
// issues the MMAs, warps 9 and 10 the TMA loads of K and V (11 completes the
// warpgroup), warps 12-19 convert.  Every wait is bounded; a timeout sets
// DSPARK_DEVFLAG_TIMEOUT and ends the kernel.  See attend.cuh for the split of the work.
//
// What bounds it: a stream's chain of scores (8 MMAs of 96 cycles: both operands come
// from shared memory), softmax and P V (16 of 64, P from tensor memory), of which
// the softmax is the longest: 256 rows by 128 positions take about 5200 cycles, their
// MMAs 3600 of those.
// The softmax in loops of 32 positions, read twice, is what the instruction caches
// hold: unrolled over the tile, with a copy for each number of row copies, the chunks
// below took 515 us for 478 (alone in a graph, at the time); loops of 16 took 499, loads
// one chunk ahead 507, two threads a row 542.
// Measured (32 query heads over 8 of 128), among other calls: two chunks of 2000 rows
// after 1000 to 7000 positions 491 us, 913 TFLOP/s of visible products (47% of the
// measured matrix rate; alone in a graph 475 us); three of 700 to 1500, 40 heads, window
// 2048, e4m3 223 us, 491 TFLOP/s: tiles at the edges of the windows are computed whole,
// an item has a dozen tiles, and every row tile converts its K and V again (four warps
// for it: 6 us more).
#include "attend.cuh"

namespace dspark {

namespace {

using namespace attend;

constexpr int kRows = 256;
constexpr int kSoftThreads = 256;  // the two softmax warpgroups, warps 0-7
constexpr int kWarpMma = 8;
constexpr int kWarpTma = 9;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;  // S at 0 and 128, O at 256 and 256 + DP
constexpr float kGrow = 8.0f;    // log2 growth of a maximum that moves the reference

template <int DP, bool E4M3>
struct Many {
  static constexpr int kThreads = E4M3 ? 640 : 384;
  static constexpr uint32_t kTile = kHalf * (DP / 64);  // a K, V or Q tile of bf16
  // Q of both streams; at an item's end 32 KB to join through and the streams' (m, l)
  static constexpr uint32_t kXch = 32768;
  static constexpr uint32_t kQBytes = 2 * kTile > kXch + 2048 ? 2 * kTile : kXch + 2048;
  static constexpr uint32_t kMisc = 1024;
  static constexpr int kRawSlots = E4M3 ? 4 : 0;        // tiles of codes
  static constexpr uint32_t kRaw = kRawSlots * (kHalf + 128);
  static constexpr int kFit = (int)((kMaxSmem - kQBytes - kMisc - kRaw) / kTile);
  static constexpr int kSlots = kFit > 12 ? 12 : kFit;
  static constexpr uint32_t kQOff = kSlots * kTile;
  static constexpr uint32_t kRawOff = kQOff + kQBytes;
  static constexpr uint32_t kExpOff = kRawOff + kRawSlots * kHalf;
  static constexpr uint32_t kMiscOff = kRawOff + kRaw;
  static constexpr uint32_t kTotal = kMiscOff + kMisc;
  static_assert(kTotal <= kMaxSmem && kSlots >= 3, "shared memory");
};

struct Misc {  // shared words
  int64_t sum[32];
  Found found[2];
  Segment seg[kSegDepth];
  uint64_t bars[2 * 12 + 2 * 4 + 2 * kSegDepth + 8];
  int abort_flag, last;
  uint32_t tmem;
  uint32_t issued[2];  // where each loading warp stopped: its next ring entry
};
static_assert(sizeof(Misc) <= 1024, "shared words");

// The last entry of a ring of n slots that was loaded into slot i, where the even entries
// (K) below k and the odd ones (V) below v were issued; none: a negative number.  In a ring
// of an odd number of slots K and V take turns in each.
__host__ __device__ constexpr int last_entry(int i, int n, int k, int v) {
  const int top = k > v ? k : v;
  int e = i + (top - i + n - 1) / n * n;
  while (e >= 0 && e >= (e & 1 ? v : k)) e -= n;
  return e;
}
static_assert(last_entry(0, 5, 0, 1) < 0 && last_entry(0, 5, 2, 1) == 0, "");
static_assert(last_entry(1, 5, 8, 7) == 6 && last_entry(1, 5, 6, 7) == 1, "K in V's slot or not");
static_assert(last_entry(4, 5, 10, 7) == 4 && last_entry(3, 5, 10, 9) == 8, "");
static_assert(last_entry(2, 12, 40, 27) == 38 && last_entry(3, 12, 40, 27) == 15, "");

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
      m[k] = max3(m[k], __uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1]));
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

// One tile's P for a warp: its rows' scores of nc * 32 positions from column col0
// of S on, the running reference and sum, and P over S's columns (zero outside
// the warp's own positions).  Loops of 32 positions at a time, read twice: the code
// of all roles' loops has to stay in the instruction caches.
template <int DP>
__device__ __forceinline__ void softmax_tile(uint32_t t_s, uint32_t t_o, int col0, int nc,
                                             bool mask, int rel_lo, int rel_hi, float c2, bool first,
                                             float& m_ref, float& l) {
  const int end = col0 + 32 * nc;
  float top = -INFINITY;
#pragma unroll 1
  for (int c = col0; c < end; c += 32) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(t_s + c, v);
    tmem_wait_ld_regs(v);
    if (mask) {
      mask_chunk(v, c, rel_lo, rel_hi);
      tmem_st_32x32b_x32(t_s + c, v);
    }
    top = max_chunk(v, top);
  }
  if (mask) tmem_wait_st();
  if (first) {
    m_ref = top;
  } else if (__any_sync(0xffffffffu, (top - m_ref) * c2 > kGrow)) {
    float f = 1.f;
    if (top > m_ref) {
      f = ex2_approx((m_ref - top) * c2);
      m_ref = top;
    }
    l *= f;
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
#pragma unroll 1
  for (int c = col0; c < end; c += 32) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(t_s + c, v);
    tmem_wait_ld_regs(v);
    exp_chunk(v, t_s + c, c2, mc, sum);
  }
  if (nc < 4) {
    uint32_t z[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) z[i] = 0;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32)
      if (c < col0 || c >= end) tmem_st_32x32b_x32(t_s + c, z);
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

template <int DP, bool E4M3>
__global__ void __launch_bounds__(Many<DP, E4M3>::kThreads, 1)
    attend_many_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  using F = Many<DP, E4M3>;
  constexpr int NS = F::kSlots, NH = DP / 64, NRAW = E4M3 ? F::kRawSlots : 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* s_kv = smem;
  uint8_t* s_q = smem + F::kQOff;
  float2* s_xch = reinterpret_cast<float2*>(s_q + F::kXch);
  Misc* ms = reinterpret_cast<Misc*>(smem + F::kMiscOff);
  const uint32_t b_full = smem_u32(ms->bars), b_empty = b_full + 8 * NS;
  const uint32_t b_segFull = b_empty + 8 * NS, b_segEmpty = b_segFull + 8 * kSegDepth;
  const uint32_t b_q = b_segEmpty + 8 * kSegDepth;
  const uint32_t b_s = b_q + 8, b_p = b_s + 16, b_o = b_p + 16, b_drain = b_o + 16;
  const uint32_t b_rawFull = b_drain + 8, b_rawEmpty = b_rawFull + 8 * F::kRawSlots;
  volatile int* s_abort = &ms->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem) & 1023) return;  // never: the declared alignment, which the swizzle needs

  if (tid == 0) {
    *s_abort = 0;
#pragma unroll 1
    for (int i = 0; i < NS; ++i) {
      mbar_init(b_full + 8 * i, E4M3 ? 8 : 1);
      mbar_init(b_empty + 8 * i, 1);
    }
    for (int i = 0; i < F::kRawSlots; ++i) {
      mbar_init(b_rawFull + 8 * i, 33);  // the load, and 32 lanes' exponent bytes
      mbar_init(b_rawEmpty + 8 * i, 1);
    }
    for (int i = 0; i < kSegDepth; ++i) {
      mbar_init(b_segFull + 8 * i, 1);
      mbar_init(b_segEmpty + 8 * i, E4M3 ? 18 : 10);  // the MMA thread and the other warps
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
  grid_dependency_wait();  // row_off, ctx, the pages
  const Range rg = plan<kRows, F::kThreads>(p, ms->sum, ms->found);
  if (rg.u0 >= rg.u1) return;  // no tiles for this block
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(&ms->tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem;

  // bf16: 384 threads of 168 registers become 256 x 208 and 128 x 88;
  // e4m3: 640 of 96 become 256 x 128 and 384 x 72
  if (warp == kWarpTma || warp == kWarpTma + 1) {
    if (E4M3) reg_dec<72>();
    else reg_dec<88>();
    // ------------------------------------------------------------ loads
    const int kv = warp - kWarpTma;  // warp 9 K, warp 10 V
    const CUtensorMap* map = kv ? &tm_v : &tm_k;
    const uint8_t* exps = kv ? p.c.v_exp : p.c.k_exp;
    const int box_rows = min(1 << p.c.log_page, kBN), n_boxes = kBN / box_rows;
    if (lane == 0) tma_prefetch(map);
    constexpr uint32_t kRing = E4M3 ? NRAW : NS;
    const uint32_t full0 = E4M3 ? b_rawFull : b_full, empty0 = E4M3 ? b_rawEmpty : b_empty;
    uint32_t e = kv;  // ring entries: K and V of each tile in turn
    // e4m3: four positions' exponent bytes a lane, stored with the next tile's load
    const int my_box = lane * 4 / box_rows, my_at = lane * 4 % box_rows;
    uint32_t held = 0, stored = kv;  // entries whose bytes are stored
    auto flush = [&]() {
      if (!E4M3 || stored >= e) return;
      const uint32_t slot = stored % kRing;
      reinterpret_cast<uint32_t*>(smem + F::kExpOff + slot * 128)[lane] = held;
      mbar_arrive(full0 + 8 * slot);
      stored += 2;
    };
    auto issue = [&](int rows, int box, int none) {
      if constexpr (E4M3) {
        const int row = __shfl_sync(0xffffffffu, rows, box + my_box);
        uint32_t now = 0x7f7f7f7fu;
        if (row != none) now = __ldg(reinterpret_cast<const uint32_t*>(exps + row + my_at));
        flush();
        held = now;
      }
      const uint32_t slot = e % kRing, full = full0 + 8 * slot;
      const bool ok = wait_bar(empty0 + 8 * slot, ((e / kRing) & 1) ^ 1, s_abort);
      if (!__all_sync(0xffffffffu, ok)) return false;
      uint32_t dst = E4M3 ? smem_u32(smem + F::kRawOff) + slot * kHalf
                          : smem_u32(s_kv) + slot * F::kTile;
      int y[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) y[b] = __shfl_sync(0xffffffffu, rows, box + b);
      if (elect_one()) {
        mbar_arrive_expect_tx(full, E4M3 ? kHalf : F::kTile);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          if (b >= n_boxes) break;
          tma_load_2d(dst, map, full, 0, y[b]);
          if (!E4M3 && NH > 1) tma_load_2d(dst + kHalf, map, full, 64, y[b]);
          dst += box_rows * 128;
        }
      }
      __syncwarp();
      e += 2;
      return true;
    };
    load_all<kRows>(p, rg, kv == 0, ms->found, ms->seg, b_segFull, b_segEmpty, s_abort, issue,
                    flush);
    ms->issued[kv] = e;
  } else if (warp == kWarpMma) {
    if (E4M3) reg_dec<72>();
    else reg_dec<88>();
    // ------------------------------------------------------------ products
    if (elect_one()) {
      constexpr uint32_t kIdS = idesc_bf16_f32(128, kBN);
      constexpr uint32_t kIdO = idesc_bf16_f32(128, DP) | kIdescTransposeB;
      const int ksteps = p.c.D / 16;
      const uint32_t q_at = smem_u32(s_q), kv_at = smem_u32(s_kv);
      uint32_t base = 0;  // tiles of the segments before
      uint32_t ph_q = 0, ph_p = 0;
      bool ok = true;
      auto need = [&](uint32_t e) {
        ok = ok && wait_bar(b_full + 8 * (e % NS), (e / NS) & 1, s_abort);
        tc_fence_after();
      };
      auto need_p = [&](int s) {
        ok = ok && wait_bar(b_p + 8 * s, (ph_p >> s) & 1, s_abort);
        ph_p ^= 1u << s;
        tc_fence_after();
      };
      auto scores = [&](int s, int qtile, uint32_t e) {
        const uint64_t a = desc_kmajor_sw128(q_at + qtile * F::kTile);
        const uint64_t b = desc_kmajor_sw128(kv_at + (e % NS) * F::kTile);
        for (int k = 0; k < ksteps; ++k) {
          const uint32_t at = (k >> 2) * (kHalf >> 4) + (k & 3) * 2;
          mma_bf16(tmem + s * kBN, a + at, b + at, kIdS, k > 0);
        }
        mma_commit(b_s + 8 * s);
      };
      auto values = [&](int s, uint32_t e, bool acc) {
        // 16 positions a step: 2048 bytes on (the sum stays within the 14 address bits)
        const uint64_t v = desc_mnmajor_sw128(kv_at + (e % NS) * F::kTile, kHalf);
#pragma unroll 1
        for (int k = 0; k < kBN / 16; ++k) {
          const uint32_t a = tmem + s * kBN + (k >> 1) * 32 + (k & 1) * 8;
          mma_bf16_ts(tmem + kColO + s * DP, a, v + k * (2048 >> 4), kIdO, acc || k > 0);
          mma_bf16_ts(tmem + kColO + s * DP, a + 16, v + k * (2048 >> 4), kIdO, 1);
        }
      };
      auto release = [&](uint32_t e) { mma_commit(b_empty + 8 * (e % NS)); };
      for (int sn = 0; ok; ++sn) {
        const int ss = sn % kSegDepth;
        ok = wait_bar(b_segFull + 8 * ss, (sn / kSegDepth) & 1, s_abort);
        if (!ok) break;
        const int nt = ms->seg[ss].ntiles;
        const bool two = ms->seg[ss].nrows > 128;
        mbar_arrive(b_segEmpty + 8 * ss);
        if (nt == 0) break;
        ok = wait_bar(b_q, ph_q, s_abort);
        if (!ok) break;
        ph_q ^= 1;
        tc_fence_after();
        const uint32_t e0 = 2 * base;  // K of tile i: e0 + 2 i, V: one more
        if (two) {
          need(e0);
          if (!ok) break;
          scores(0, 0, e0);
          scores(1, 1, e0);
          release(e0);
          for (int i = 0; i < nt && ok; ++i) {
            const uint32_t ev = e0 + 2 * i + 1, ek = ev + 1;
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
            const uint32_t ev = e0 + 2 * i + 1;
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
  } else if (warp < 8) {
    if (E4M3) reg_inc<128>();
    else reg_inc<208>();
    // ------------------------------------------------------------ softmax
    const int s = warp >> 2;  // the stream
    const int lrow = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + s * kBN, t_o = tmem + lanes + kColO + s * DP;
    const float c2 = p.scale * kLog2e;
    uint32_t ph_s = 0, ph_o = 0;
    uint32_t base = 0;
    for (int sn = 0;; ++sn) {
      const int ss = sn % kSegDepth;
      const bool got = wait_bar(b_segFull + 8 * ss, (sn / kSegDepth) & 1, s_abort);
      // all leave together; the barrier also ends the previous segment's use of s_q
      if (group_any(1, kSoftThreads, !got)) break;
      const Segment sg = ms->seg[ss];
      __syncwarp();
      if (lane == 0) mbar_arrive(b_segEmpty + 8 * ss);
      if (sg.ntiles == 0) break;
      const bool two = sg.nrows > 128;
      const int rep = two || sg.nrows > 64 ? 1 : sg.nrows > 32 ? 2 : 4;
      const int rp = 128 / rep;  // rows of a copy

      // Q: rows past the item's are zero; eight loads in flight
      {
        uint8_t* dst = s_q + (two ? s * F::kTile : 0);
        const int r_first = sg.r0 + (two ? s * 128 : 0), r_end = sg.r0 + sg.nrows;
        const int threads = two ? 128 : 256;
#pragma unroll 1
        for (int i0 = two ? lrow : tid; i0 < 128 * (DP / 8); i0 += 8 * threads) {
          uint4 x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * threads, r = r_first + (i / (DP / 8)) % rp;
            x[k] = make_uint4(0, 0, 0, 0);
            if (i < 128 * (DP / 8) && r < r_end)
              x[k] = load_q(p, sg.row0, sg.h, r, i % (DP / 8) * 8);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * threads, row = i / (DP / 8), ch = i % (DP / 8);
            if (i < 128 * (DP / 8))
              *reinterpret_cast<uint4*>(dst + (ch >> 3) * kHalf + row * 128 +
                                        (((ch & 7) ^ (row & 7)) << 4)) = x[k];
          }
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
      const int col0 = ((warp & 3) * rep >> 2) * (kBN / rep);  // this copy's positions

      float m_ref = -INFINITY, l = 0.f;
      const int step = two ? 1 : 2, i0 = two ? 0 : s;
      for (int i = i0; i < sg.ntiles; i += step) {
        const int t0 = (sg.tile0 + i) * kBN;
        wait_bar(b_s + 8 * s, ph_s, s_abort);
        __syncwarp();
        ph_s ^= 1;
        tc_fence_after();
        const bool mask = t0 < max_lo || t0 + kBN > min_hi;
        const bool first = i == i0;
        const int rel_lo = row_lo - t0, rel_hi = row_hi - t0;
        softmax_tile<DP>(t_s, t_o, col0, 4 / rep, mask, rel_lo, rel_hi, c2, first, m_ref, l);
        // (e4m3: the conversion has zeroed them)
        if (!E4M3 && (!two || s == 0) && (t0 < sg.lo || t0 + kBN > sg.hi)) {
          const uint32_t e = 2 * (base + i) + 1, slot = e % NS;
          wait_bar(b_full + 8 * slot, (e / NS) & 1, s_abort);
          uint8_t* tile = s_kv + slot * F::kTile;
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
        wait_bar(b_o + 8 * s, ph_o, s_abort);
        __syncwarp();
        ph_o ^= 1;
        tc_fence_after();
      }
      base += sg.ntiles;

      float* rec = p.part +
                   ((size_t)blockIdx.x * 2 + (sg.split == 2 ? 1 : 0)) * record_floats(kRows, DP);
      const float mine = m_ref == -INFINITY ? -INFINITY : m_ref * c2;
      if (two) {
        const int64_t at = out_row(p, sg.row0, sg.h, sg.r0 + my);
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int ch = 0; ch < DP; ch += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(t_o + ch, o);
          tmem_wait_ld_regs(o);
          if (live && !sg.split) {
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
          if (sg.split)
            __stcg(reinterpret_cast<float2*>(rec + (size_t)kRows * DP) + my, make_float2(mine, l));
          else if (p.lse != nullptr)
            p.lse[at] = l == 0.f ? -INFINITY : (mine + log2f(l)) * kLn2;
        }
      } else {
        // the copies of a row in the streams: a common reference first
        const int parts = sg.ntiles > 1 ? 2 * rep : rep;
        s_xch[tid] = make_float2(mine, l);
        group_sync(1, kSoftThreads);
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
        group_sync(1, kSoftThreads);
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
          group_sync(1, kSoftThreads);
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
            if (sg.split) {
              __stcg(reinterpret_cast<float4*>(rec) + (size_t)(ch / 4 + d4) * kRows + row, x);
            } else if (ch + d4 * 4 < p.c.D) {
              const float Lr = s_xch[row].y;
              const float inv = Lr == 0.f ? 0.f : 1.f / Lr;
              const int64_t at = out_row(p, sg.row0, sg.h, sg.r0 + row);
              *reinterpret_cast<uint2*>(p.out + at * p.c.D + ch + d4 * 4) =
                  make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
            }
          }
          group_sync(1, kSoftThreads);
        }
        if (tid < sg.nrows) {
          if (sg.split) {
            __stcg(reinterpret_cast<float2*>(rec + (size_t)kRows * DP) + tid, make_float2(M, L));
          } else if (p.lse != nullptr) {
            p.lse[out_row(p, sg.row0, sg.h, sg.r0 + tid)] =
                L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
          }
        }
      }
      if (sg.split)
        finish_split<DP, kRows, kSoftThreads, true>(p, sg, &ms->last, reinterpret_cast<float2*>(s_q));
      tc_fence_before();
    }
  } else if (warp < 12) {
    if (E4M3) reg_dec<72>();
    else reg_dec<88>();  // completes the warpgroup
  } else if (E4M3) {
    reg_dec<72>();
    // ------------------------------------------------------------ codes to bf16
    const int ct = tid - 384;
    const Converter<DP, 8> convert(ct >> 5, lane);
    uint32_t e = 0;
    for (int sn = 0;; ++sn) {
      const int ss = sn % kSegDepth;
      const bool got = wait_bar(b_segFull + 8 * ss, (sn / kSegDepth) & 1, s_abort);
      if (group_any(4, 256, !got)) break;
      const int nt = ms->seg[ss].ntiles, tile0 = ms->seg[ss].tile0;
      const int lo = ms->seg[ss].lo, hi = ms->seg[ss].hi;
      __syncwarp();
      if (lane == 0) mbar_arrive(b_segEmpty + 8 * ss);
      if (nt == 0) break;
#pragma unroll 1
      for (int i = 0; i < 2 * nt; ++i, ++e) {
        const uint32_t raw = e % NRAW, slot = e % NS;
        const int t0 = (tile0 + (i >> 1)) * kBN;
        wait_bar(b_rawFull + 8 * raw, (e / NRAW) & 1, s_abort);
        wait_bar(b_empty + 8 * slot, ((e / NS) & 1) ^ 1, s_abort);
        convert(smem + F::kRawOff + raw * kHalf, smem + F::kExpOff + raw * 128,
                s_kv + slot * F::kTile, lo - t0, hi - t0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_full + 8 * slot);
        group_sync(4, 256);
        if (ct == 0) mbar_arrive(b_rawEmpty + 8 * raw);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *s_abort) {
    set_flag(p.c.status, kFlagWaitTimeout);
    // the copies in flight land before the block's shared memory goes
    constexpr int kRing = E4M3 ? NRAW : NS;
    for (int i = 0; i < kRing; ++i) {
      const int e = last_entry(i, kRing, (int)ms->issued[0], (int)ms->issued[1]);
      if (e >= 0) mbar_wait((E4M3 ? b_rawFull : b_full) + 8 * i, (e / kRing) & 1);
    }
  }
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int DP, bool E4M3>
cudaError_t launch_one(const AttendArgs& a, const Params& p, cudaStream_t st) {
  using F = Many<DP, E4M3>;
  auto kernel = attend_many_kernel<DP, E4M3>;
  cudaError_t e = ensure_smem_attr((const void*)kernel, F::kTotal);
  if (e != cudaSuccess) return e;
  const int grid = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
  DSPARK_LAUNCH(kKindAttend, st,
                e = launch_pdl(kernel, dim3(grid), dim3(F::kThreads), F::kTotal, st, a.desc->tm_k,
                               a.desc->tm_v, p));
  return e;
}

}  // namespace

cudaError_t launch_attend_many(const AttendArgs& a, const attend::Params& p, cudaStream_t st) {
  const bool e4m3 = p.c.k_exp != nullptr;
  if (p.c.D > 64) return e4m3 ? launch_one<128, true>(a, p, st) : launch_one<128, false>(a, p, st);
  return e4m3 ? launch_one<64, true>(a, p, st) : launch_one<64, false>(a, p, st);
}

}  // namespace dspark
