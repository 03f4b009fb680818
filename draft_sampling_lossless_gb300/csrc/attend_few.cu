// Attention of up to 32 packed rows a head (single tokens, verified blocks) over
// the paged cache.
//
// HBM bounds it: a position's key and value (512 bytes of bf16 at D = 128) meet
// 32 rows at most, far below the tensor cores' 284 operations a byte.  What is left
// is to keep up with the loads, so both products are turned over, with the
// positions or D as the 128 MMA rows and the few packed rows as N:
//
//   S^T = K Q^T    (128 positions x rows),   O^T = V^T P^T   (D x rows)
//
// A softmax thread is a position: it has that position's scores of all rows and
// sums its own exponentials, joined over the positions once, at the end.
// P = 2^(s - m) against a reference m of each row, the maximum of the first tile of
// the row's part.  Any reference gives the same quotient as long as P stays in
// range; where a score passes it by 24 powers of two, the row's reference moves to the
// tile's maximum, O and the sum with it.
// (24 and not the 64 that sums of P alone would allow: a value up to 2^80 times such a P
// still leaves O finite over 2^24 positions.)
//
// P enters its product as two bf16 terms, its rounding and the rounding of the rest
// (columns of N side by side): 16 bits of it however small it is.  A row that one position
// dominates would otherwise carry that rounding straight into the result, and a long
// context beside one dominant position is a sum of small P.
//
// e4m3: K's codes are multiplied as they are stored.  Q comes as two e4m3 terms,
// q 2^-a = q1 + q2 / 16, which hold a bf16's eight bits exactly (down to 2^-13 of the row's
// largest; below, to 2^-21 of it); a position's scale is its thread's own, a factor of
// the scores.  V's codes become bf16 on the way, scales and all (exact).  P as e4m3 terms
// over V's codes (four of them) was as fast over 32 rows and took 124 us for 256 single
// tokens instead of 147, but its range ends at 2^-22 of the reference: what lies below was
// in l and not in O.
//
// Two streams, each a warpgroup with its own P, O and m, take alternate tiles.
// Roles: warps 0-7 softmax, one warp issues the MMAs of the scores (as many tiles ahead
// as S has buffers, over the ends of items too), two load K and V through a ring each,
// one fetches the next item's Q and the scales, one issues the MMAs of O; e4m3: eight
// convert V into a ring of three tiles (four warps: 184 us for single tokens; two tiles:
// 159).  One thread for both products was not enough: its MMAs (64 cycles each), commits
// and waits took as long as a tile of e4m3 does (8 verified rows of bf16: 191 us, with two
// 184, at the time).
// What a tile costs besides the loads is fetching instructions: with the loops over
// rows unrolled, the blocks' roles asked for more than the instruction caches give
// (23% of the fetches missed the SM's, the next level ran at 90% of its rate), and
// that, not the arithmetic, set the pace.  Every wait is bounded.  See attend.cuh for
// the split of the work.
//
// Measured among other calls (32 query heads over 8 of 128, of the measured copy rate):
//   64 requests of 1 to 8 rows, 500 to 8000 positions  181 us, 6.3 TB/s, 93%
//   3 of 5 to 8 rows, 90 to 180 thousand positions     224 us, 6.7 TB/s, 99%
//   the first, e4m3: 182 us, 3.3 TB/s, 48%; 256 single tokens, e4m3: 147 us, 3.9 TB/s,
//     57%: the softmax threads' chains of instructions, which the converting warps'
//     instructions stretch (58% of the issue slots are taken)
//   64 drafter's blocks of 7 rows, 16 heads over 8 of 64: 59 us, 4.9 TB/s, 73%: the
//     ends of items
//   one token, 700 positions: 10.5 us, latency: the plan of the work (2 us), the first
//     loads (2 us), six tiles, the join
#include "attend.cuh"

namespace dspark {

namespace {

using namespace attend;

constexpr float kUnset = 3.0e38f;     // -m of a row that has seen nothing
constexpr int kExpDepth = 8;          // tiles of exponent bytes held

template <int DP, int NR, bool E4M3>
struct Few {
  static constexpr int kSoft = 256;  // softmax threads, two warpgroups; then five warps
  static constexpr int kWarpS = kSoft / 32, kWarpTma = kWarpS + 1, kWarpO = kWarpS + 4;
  static constexpr int kConv = E4M3 ? 8 : 0;  // warps that convert V
  static constexpr int kThreads = kSoft + 160 + 32 * kConv;
  static constexpr int kNH = DP / 64;
  static constexpr int kPN = 2 * NR;                                  // N of the products
  static constexpr int kQRows = E4M3 ? 2 * NR : (NR < 16 ? 16 : NR);  // N of the scores
  static constexpr int kSBufs = 4;  // tiles of scores ahead
  // tensor memory: S, 64 columns each, then O of the streams, then the positions' own
  // sums, l
  static constexpr uint32_t kColO = 64 * kSBufs, kOCols = 64;
  static constexpr uint32_t kColL = kColO + 2 * kOCols;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kTile = kHalf * kNH;                      // a tile of bf16
  static constexpr uint32_t kSlot = E4M3 ? kHalf : kTile;             // a tile as loaded
  static constexpr int kConvSlots = E4M3 ? (kNH > 1 ? 3 : 4) : 0;     // tiles converted
  static constexpr uint32_t kQHalf = kQRows * 128;
  static constexpr uint32_t kQBytes = kQHalf * (E4M3 ? 1 : kNH);
  static constexpr uint32_t kExp = E4M3 ? kExpDepth * 256 : 0;
  static constexpr uint32_t kMisc = 4096;
  static constexpr int kFit =
      (int)((kMaxSmem - 2 * kHalf - kConvSlots * kTile - 2 * kQBytes - kExp - kMisc) / kSlot);
  static constexpr int kSlots = kFit > 12 ? 12 : kFit;
  static constexpr int kSlotsK = kSlots / 2, kSlotsV = kSlots - kSlotsK;
  // P of each stream (at an item's end its O, then the join's buffer)
  static constexpr uint32_t kPOff = kSlots * kSlot;
  static constexpr uint32_t kConvOff = kPOff + 2 * kHalf;
  static constexpr uint32_t kQOff = kConvOff + kConvSlots * kTile;
  static constexpr uint32_t kExpOff = kQOff + 2 * kQBytes;
  static constexpr uint32_t kMiscOff = kExpOff + kExp;
  static constexpr uint32_t kTotal = kMiscOff + kMisc;
  static_assert(kTotal <= kMaxSmem && kSlots >= 4, "shared memory");
};

struct Misc {  // shared words
  float nm[2][32];      // -m of each stream's rows
  float f[2][32];       // what a move of the references multiplies by
  float wm[2][4][32];   // the warps' maxima, then sums
  float a[2][32];       // e4m3: scale of the scores of a row, of each Q buffer
  int64_t sum[32];
  Found found[2];
  Segment seg[kSegDepth];
  uint64_t bars[2 * 12 + 2 * kSegDepth + 4 + 8 + 4 + 2 * kExpDepth + 2 * 4 + 2];
  int abort_flag, last;
  uint32_t tmem;
};
static_assert(sizeof(Misc) <= 4096, "shared words");

// Reduces v[r] over a warp's lanes; row r's result lands in lanes r * 32 / NR on.
template <int NR, class Op>
__device__ __forceinline__ float reduce_rows(float (&v)[NR], Op op) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int half = NR / 2; half >= 1; half >>= 1, o >>= 1) {
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const bool up = lane & o;
      const float keep = up ? v[i + half] : v[i], send = up ? v[i] : v[i + half];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
#pragma unroll
  for (; o >= 1; o >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}

template <int DP, int NR, bool E4M3>
__global__ void __launch_bounds__(Few<DP, NR, E4M3>::kThreads, 1)
    attend_few_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  using F = Few<DP, NR, E4M3>;
  constexpr int NS = F::kSlots, NK = F::kSlotsK, NV = F::kSlotsV, NH = F::kNH, SB = F::kSBufs;
  // V as it is multiplied: as loaded, or converted
  constexpr int NM = E4M3 ? F::kConvSlots : NV;
  constexpr uint32_t kVOff = E4M3 ? F::kConvOff : NK * F::kSlot;
  // P's largest exponent; rows above half of it move along with one that passed it
  constexpr float kLimit = 24.f;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc* ms = reinterpret_cast<Misc*>(smem + F::kMiscOff);
  const uint32_t b_full = smem_u32(ms->bars), b_empty = b_full + 8 * NS;
  const uint32_t b_segFull = b_empty + 8 * NS, b_segEmpty = b_segFull + 8 * kSegDepth;
  const uint32_t b_qFull = b_segEmpty + 8 * kSegDepth, b_qEmpty = b_qFull + 16;
  const uint32_t b_s = b_qEmpty + 16, b_sFree = b_s + 32, b_p = b_sFree + 32, b_o = b_p + 16;
  const uint32_t b_expFull = b_o + 16, b_expEmpty = b_expFull + 8 * kExpDepth;
  const uint32_t b_conv = b_expEmpty + 8 * kExpDepth, b_convFree = b_conv + 8 * F::kConvSlots;
  const uint32_t b_drain = b_convFree + 8 * F::kConvSlots;
  // V's tiles: ready for the product, and no longer read by it
  const uint32_t b_v = E4M3 ? b_conv : b_full + 8 * NK;
  const uint32_t b_vFree = E4M3 ? b_convFree : b_empty + 8 * NK;
  volatile int* s_abort = &ms->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem) & 1023) return;  // never: the declared alignment, which the swizzle needs

  // a barrier a thread: its address is that of its place, its count its role's
  if (warp == F::kWarpS) {
    for (uint32_t bar = b_full + 8 * lane; bar <= b_drain + 8; bar += 8 * 32) {
      uint32_t n = 1;
      if (E4M3 && bar >= b_empty + 8 * NK && bar < b_segFull) n = F::kConv;
      else if (bar >= b_segEmpty && bar < b_qFull)
        n = 4 + F::kConv + F::kSoft / 32;  // all but the warp that fills
      else if (bar >= b_qFull && bar < b_qEmpty) n = 32;
      else if (E4M3 && bar >= b_qEmpty && bar < b_s) n = 1 + F::kSoft / 32;  // a's readers
      else if (bar >= b_sFree && bar < b_o) n = F::kSoft / 64;  // a stream's warps
      else if (bar >= b_expFull && bar < b_expEmpty) n = 32;
      else if (bar >= b_expEmpty && bar < b_conv) n = F::kSoft / 64 + F::kConv;
      else if (bar >= b_conv && bar < b_convFree) n = F::kConv;
      mbar_init(bar, n);
    }
    if (lane == 0) *s_abort = 0;
    fence_mbar_init();
    tmem_alloc(smem_u32(&ms->tmem), F::kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  grid_dependency_wait();  // row_off, ctx, the pages
  const Range rg = plan<32, F::kThreads>(p, ms->sum, ms->found);
  tc_fence_after();
  const uint32_t tmem = ms->tmem;
  if (rg.u0 >= rg.u1) {  // no tiles for this block
    if (warp == F::kWarpS) tmem_dealloc(tmem, F::kTmemCols);
    return;
  }

  if (warp == F::kWarpTma || warp == F::kWarpTma + 1) {
    // ------------------------------------------------------------ loads
    const int kv = warp - F::kWarpTma;  // the first K, the second V
    const CUtensorMap* map = kv ? &tm_v : &tm_k;
    const int box_rows = min(1 << p.c.log_page, kBN), n_boxes = kBN / box_rows;
    if (lane == 0) tma_prefetch(map);
    const int slots = kv ? NV : NK, slot0 = kv ? NK : 0;  // its ring
    uint32_t at = 0, tiles = 0, parity = 1;
    auto issue = [&](int rows, int box, int) {
      const uint32_t slot = slot0 + at, full = b_full + 8 * slot;
      const bool ok = wait_bar(b_empty + 8 * slot, parity, s_abort);
      if (!__all_sync(0xffffffffu, ok)) return false;
      uint32_t dst = smem_u32(smem) + slot * F::kSlot;
      int y[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) y[b] = __shfl_sync(0xffffffffu, rows, box + b);
      if (elect_one()) {
        mbar_arrive_expect_tx(full, F::kSlot);
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          if (b >= n_boxes) break;
          tma_load_2d(dst, map, full, 0, y[b]);
          if (!E4M3 && NH > 1) tma_load_2d(dst + kHalf, map, full, 64, y[b]);
          dst += box_rows * 128;
        }
      }
      __syncwarp();
      ++tiles;
      if (++at == slots) {
        at = 0;
        parity ^= 1;
      }
      return true;
    };
    load_all<32>(p, rg, kv == 0, ms->found, ms->seg, b_segFull, b_segEmpty, s_abort, issue,
                 [] {});
    if (*s_abort) {
      // the copies in flight land before the block's shared memory goes
      for (uint32_t i = tiles > slots ? tiles - slots : 0; i < tiles; ++i)
        mbar_wait(b_full + 8 * (slot0 + i % slots), (i / slots) & 1);
    }
  } else if (warp == F::kWarpS) {
    // ------------------------------------------------------------ scores
    if (elect_one()) {
      constexpr uint32_t kIdS = E4M3 ? idesc_e4m3_f32(128, F::kQRows) : idesc_bf16_f32(128, F::kQRows);
      const int ksteps = E4M3 ? (p.c.D + 31) / 32 : p.c.D / 16;
      const uint64_t k0 = desc_kmajor_sw128(smem_u32(smem));
      const uint64_t q0 = desc_kmajor_sw128(smem_u32(smem) + F::kQOff);
      uint32_t t = 0, at = 0, parity = 0;  // tiles so far, the ring's slot
      bool ok = true;
#pragma unroll 1
      for (int sn = 0; ok; ++sn) {
        const int ss = sn % kSegDepth, qb = sn & 1;
        ok = wait_bar(b_segFull + 8 * ss, (sn / kSegDepth) & 1, s_abort);
        if (!ok) break;
        const int nt = ms->seg[ss].ntiles;
        mbar_arrive(b_segEmpty + 8 * ss);
        if (nt == 0) break;
        ok = wait_bar(b_qFull + 8 * qb, (sn >> 1) & 1, s_abort);
#pragma unroll 1
        for (int i = 0; i < nt && ok; ++i, ++t) {
          const uint32_t sb = t % SB;
          ok = wait_bar(b_sFree + 8 * sb, ((t / SB) & 1) ^ 1, s_abort) &&
               wait_bar(b_full + 8 * at, parity, s_abort);
          if (!ok) break;
          tc_fence_after();
          uint64_t a = k0 + at * (F::kSlot >> 4), b = q0 + qb * (F::kQBytes >> 4);
#pragma unroll 2
          for (int k = 0; k < ksteps; ++k) {
            if constexpr (E4M3) {
              mma_e4m3(tmem + sb * 64, a, b, kIdS, k > 0);
            } else {
              mma_bf16(tmem + sb * 64, a, b, kIdS, k > 0);
            }
            a += 2;
            b += 2;
            if (!E4M3 && k == 3) {
              a += (kHalf >> 4) - 8;
              b += (F::kQHalf >> 4) - 8;
            }
          }
          mma_commit(b_s + 8 * sb);
          mma_commit(b_empty + 8 * at);
          if (++at == NK) {
            at = 0;
            parity ^= 1;
          }
        }
        if (ok) mma_commit(b_qEmpty + 8 * qb);
      }
      if (!ok) {
        mma_commit(b_drain);
        mbar_wait(b_drain, 0);
      }
    }
    __syncwarp();
  } else if (warp == F::kWarpO) {
    // ------------------------------------------------------------ outputs
    if (elect_one()) {
      constexpr uint32_t kIdO =
          idesc_bf16_f32(128, F::kPN) | kIdescTransposeA | kIdescTransposeB;
      // D = 64: both groups of 64 MMA rows read the same values
      const uint64_t v0 = desc_mnmajor_sw128(smem_u32(smem) + kVOff, NH > 1 ? kHalf : 0);
      const uint64_t p0 = desc_mnmajor_sw128(smem_u32(smem) + F::kPOff, 0);
      uint32_t at = 0, parity = 0, ph_p = 0;
      bool ok = true;
#pragma unroll 1
      for (int sn = 0; ok; ++sn) {
        const int ss = sn % kSegDepth;
        ok = wait_bar(b_segFull + 8 * ss, (sn / kSegDepth) & 1, s_abort);
        if (!ok) break;
        const int nt = ms->seg[ss].ntiles;
        mbar_arrive(b_segEmpty + 8 * ss);
        if (nt == 0) break;
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
          const int s = i & 1;
          ok = wait_bar(b_v + 8 * at, parity, s_abort) &&
               wait_bar(b_p + 8 * s, (ph_p >> s) & 1, s_abort);
          if (!ok) break;
          ph_p ^= 1u << s;
          tc_fence_after();
          uint64_t a = v0 + at * (F::kTile >> 4), b = p0 + s * (kHalf >> 4);
          const uint32_t o = tmem + F::kColO + s * F::kOCols;
#pragma unroll 2
          for (int k = 0; k < kBN / 16; ++k) {  // steps of 16 positions, 2048 bytes
            mma_bf16(o, a, b, kIdO, i >= 2 || k > 0);
            a += 2048 >> 4;
            b += 2048 >> 4;
          }
          mma_commit(b_vFree + 8 * at);
          mma_commit(b_o + 8 * s);
          if (++at == NM) {
            at = 0;
            parity ^= 1;
          }
        }
      }
      if (!ok) {
        mma_commit(b_drain + 8);
        mbar_wait(b_drain + 8, 0);
      }
    }
    __syncwarp();
  } else if (warp < F::kSoft / 32) {
    // ------------------------------------------------------------ softmax
    // Every step goes over the rows in a loop of eight at a time: the code of a tile
    // has to stay in the instruction caches, which all roles share.
    const int s = warp >> 2;   // the stream
    const int wg = 2 + s;      // its barrier
    const int pt = tid & 127;  // position of the tile, value of D at the end
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_o = tmem + lanes + F::kColO + s * F::kOCols;
    const uint32_t t_l = tmem + lanes + F::kColL + s * 32;
    const float c2 = p.scale * kLog2e;
    float* nm = ms->nm[s];
    float* f = ms->f[s];
    uint8_t* my_p = smem + F::kPOff + s * kHalf + pt * 128;
    uint32_t ph_o = 0, base = 0;  // base: tiles of the segments before
    // this position's sums of 8 rows
    auto load_l = [&](int r0, float (&v)[8]) {
      uint32_t u[8];
      tmem_ld_32x32b_x8(t_l + r0, u);
      tmem_wait_ld_regs(u);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(u[k]);
    };
    auto store_l = [&](int r0, const float (&v)[8]) {
      uint32_t u[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(v[k]);
      tmem_st_32x32b_x8(t_l + r0, u);
    };
#pragma unroll 1
    for (int sn = 0;; ++sn) {
      const int ss = sn % kSegDepth;
      const bool got = wait_bar(b_segFull + 8 * ss, (sn / kSegDepth) & 1, s_abort);
      // all leave together
      if (group_any(1, F::kSoft, !got)) break;
      const Segment sg = ms->seg[ss];
      __syncwarp();
      if (lane == 0) mbar_arrive(b_segEmpty + 8 * ss);
      if (sg.ntiles == 0) break;

      if (pt < NR) nm[pt] = pt < sg.nrows ? kUnset : 0.f;
      {
        const float zero[8] = {};
#pragma unroll 1
        for (int r0 = 0; r0 < sg.nrows; r0 += 8) store_l(r0, zero);
      }
      group_sync(wg, 128);
      // positions that every row sees
      const int all_hi = p.causal ? sg.ctx + p.by_G(sg.r0) + 1 : sg.ctx + sg.m;
      const int all_lo =
          p.window == 0 ? 0 : sg.ctx + p.by_G(sg.r0 + sg.nrows - 1) - p.window + 1;
      if (E4M3) wait_bar(b_qFull + 8 * (sn & 1), (sn >> 1) & 1, s_abort);
      const float* row_scale = ms->a[sn & 1];
#pragma unroll 1
      for (int i = s; i < sg.ntiles; i += 2) {
        const int t0 = (sg.tile0 + i) * kBN;
        float ck = 0.f;
        if constexpr (E4M3) {
          // the scale of this thread's key
          const uint32_t q = (base + i) % kExpDepth;
          wait_bar(b_expFull + 8 * q, ((base + i) / kExpDepth) & 1, s_abort);
          const uint32_t ek = exponent_byte(smem[F::kExpOff + q * 256 + pt]);
          __syncwarp();
          if (lane == 0) mbar_arrive(b_expEmpty + 8 * q);
          ck = __uint_as_float(ek << 23);
        }
        const uint32_t sb = (base + i) % SB, t_s = tmem + lanes + sb * 64;
        wait_bar(b_s + 8 * sb, ((base + i) / SB) & 1, s_abort);
        __syncwarp();
        tc_fence_after();
        // rows r_lo .. r_hi - 1 see this thread's position
        int r_lo = 0, r_hi = NR;
        const bool mask = t0 < all_lo || t0 + kBN > all_hi;
        if (mask) {
          const int c = t0 + pt;
          if (!p.causal) {
            if (c >= sg.ctx + sg.m) r_lo = NR;
          } else {
            // row r is at position ctx + r / G: it sees c from r = (c - ctx) G on
            r_lo = min(max(min(max(c - sg.ctx, 0), 1 << 20) * p.G - sg.r0, 0), NR);
            if (p.window > 0) {
              const int j = min((int64_t)c + p.window - sg.ctx, (int64_t)1 << 20);
              r_hi = min(max(max(j, 0) * p.G - sg.r0, 0), NR);
            }
          }
        }
        // The logarithms to base 2 of the rows' exponentials, back to S, and whether one
        // passes its reference by too much.  Eights of rows that the item does not have are
        // left out throughout.
        float top = -INFINITY;
#pragma unroll 1
        for (int r0 = 0; r0 < sg.nrows; r0 += 8) {
          uint32_t u[8];
          float y[8];
          tmem_ld_32x32b_x8(t_s + r0, u);
          if constexpr (E4M3) {
            uint32_t v[8];
            tmem_ld_32x32b_x8(t_s + NR + r0, v);
            tmem_wait_ld_regs(u, v);
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
              const float2 a = *reinterpret_cast<const float2*>(row_scale + r0 + k);
              const unsigned long long x =
                  fma2(pack2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])),
                       pack2(0.0625f, 0.0625f),
                       pack2(__uint_as_float(u[k]), __uint_as_float(u[k + 1])));
              unpack2(mul2(mul2(x, pack2(a.x, a.y)), pack2(ck, ck)), y[k], y[k + 1]);
            }
          } else {
            tmem_wait_ld_regs(u);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = __uint_as_float(u[k]) * c2;
          }
          if (mask)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (r0 + k < r_lo || r0 + k >= r_hi) y[k] = -INFINITY;
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            top = max3(top, y[k] + nm[r0 + k], y[k + 1] + nm[r0 + k + 1]);
            u[k] = __float_as_uint(y[k]);
            u[k + 1] = __float_as_uint(y[k + 1]);
          }
          tmem_st_32x32b_x8(t_s + r0, u);
        }
        tmem_wait_st();
        const bool moves = group_any(wg, 128, top > kLimit);
        if (i >= 2) {  // the products before this tile's are done
          wait_bar(b_o + 8 * s, ph_o, s_abort);
          __syncwarp();
          ph_o ^= 1;
          tc_fence_after();
        }
        if (moves) {
          // references move to the tile's maxima
#pragma unroll 1
          for (int r0 = 0; r0 < sg.nrows; r0 += 8) {
            uint32_t u[8];
            tmem_ld_32x32b_x8(t_s + r0, u);
            tmem_wait_ld_regs(u);
            int best = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              // integers in the order of the floats
              const int b = (int)u[k];
              const int m = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7fffffff));
              if (lane == k) best = m;
            }
            if (lane < 8)
              ms->wm[s][warp & 3][r0 + lane] = __int_as_float(best ^ ((best >> 31) & 0x7fffffff));
          }
          group_sync(wg, 128);
          if (pt < sg.nrows) {
            const float old = -nm[pt];
            const float m = max3(fmaxf(ms->wm[s][0][pt], ms->wm[s][1][pt]), ms->wm[s][2][pt],
                                 ms->wm[s][3][pt]);
            const bool moved = m - old > kLimit / 2;
            if (moved) nm[pt] = -m;
            f[pt] = moved ? ex2_approx(old - m) : 1.f;
          } else if (pt < NR) {
            f[pt] = 1.f;
          }
          group_sync(wg, 128);
          if (i >= 2) {
#pragma unroll 1
            for (int r0 = 0; r0 < sg.nrows; r0 += 8) {
              float w[8], v[8];
              bool moved = false;  // alike in every thread
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                w[k] = f[r0 + k];
                moved |= w[k] != 1.f;
              }
              if (!moved) continue;
              load_l(r0, v);
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] *= w[k];
              store_l(r0, v);
#pragma unroll 1
              for (int q = 0; q < 2; ++q) {
                uint32_t o[8];
                tmem_ld_32x32b_x8(t_o + q * NR + r0, o);
                tmem_wait_ld_regs(o);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * w[k]);
                tmem_st_32x32b_x8(t_o + q * NR + r0, o);
              }
            }
            tmem_wait_st();
          }
        }
        // P: the position's row of its terms
#pragma unroll 1
        for (int r0 = 0; r0 < sg.nrows; r0 += 8) {
          uint32_t u[8];
          float l[8];
          tmem_ld_32x32b_x8(t_s + r0, u);
          load_l(r0, l);
          tmem_wait_ld_regs(u);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            u[k] = __float_as_uint(ex2_approx(__uint_as_float(u[k]) + nm[r0 + k]));
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = __uint_as_float(u[2 * k]), b = __uint_as_float(u[2 * k + 1]);
            l[2 * k] += a;
            l[2 * k + 1] += b;
            hi[k] = pack_bf16(a, b);
            lo[k] = pack_bf16(a - __uint_as_float(hi[k] << 16),
                              b - __uint_as_float(hi[k] & 0xffff0000u));
          }
          *reinterpret_cast<uint4*>(my_p + (((r0 >> 3) ^ (pt & 7)) << 4)) =
              make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(my_p + ((((NR + r0) >> 3) ^ (pt & 7)) << 4)) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
          store_l(r0, l);
        }
        // values that no row sees: 0 * NaN must not reach a sum (e4m3: converted to zeros)
        if (!E4M3 && (t0 < sg.lo || t0 + kBN > sg.hi)) {
          const uint32_t slot = NK + (base + i) % NV;
          wait_bar(b_full + 8 * slot, ((base + i) / NV) & 1, s_abort);
          if (t0 + pt < sg.lo || t0 + pt >= sg.hi) {
            uint8_t* v = smem + slot * F::kSlot + pt * 128;
#pragma unroll
            for (int k = 0; k < (int)(F::kSlot / 2048); ++k)
              *reinterpret_cast<uint4*>(v + (k >> 3) * kHalf + (k & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_p + 8 * s);
          mbar_arrive(b_sFree + 8 * sb);
        }
      }
      __syncwarp();
      if (E4M3 && lane == 0) mbar_arrive(b_qEmpty + 8 * (sn & 1));
      const bool has = s < sg.ntiles;
      if (has) {
        wait_bar(b_o + 8 * s, ph_o, s_abort);
        ph_o ^= 1;
      }
      __syncwarp();
      tc_fence_after();
      tmem_wait_st();
      base += sg.ntiles;

      // The streams' sums, then their O, a thread's value of D, through shared memory
      // (P is no longer read)
      float* o_s = reinterpret_cast<float*>(smem + F::kPOff + s * kHalf);
#pragma unroll 1
      for (int r0 = 0; r0 < sg.nrows; r0 += 8) {
        float v[8];
        load_l(r0, v);
        const float sum = reduce_rows<8>(v, [](float a, float b) { return a + b; });
        if (lane % 4 == 0) ms->wm[s][warp & 3][r0 + lane / 4] = sum;
        if (has) {
          uint32_t hi[8], lo[8];
          tmem_ld_32x32b_x8(t_o + r0, hi);
          tmem_ld_32x32b_x8(t_o + NR + r0, lo);
          tmem_wait_ld_regs(hi, lo);
          if (pt < DP)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              o_s[(r0 + k) * DP + pt] = __uint_as_float(hi[k]) + __uint_as_float(lo[k]);
        }
      }
      group_sync(1, F::kSoft);
      const bool both = sg.ntiles > 1;
      const float* o0 = reinterpret_cast<const float*>(smem + F::kPOff);
      float* rec = p.part + ((size_t)blockIdx.x * 2 + (sg.split == 2 ? 1 : 0)) *
                                record_floats(32, DP);
#pragma unroll 1
      for (int task = tid; task < sg.nrows * (DP / 8); task += F::kSoft) {
        const int r = task / (DP / 8), d = task % (DP / 8) * 8;
        float m[2], t[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          t[k] = (ms->wm[k][0][r] + ms->wm[k][1][r]) + (ms->wm[k][2][r] + ms->wm[k][3][r]);
          m[k] = k == 0 || both ? -ms->nm[k][r] : -kUnset;
        }
        const float M = fmaxf(m[0], m[1]);
        float w0 = ex2_approx(m[0] - M), w1 = both ? ex2_approx(m[1] - M) : 0.f;
        const float L = both ? fmaf(t[0], w0, t[1] * w1) : t[0] * w0;
        if (!sg.split) {
          const float inv = L == 0.f ? 0.f : 1.f / L;
          w0 *= inv;
          w1 *= inv;
        }
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
          const float4 a = *reinterpret_cast<const float4*>(o0 + r * DP + d + k);
          v[k] = a.x * w0, v[k + 1] = a.y * w0, v[k + 2] = a.z * w0, v[k + 3] = a.w * w0;
          if (both) {
            const float4 b = *reinterpret_cast<const float4*>(o0 + kHalf / 4 + r * DP + d + k);
            v[k] = fmaf(b.x, w1, v[k]);
            v[k + 1] = fmaf(b.y, w1, v[k + 1]);
            v[k + 2] = fmaf(b.z, w1, v[k + 2]);
            v[k + 3] = fmaf(b.w, w1, v[k + 3]);
          }
        }
        if (sg.split) {
          float4* to = reinterpret_cast<float4*>(rec + r * DP + d);
          __stcg(to, make_float4(v[0], v[1], v[2], v[3]));
          __stcg(to + 1, make_float4(v[4], v[5], v[6], v[7]));
          if (d == 0)
            __stcg(reinterpret_cast<float2*>(rec + 32 * DP) + r,
                   make_float2(M == -kUnset ? -INFINITY : M, L));
        } else {
          const int64_t at = out_row(p, sg.row0, sg.h, sg.r0 + r);
          if (d < p.c.D)
            *reinterpret_cast<uint4*>(p.out + at * p.c.D + d) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                           pack_bf16(v[6], v[7]));
          if (d == 0 && p.lse != nullptr)
            p.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
        }
      }
      if (sg.split)
        finish_split<DP, 32, F::kSoft, false>(p, sg, &ms->last,
                                              reinterpret_cast<float2*>(smem + F::kPOff));
      tc_fence_before();
    }
  } else if (E4M3 && warp > F::kWarpO) {
    // ------------------------------------------------------------ V's codes to bf16
    const Converter<DP, F::kConv ? F::kConv : 4> convert(warp - F::kWarpO - 1, lane);
    uint32_t t = 0, at = 0, parity = 0;  // tiles so far, the ring's slot
    bool ok = true;
#pragma unroll 1
    for (int sn = 0; ok; ++sn) {
      const int ss = sn % kSegDepth;
      ok = __all_sync(0xffffffffu, wait_bar(b_segFull + 8 * ss, (sn / kSegDepth) & 1, s_abort));
      if (!ok) break;
      const int nt = ms->seg[ss].ntiles, lo = ms->seg[ss].lo, hi = ms->seg[ss].hi;
      int t0 = ms->seg[ss].tile0 * kBN;
      __syncwarp();
      if (lane == 0) mbar_arrive(b_segEmpty + 8 * ss);
      if (nt == 0) break;
#pragma unroll 1
      for (int i = 0; i < nt; ++i, ++t, t0 += kBN) {
        const uint32_t q = t % kExpDepth, to = t % NM;
        ok = wait_bar(b_full + 8 * (NK + at), parity, s_abort) &&
             wait_bar(b_expFull + 8 * q, (t / kExpDepth) & 1, s_abort) &&
             wait_bar(b_convFree + 8 * to, ((t / NM) & 1) ^ 1, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        convert(smem + (NK + at) * F::kSlot, smem + F::kExpOff + q * 256 + 128,
                smem + F::kConvOff + to * F::kTile, lo - t0, hi - t0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_conv + 8 * to);
          mbar_arrive(b_empty + 8 * (NK + at));
          mbar_arrive(b_expEmpty + 8 * q);
        }
        if (++at == NV) {
          at = 0;
          parity ^= 1;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ Q, e4m3's scales
    uint32_t base = 0;  // tiles of the segments before
#pragma unroll 1
    for (int sn = 0;; ++sn) {
      const int ss = sn % kSegDepth, qb = sn & 1;
      const bool got = wait_bar(b_segFull + 8 * ss, (sn / kSegDepth) & 1, s_abort) &&
                       wait_bar(b_qEmpty + 8 * qb, ((sn >> 1) & 1) ^ 1, s_abort);
      if (__any_sync(0xffffffffu, !got)) break;
      const Segment sg = ms->seg[ss];
      __syncwarp();
      if (lane == 0) mbar_arrive(b_segEmpty + 8 * ss);
      if (sg.ntiles == 0) break;
      // Q: 16 lanes a row, 8 values a lane, four rows in flight; what its last 8 rows hold
      // past the item's are zeros (the columns of S beyond are not read)
      const int ch = lane & 15;
#pragma unroll 1
      for (int r8 = 0; r8 < sg.nrows; r8 += 8) {
        const int row0 = r8 + (lane >> 4);
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[k] = make_uint4(0, 0, 0, 0);
          if (row0 + 2 * k < sg.nrows)
            x[k] = load_q(p, sg.row0, sg.h, sg.r0 + row0 + 2 * k, ch * 8);
        }
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          const int row = row0 + 2 * k;
          const uint4 now = x[0];
          x[0] = x[1];
          x[1] = x[2];
          x[2] = x[3];
          uint8_t* dst = smem + F::kQOff + qb * F::kQBytes + row * 128;
          if constexpr (!E4M3) {
            if (ch < DP / 8)
              *reinterpret_cast<uint4*>(dst + (ch >> 3) * F::kQHalf +
                                        (((ch & 7) ^ (row & 7)) << 4)) = now;
          } else {
            const uint32_t w[4] = {now.x, now.y, now.z, now.w};
            float f[8], amax = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              f[2 * j] = __uint_as_float(w[j] << 16);
              f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
              amax = max3(amax, fabsf(f[2 * j]), fabsf(f[2 * j + 1]));
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
              amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o, 16));
            // q 2^-a within the codes' range
            const int a = min(max((int)(__float_as_uint(amax) >> 23) - 127 - 7, -126), 120);
            const float inv = __uint_as_float((uint32_t)(127 - a) << 23);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float u = f[2 * j] * inv, v = f[2 * j + 1] * inv;
              hi[j] = e4m3x2(u, v);
              uint32_t h;
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)hi[j]));
              const float2 g = __half22float2(*reinterpret_cast<__half2*>(&h));
              lo[j] = e4m3x2((u - g.x) * 16.f, (v - g.y) * 16.f);
            }
            // 8 codes a lane: half a 16-byte chunk
            const uint32_t to = ((((uint32_t)ch >> 1) ^ (row & 7)) << 4) + (ch & 1) * 8;
            *reinterpret_cast<uint2*>(dst + to) =
                make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
            *reinterpret_cast<uint2*>(dst + NR * 128 + to) =
                make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
            // an infinite q has no product with a value
            if (ch == 0)
              ms->a[qb][row] = amax < INFINITY ? __uint_as_float((uint32_t)(127 + a) << 23) *
                                                     (p.scale * kLog2e)
                                               : NAN;
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(b_qFull + 8 * qb);
      if constexpr (!E4M3) continue;
      // the exponent bytes of K and V, four positions a lane; a tile's are loaded while
      // those of the one before wait for room.  Where no row looks, any scale does.
      const int log_page = p.c.log_page, end_pos = min(sg.hi, p.c.max_pages << log_page);
      const int32_t* table = p.c.pages + (int64_t)sg.n * p.c.max_pages;
      auto page = [&](int pos) {
        return pos < end_pos && pos + 4 > sg.lo ? __ldg(table + (pos >> log_page)) : -1;
      };
      int pos = sg.tile0 * kBN + lane * 4, id = page(pos);
#pragma unroll 1
      for (uint32_t tile = base, end = base + sg.ntiles; tile < end; ++tile, pos += kBN) {
        uint32_t x = 0x7f7f7f7fu, y = x;
        if (id >= 0 && id < p.c.n_pages) {
          const int64_t at = (((int64_t)id * p.c.Hkv + sg.h) << log_page) +
                             (pos & ((1 << log_page) - 1));
          x = __ldg(reinterpret_cast<const uint32_t*>(p.c.k_exp + at));
          y = __ldg(reinterpret_cast<const uint32_t*>(p.c.v_exp + at));
        }
        id = page(pos + kBN);
        const uint32_t q = tile % kExpDepth;
        wait_bar(b_expEmpty + 8 * q, ((tile / kExpDepth) & 1) ^ 1, s_abort);
        uint32_t* to = reinterpret_cast<uint32_t*>(smem + F::kExpOff + q * 256) + lane;
        to[0] = x;
        to[32] = y;
        mbar_arrive(b_expFull + 8 * q);
      }
      base += sg.ntiles;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *s_abort) set_flag(p.c.status, kFlagWaitTimeout);
  if (warp == F::kWarpS) {
    tc_fence_after();
    tmem_dealloc(tmem, F::kTmemCols);
  }
}

template <int DP, int NR, bool E4M3>
cudaError_t launch_one(const AttendArgs& a, const Params& p, cudaStream_t st) {
  using F = Few<DP, NR, E4M3>;
  auto kernel = attend_few_kernel<DP, NR, E4M3>;
  cudaError_t e = ensure_smem_attr((const void*)kernel, F::kTotal);
  if (e != cudaSuccess) return e;
  const int grid = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
  DSPARK_LAUNCH(kKindAttend, st,
                e = launch_pdl(kernel, dim3(grid), dim3(F::kThreads), F::kTotal, st, a.desc->tm_k,
                               a.desc->tm_v, p));
  return e;
}

template <int DP, bool E4M3>
cudaError_t launch_rows(const AttendArgs& a, const Params& p, cudaStream_t st) {
  const int rows = p.max_rows * p.G;
  if (rows <= 8) return launch_one<DP, 8, E4M3>(a, p, st);
  if (rows <= 16) return launch_one<DP, 16, E4M3>(a, p, st);
  return launch_one<DP, 32, E4M3>(a, p, st);
}

}  // namespace

cudaError_t launch_attend_few(const AttendArgs& a, const attend::Params& p, cudaStream_t st) {
  const bool e4m3 = p.c.k_exp != nullptr;
  if (p.c.D > 64)
    return e4m3 ? launch_rows<128, true>(a, p, st) : launch_rows<128, false>(a, p, st);
  return e4m3 ? launch_rows<64, true>(a, p, st) : launch_rows<64, false>(a, p, st);
}

}  // namespace dspark
