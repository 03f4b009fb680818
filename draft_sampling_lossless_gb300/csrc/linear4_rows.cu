// Products of a few rows with 4-bit weights: x W^T, and act(x G^T) * (x U^T), T <= 32.
//
// The weights' bytes are all the time there is (4.25 bits a value), so a warp takes them
// from memory into registers, several loads ahead, and the values never stop in shared
// memory.  mma.sync (16 weight rows by 8 rows of x by 16) sums them in fp32: with one to
// sixteen rows there is nothing for larger MMAs to share, and a launch of these warps has no
// tensor memory, barriers or first kernel to wait for.
//
// A lane (g, t) = (lane / 4, lane % 4) loads 16 bytes, the group of 32 columns 4 s + t, of rows g
// and g + 8: 64 bytes a row and step s.  The columns' order within a product is free, so what
// the lane has loaded is its own part of eight MMAs' A: a pair of codes (p, p + 4 of a word's
// eight) moves to the bits of two bf16 in a few operations, and one multiplication by the
// group's power of two makes them values (exactly).  x lies in shared memory in the same
// order, 16 bytes a lane and two MMAs.
//
// What bounds it: for small matrices latency (one row by 1000 x 1024 3.0 us among calls in a
// graph: a launch, one round trip to memory, the sums of a tile's warps); past that the
// conversions, 21 values a cycle an SM (4.8 instructions a value with everything; one row by 6144 x
// 2560 5.5 us, half of it the three row tiles of the busiest SM), so larger matrices go to
// the tensor cores' kernel.  Conversions by e2m1x2 to
// f16x2, with x in f16 and scales after the MMAs, were no faster (one row 5.4 us, eight 6.6 for
// 6.3, 151936 x 2560 68 for 63).
#include "linear4.cuh"

namespace dspark {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxRows = 32;
constexpr size_t kMaxSmemX = 196608;  // x's bytes in shared memory

// Row m (of 16) of row tile j (of 8) of a block of 128: four neighbours from each quarter, whose
// scales share two sectors.
__device__ __forceinline__ int row_of(int tile, int m) {
  return (tile >> 3) * 128 + (m >> 2) * 32 + (tile & 7) * 4 + (m & 3);
}

__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The threads of a group of warps: at most eight groups have a barrier (1 to 8), a single
// warp needs none.
__device__ __forceinline__ void group_sync(int group, int threads) {
  if (threads == 32) __syncwarp();
  else asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
}

struct Params {
  const uint8_t *w, *u;  // the matrices' tiles
  int N, T, K, Kp, KB, tiles, splits, act;
  const __nv_bfloat16* x;
  int64_t x_stride;
  __nv_bfloat16* out;
  int64_t out_stride;
};

// What a lane loads for one matrix and step.
struct Slot {
  uint4 c0, c1;
  uint32_t s0, s1;
};

// NT: eights of rows of x; DEPTH: steps whose loads are in flight.
template <int MATS, int NT, int DEPTH>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const Params p) {
  constexpr int kRedNT = NT < 2 ? NT : 2;  // eights of rows that are added up at a time
  extern __shared__ uint4 s_x[];           // [KB][4][T][4]: step, word, row, lane's t
  __shared__ float4 red[kWarps][MATS][kRedNT][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  grid_dependency_wait();

  // `splits` warps share a row tile, each a range of K; the groups of warps take tiles in
  // turn, neighbouring tiles in different blocks.
  const int group = warp / p.splits, ks = warp - group * p.splits, groups = kWarps / p.splits;
  const int first = group * gridDim.x + blockIdx.x, stride = gridDim.x * groups;
  const int k0 = p.KB * ks / p.splits, k1 = p.KB * (ks + 1) / p.splits, steps = k1 - k0;
  const int mine = group < groups && first < p.tiles ? (p.tiles - first + stride - 1) / stride : 0;
  const int items = mine * steps;

  Slot ring[DEPTH][MATS];
  int at_tile = first, left = steps, loaded = 0;  // what is loaded next
  // the codes of rows g and g + 8 (64 rows on in the tile), their scales
  const int local = (g >> 2) * 32 + (g & 3), c_lane = local * 64 + t * 16;
  const int s_lane = kTileCodes + (g & 3) * 16 + (g >> 2) * 4 + t;
  int64_t at_c = 0;
  auto place = [&]() {  // (rows past N have zero codes)
    at_c = ((int64_t)(at_tile >> 3) * p.KB + k0) * kTileBytes;
  };
  if (items > 0) place();
  auto load = [&](Slot (&s)[MATS]) {
    if (loaded >= items) return;
    ++loaded;
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
      const uint8_t* tile = (m ? p.u : p.w) + at_c;
      const uint8_t* c = tile + (at_tile & 7) * 256 + c_lane;
      const uint8_t* sc = tile + (at_tile & 7) * 64 + s_lane;
      s[m].c0 = load_codes(c);
      s[m].c1 = load_codes(c + 4096);
      s[m].s0 = __ldg(sc);
      s[m].s1 = __ldg(sc + 8);
    }
    at_c += kTileBytes;
    if (--left == 0) {
      left = steps;
      at_tile += stride;
      if (at_tile < p.tiles) place();
    }
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) load(ring[i]);

  // x in the lanes' order, the columns of eight as (0, 4, 1, 5, 2, 6, 3, 7); zeros past K
  const int chunks = p.Kp >> 3;
  constexpr int kBatch = 8;  // loads in flight
  const int r_step = kThreads / chunks, c_step = kThreads - r_step * chunks;
  int r = tid / chunks, c = tid - r * chunks;
  while (r < p.T) {
    uint4 v[kBatch];
    int at[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      v[b] = make_uint4(0, 0, 0, 0);
      at[b] = r < p.T ? (((c >> 4) * 4 + (c & 3)) * p.T + r) * 4 + ((c >> 2) & 3) : -1;
      if (r < p.T && c * 8 < p.K)
        v[b] = __ldg(reinterpret_cast<const uint4*>(p.x + r * p.x_stride + c * 8));
      r += r_step;
      c += c_step;
      if (c >= chunks) {
        c -= chunks;
        ++r;
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (at[b] >= 0)
        s_x[at[b]] = make_uint4(
            __byte_perm(v[b].x, v[b].z, 0x5410), __byte_perm(v[b].x, v[b].z, 0x7632),
            __byte_perm(v[b].y, v[b].w, 0x5410), __byte_perm(v[b].y, v[b].w, 0x7632));
  }
  __syncthreads();

  float d[MATS][NT][4] = {};
  int tile = first, step = 0;
  const int x_word = p.T * 4;
  const int x_first = k0 * 4 * x_word + t;
  int x_at = x_first;
  // columns of the products past T take the last row of x: they are not stored
  auto x_of = [&](int nt) { return s_x[x_at + min(g + 8 * nt, p.T - 1) * 4]; };
  auto use = [&](const Slot (&s)[MATS]) {
    // a group's power of two, times 2^126 for the codes' bits, in one factor or (scales above 2) two
    uint32_t f0[MATS], f1[MATS];
    bool big = false;
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
      f0[m] = min(s[m].s0 + 126u, 254u) * 0x00800080u;
      f1[m] = min(s[m].s1 + 126u, 254u) * 0x00800080u;
      big |= s[m].s0 > 128u || s[m].s1 > 128u;
    }
    big = __any_sync(0xffffffffu, big);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint4 b[NT];  // (NT > 2: read again for the second matrix)
      if (NT <= 2) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) b[nt] = x_of(nt);
      }
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        const uint32_t w0 = w == 0 ? s[m].c0.x : w == 1 ? s[m].c0.y : w == 2 ? s[m].c0.z : s[m].c0.w;
        const uint32_t w1 = w == 0 ? s[m].c1.x : w == 1 ? s[m].c1.y : w == 2 ? s[m].c1.z : s[m].c1.w;
        uint32_t lo[4] = {mul_bf16x2(pair_bits<0>(w0), f0[m]), mul_bf16x2(pair_bits<0>(w1), f1[m]),
                          mul_bf16x2(pair_bits<1>(w0), f0[m]), mul_bf16x2(pair_bits<1>(w1), f1[m])};
        uint32_t hi[4] = {mul_bf16x2(pair_bits<2>(w0), f0[m]), mul_bf16x2(pair_bits<2>(w1), f1[m]),
                          mul_bf16x2(pair_bits<3>(w0), f0[m]), mul_bf16x2(pair_bits<3>(w1), f1[m])};
        if (big) {
          const uint32_t h0 = s[m].s0 > 128u ? (s[m].s0 - 1u) * 0x00800080u : 0x3f803f80u;
          const uint32_t h1 = s[m].s1 > 128u ? (s[m].s1 - 1u) * 0x00800080u : 0x3f803f80u;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lo[i] = mul_bf16x2(lo[i], i & 1 ? h1 : h0);
            hi[i] = mul_bf16x2(hi[i], i & 1 ? h1 : h0);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (NT > 2) b[nt] = x_of(nt);
          mma_16816(d[m][nt], lo, b[nt].x, b[nt].y);
          mma_16816(d[m][nt], hi, b[nt].z, b[nt].w);
        }
      }
      x_at += x_word;
    }
    if (++step < steps) return;
    // the tile's end: the group's partial sums, added in the order of their ranges
    step = 0;
    x_at = x_first;
    const int n_threads = p.splits * 32;
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += kRedNT) {
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int k = 0; k < kRedNT; ++k) {
          float(&v)[4] = d[m][n0 + k];
          red[warp][m][k][lane] = make_float4(v[0], v[1], v[2], v[3]);
          v[0] = v[1] = v[2] = v[3] = 0.f;
        }
      group_sync(group, n_threads);
      for (int e = tid - group * n_threads; e < kRedNT * 128; e += n_threads) {
        // neighbouring threads take neighbouring features: e = (row of x, feature of the tile)
        const int k = e >> 7, c = (e >> 4) & 7, row = e & 15;
        const int l = (row & 7) * 4 + (c >> 1), j = (row >> 3) * 2 + (c & 1);
        float v[MATS];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          v[m] = 0.f;
          for (int q = 0; q < p.splits; ++q)
            v[m] += reinterpret_cast<const float*>(&red[group * p.splits + q][m][k][l])[j];
        }
        float o = v[0];
        if (MATS == 2) o = activation(p.act, o) * v[MATS - 1];
        const int n = row_of(tile, row), r = (n0 + k) * 8 + c;
        if (n < p.N && r < p.T) p.out[r * p.out_stride + n] = __float2bfloat16(o);
      }
      group_sync(group, n_threads);
    }
    tile += stride;
  };
#pragma unroll 1
  for (int i = 0; i < items; i += DEPTH) {
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) {
      if (i + k < items) {
        use(ring[k]);
        load(ring[k]);
      }
    }
  }
}

template <int MATS, int NT, int DEPTH>
cudaError_t launch(const Linear4Args& a, cudaStream_t st) {
  auto kernel = rows_kernel<MATS, NT, DEPTH>;
  Params p;
  p.w = a.w->store;
  p.u = a.up ? a.up->store : nullptr;
  p.N = a.w->N;
  p.T = a.T;
  p.K = a.w->K;
  p.Kp = a.w->Kp;
  p.KB = p.Kp / 128;
  p.tiles = (p.N + 127) / 128 * 8;
  p.act = a.act;
  p.x = a.x;
  p.x_stride = a.x_stride;
  p.out = a.out;
  p.out_stride = a.out_stride;
  const size_t smem = (size_t)p.T * p.Kp * 2;
  cudaError_t e = ensure_smem_attr((const void*)kernel, (int)kMaxSmemX);
  if (e != cudaSuccess) return e;
  const int grid = sm_count();
  // the warps that share a tile: the fewest steps of the busiest warp (a tile's end counts as
  // one more)
  int64_t least = INT64_MAX;
  for (int s = 1; s <= kWarps && s <= p.KB; ++s) {
    const int64_t slots = (int64_t)grid * (kWarps / s);
    const int64_t steps = (p.tiles + slots - 1) / slots * ((p.KB + s - 1) / s + 1);
    if (steps < least) least = steps, p.splits = s;
  }
  DSPARK_LAUNCH(kKindLinear4, st,
                e = launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, st, p));
  return e;
}

}  // namespace

bool linear4_rows_fits(int T, int Kp) {
  return T <= kMaxRows && (size_t)T * Kp * 2 <= kMaxSmemX;
}

// Its time but for what every call takes: the values of the SM with the most row tiles, at 21 a
// cycle with up to 8 rows (the conversions bound it), 15 and 9 with up to 16 and 32, and x's way
// into shared memory.
int64_t linear4_rows_cycles(const Linear4Args& a) {
  const int tiles = (a.w->N + 127) / 128 * 8, sms = sm_count();
  const int64_t values = (int64_t)((tiles + sms - 1) / sms) * 16 * a.w->Kp * (a.up ? 2 : 1);
  const int64_t rate = a.T <= 8 ? 210 : a.T <= 16 ? 150 : 90;
  return values * 10 / rate + (int64_t)a.T * a.w->Kp * 2 / 40;
}

cudaError_t launch_linear4_rows(const Linear4Args& a, cudaStream_t st) {
  if (a.T <= 8) return a.up ? launch<2, 1, 3>(a, st) : launch<1, 1, 5>(a, st);
  if (a.T <= 16) return a.up ? launch<2, 2, 3>(a, st) : launch<1, 2, 5>(a, st);
  return a.up ? launch<2, 4, 2>(a, st) : launch<1, 4, 4>(a, st);
}

}  // namespace dspark
