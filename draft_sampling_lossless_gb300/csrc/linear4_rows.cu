// Products of a few rows with 4-bit weights: x W^T, and act(x G^T) * (x U^T), T <= 16.
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
#include "linear4.cuh"

namespace dspark {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxRows = 16;
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

// Codes p and p + 4 of a word as two bf16, 2^-126 of their values (0.5 is a subnormal).
template <int P>
__device__ __forceinline__ uint32_t pair_bits(uint32_t w) {
  const uint32_t u = P == 3 ? w : w << (12 - 4 * P);
  return (u & 0x80008000u) | ((u >> 6) & 0x01c001c0u);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 c = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&c);
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The threads of a group of warps: at most eight groups have a barrier (1 to 8), a single
// warp needs none.
__device__ __forceinline__ void group_sync(int group, int threads) {
  if (threads == 32) __syncwarp();
  else asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
}

struct Params {
  const uint8_t *cw, *sw, *cu, *su;
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

// A pair's A fragments of rows g and g + 8: the values, times 2^126 2^(b - 127) in one step, or in
// two where that passes bf16's range.
struct Scale {
  uint32_t f, g;
  __device__ __forceinline__ explicit Scale(uint32_t b) {
    f = min(b + 126u, 254u) * 0x00800080u;
    g = b > 128u ? (b - 1u) * 0x00800080u : 0x3f803f80u;
  }
};

template <int MATS, int NT, int DEPTH>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const Params p) {
  extern __shared__ uint4 s_x[];  // [KB][4][T][4]: step, word, row, lane's t
  __shared__ float4 red[kWarps][MATS][NT][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  grid_dependency_wait();

  // `splits` warps share a row tile, each a range of K; the groups of warps take tiles in
  // turn, neighbouring tiles in different blocks.
  const int group = warp / p.splits, ks = warp - group * p.splits;
  const int first = group * gridDim.x + blockIdx.x, stride = gridDim.x * (kWarps / p.splits);
  const int k0 = p.KB * ks / p.splits, k1 = p.KB * (ks + 1) / p.splits, steps = k1 - k0;
  const int mine = first < p.tiles ? (p.tiles - first + stride - 1) / stride : 0;
  const int items = mine * steps;

  Slot ring[DEPTH][MATS];
  int at_tile = first, at_step = k0, loaded = 0;  // what is loaded next
  auto load = [&](Slot (&s)[MATS]) {
    if (loaded >= items) return;
    ++loaded;
    const int n0 = row_of(at_tile, g), n1 = row_of(at_tile, g + 8);
    const int64_t col = (int64_t)at_step * 64 + t * 16;
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
      const uint8_t* c = m ? p.cu : p.cw;
      const uint8_t* sc = (m ? p.su : p.sw) +
                          ((size_t)(at_tile >> 3) * p.KB + at_step) * 512 + (at_tile & 7) * 64 + t;
      s[m].c0 = n0 < p.N ? load_codes(c + (int64_t)n0 * (p.Kp >> 1) + col) : make_uint4(0, 0, 0, 0);
      s[m].c1 = n1 < p.N ? load_codes(c + (int64_t)n1 * (p.Kp >> 1) + col) : make_uint4(0, 0, 0, 0);
      s[m].s0 = __ldg(sc + (g & 3) * 16 + (g >> 2) * 4);
      s[m].s1 = __ldg(sc + (g & 3) * 16 + (g >> 2) * 4 + 8);
    }
    if (++at_step == k1) {
      at_step = k0;
      at_tile += stride;
    }
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) load(ring[i]);

  // x in the lanes' order, the columns of eight as (0, 4, 1, 5, 2, 6, 3, 7); zeros past K
  const int chunks = p.Kp >> 3;
  for (int i = tid; i < p.T * chunks; i += kThreads) {
    const int r = i / chunks, c = i - r * chunks;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c * 8 < p.K) v = __ldg(reinterpret_cast<const uint4*>(p.x + r * p.x_stride + c * 8));
    s_x[(((c >> 4) * 4 + (c & 3)) * p.T + r) * 4 + ((c >> 2) & 3)] =
        make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                   __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
  }
  __syncthreads();

  float d[MATS][NT][4] = {};
  int tile = first, step = k0;
  auto use = [&](const Slot (&s)[MATS]) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint4 b[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        b[nt] = make_uint4(0, 0, 0, 0);
        if (g + 8 * nt < p.T) b[nt] = s_x[((step * 4 + w) * p.T + g + 8 * nt) * 4 + t];
      }
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        const Scale a0(s[m].s0), a1(s[m].s1);
        const uint32_t w0 = w == 0 ? s[m].c0.x : w == 1 ? s[m].c0.y : w == 2 ? s[m].c0.z : s[m].c0.w;
        const uint32_t w1 = w == 0 ? s[m].c1.x : w == 1 ? s[m].c1.y : w == 2 ? s[m].c1.z : s[m].c1.w;
        uint32_t lo[4] = {mul_bf16x2(pair_bits<0>(w0), a0.f), mul_bf16x2(pair_bits<0>(w1), a1.f),
                          mul_bf16x2(pair_bits<1>(w0), a0.f), mul_bf16x2(pair_bits<1>(w1), a1.f)};
        uint32_t hi[4] = {mul_bf16x2(pair_bits<2>(w0), a0.f), mul_bf16x2(pair_bits<2>(w1), a1.f),
                          mul_bf16x2(pair_bits<3>(w0), a0.f), mul_bf16x2(pair_bits<3>(w1), a1.f)};
        if (s[m].s0 > 128u || s[m].s1 > 128u) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lo[i] = mul_bf16x2(lo[i], i & 1 ? a1.g : a0.g);
            hi[i] = mul_bf16x2(hi[i], i & 1 ? a1.g : a0.g);
          }
        }
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816(d[m][nt], lo, b[nt].x, b[nt].y);
          mma_16816(d[m][nt], hi, b[nt].z, b[nt].w);
        }
      }
    }
    if (++step < k1) return;
    // the tile's end: the group's partial sums, added in the order of their ranges
    step = k0;
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        red[warp][m][nt][lane] = make_float4(d[m][nt][0], d[m][nt][1], d[m][nt][2], d[m][nt][3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[m][nt][j] = 0.f;
      }
    const int n_threads = p.splits * 32;
    group_sync(group, n_threads);
    for (int e = tid - group * n_threads; e < NT * 128; e += n_threads) {
      const int nt = e >> 7, l = (e >> 2) & 31, j = e & 3;
      float v[MATS];
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        v[m] = 0.f;
        for (int k = 0; k < p.splits; ++k)
          v[m] += reinterpret_cast<const float*>(&red[group * p.splits + k][m][nt][l])[j];
      }
      float o = v[0];
      if (MATS == 2) o = activation(p.act, o) * v[MATS - 1];
      const int n = row_of(tile, (l >> 2) + (j >> 1) * 8), r = nt * 8 + (l & 3) * 2 + (j & 1);
      if (n < p.N && r < p.T) p.out[r * p.out_stride + n] = __float2bfloat16(o);
    }
    group_sync(group, n_threads);
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

template <int MATS, int NT>
cudaError_t launch(const Linear4Args& a, cudaStream_t st) {
  auto kernel = rows_kernel<MATS, NT, MATS == 2 ? 3 : 5>;
  Params p;
  p.cw = a.w->codes;
  p.sw = a.w->scales;
  p.cu = a.up ? a.up->codes : nullptr;
  p.su = a.up ? a.up->scales : nullptr;
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
  // the warps that share a tile: as many steps as the busiest warp has, the fewest
  int64_t least = INT64_MAX;
  for (int s = 1; s <= kWarps && s <= p.KB; s *= 2) {
    const int64_t slots = (int64_t)grid * (kWarps / s);
    const int64_t steps = (p.tiles + slots - 1) / slots * ((p.KB + s - 1) / s);
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

cudaError_t launch_linear4_rows(const Linear4Args& a, cudaStream_t st) {
  if (a.T <= 8) return a.up ? launch<2, 1>(a, st) : launch<1, 1>(a, st);
  return a.up ? launch<2, 2>(a, st) : launch<1, 2>(a, st);
}

}  // namespace dspark
