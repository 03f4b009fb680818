// Attention of packed rows over the paged cache: which kernel runs.
#include "attend.cuh"

namespace dspark {

using namespace attend;

// Up to 32 packed rows a head (max_rows is the host's bound of a request's rows)
// are the N side of the products, as far as its two terms of P and S's columns go; more
// are their M side.  With 32 the first kernel is still ahead: 64 requests of 1 to 8
// rows of a group of 4 take 184 us (the other 218), over e4m3 184 us (274), of 8 rows each
// 193 us (217) and 204 us (289); single tokens over e4m3 150 us (287), one token 12.7 us
// (16.8), each in a graph.  Past 32 there is the second kernel only: requests of 1 to 9
// rows 179 us, 78% of the measured copy rate, over e4m3 319 us, 29%.
static bool few(int max_rows, int group) { return (int64_t)max_rows * group <= 32; }

size_t attend_workspace_bytes(int T, int group, int D) {
  return kPartOffset + (size_t)kMaxCtas * 2 * sizeof(float) *
                           record_floats(few(T, group) ? 32 : 256, D > 64 ? 128 : 64);
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st) {
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
  return few(p.max_rows, p.G) ? launch_attend_few(a, p, st) : launch_attend_many(a, p, st);
}

}  // namespace dspark
