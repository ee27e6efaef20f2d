// Tokens of the 8-bit cache as bf16 rows: bf16(code * scale).
//
// One byte in, two out: bound by memory.  The tokens of a page and head lie in
// one piece, in the cache as in the output, so a CTA streams the part of a
// page that is wanted, K and V, in vectors of 8 codes (8 bytes in, 16 out: any
// d that is a multiple of 8, any first token).
#include "kvcache_step_internal.cuh"
#include "sm103_ptx.cuh"

namespace kvcache {
namespace {

using dropkv::grid_dep_launch;
using dropkv::grid_dep_wait;
using dropkv::launch_pdl;

constexpr int kThreads = 256, kBatch = 4;

// Two codes (the low bytes of w) times the scale, as a bf16 pair.
template <int CODE>
__device__ __forceinline__ uint32_t decode2(uint32_t w, float scale) {
  float lo, hi;
  if (CODE == KVCACHE_E4M3) {
    const uint32_t h = e4m3x2_to_half2(w & 0xFFFFu);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    lo = f.x;
    hi = f.y;
  } else {
    lo = (float)(int8_t)w;
    hi = (float)(int8_t)(w >> 8);
  }
  const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(lo, scale), __fmul_rn(hi, scale));
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <int CODE>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadCall p) {
  grid_dep_wait();
  grid_dep_launch();
  const Cache& c = p.c;
  const int tid = threadIdx.x, i = blockIdx.z, h = blockIdx.y;
  const int s = p.seqs ? p.seqs[i] : i;
  if (s < 0 || s >= c.S) {
    if (tid == 0) flag(c.status, KVCACHE_FLAG_BAD_SEQ);
    return;
  }
  const int len = c.length[s], held = c.count[s], from = p.starts ? p.starts[i] : 0;
  const int cnt = p.counts ? p.counts[i] : from <= len ? len - from : -1;
  if (len < 0 || held < 0 || held > c.M || (long long)len > ((long long)held << c.page_log2) || from < 0 || from > len ||
      cnt < 0 || cnt > p.rows || cnt > len - from) {
    if (tid == 0) flag(c.status, DROPKV_FLAG_BAD_LENGTH);
    return;
  }
  const int col = (from >> c.page_log2) + blockIdx.x;
  if (cnt == 0 || col > (from + cnt - 1) >> c.page_log2) return;
  const int base = col << c.page_log2;
  const int t0 = max(from, base), t1 = min(from + cnt, base + c.page);
  const int pg = c.table[(size_t)s * c.M + col];
  if (pg < 0 || pg >= c.P) {
    if (tid == 0) flag(c.status, KVCACHE_FLAG_BAD_PAGE);
    return;
  }
  const size_t unit = (size_t)pg * c.Hkv + h;
  const float scale[2] = {c.ks[unit], c.vs[unit]};
  const size_t at = (unit * c.page + (t0 - base)) * c.d;
  const size_t to = (((size_t)i * c.Hkv + h) * p.rows + (t0 - from)) * c.d;
  const int n = (t1 - t0) * (c.d / 8);
  for (int v0 = tid; v0 < n; v0 += kThreads * kBatch) {
    uint2 x[2][kBatch];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (v0 + u * kThreads < n)
          x[w][u] = __ldcs(reinterpret_cast<const uint2*>((w ? c.v : c.k) + at) + v0 + u * kThreads);
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (v0 + u * kThreads < n)
          reinterpret_cast<uint4*>((w ? p.v : p.k) + to)[v0 + u * kThreads] =
              make_uint4(decode2<CODE>(x[w][u].x, scale[w]), decode2<CODE>(x[w][u].x >> 16, scale[w]),
                         decode2<CODE>(x[w][u].y, scale[w]), decode2<CODE>(x[w][u].y >> 16, scale[w]));
  }
}

}  // namespace

cudaError_t launch_read(const ReadCall& p, cudaStream_t st) {
  const int touched = (int)(((long long)p.rows + p.c.page - 2) / p.c.page) + 1;   // most pages `rows` tokens touch
  const dim3 grid(std::min(touched, p.c.M), p.c.Hkv, p.n);
  return launch_pdl(p.c.code == KVCACHE_INT8 ? read_kernel<KVCACHE_INT8> : read_kernel<KVCACHE_E4M3>, grid,
                    dim3(kThreads), 0, st, p);
}

}  // namespace kvcache
