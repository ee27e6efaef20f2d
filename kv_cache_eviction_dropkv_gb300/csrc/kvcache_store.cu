// Store of bf16 rows into the paged 8-bit cache.
//
// For the new values x of a (page, head): s = f(max|x|), or the larger of
// that and the old scale where the page holds earlier tokens; codes are
// rn(x / s), and earlier codes c become rn(c s_old / s) when the scale grows.
//
// A CTA holds one (page, head) of K or V in registers (at most 8 vectors of 8
// values a thread), so the values are read once: their largest magnitude is
// an unsigned maximum over the bf16 bit patterns without sign, which also
// shows infinities and not-a-number.
#include "kvcache_internal.cuh"
#include "sm103_ptx.cuh"

namespace kvcache {
namespace {

using dropkv::grid_dep_launch;
using dropkv::grid_dep_wait;
using dropkv::launch_pdl;

constexpr int kVecs = 8;                   // vectors of 8 values a thread holds

template <int PAGE>
__global__ void __launch_bounds__(PAGE * 2) store_kernel(const StoreCall p) {
  constexpr int kThreads = PAGE * 2, kWarps = kThreads / 32;   // d <= 128: PAGE * d / 8 / kThreads <= 8
  grid_dep_wait();
  grid_dep_launch();
  __shared__ uint32_t s_max[kWarps];
  const Cache& c = p.c;
  const int tid = threadIdx.x;
  const int i = blockIdx.z, h = blockIdx.y >> 1, which = blockIdx.y & 1;
  const int s = p.seqs ? p.seqs[i] : i;
  bool again = false;                       // the sequence was named before: that entry stores it
  if (p.seqs)
    for (int j = tid; j < i; j += kThreads) again |= p.seqs[j] == s;
  const bool dup = p.seqs ? __syncthreads_or(again) : false;
  if (s < 0 || s >= c.S || dup) {
    if (tid == 0) flag(c.status, KVCACHE_FLAG_BAD_SEQ);
    return;
  }
  const int len = c.length[s], held = c.count[s], cnt = p.counts ? p.counts[i] : p.rows;
  if (cnt < 0 || cnt > p.rows || cnt > len || held < 0 || held > c.M || (long long)len > (long long)held * PAGE) {
    if (tid == 0) flag(c.status, DROPKV_FLAG_BAD_LENGTH);
    return;
  }
  const int start = len - cnt;
  const int col = start / PAGE + blockIdx.x;
  // by page: the grid covers `rows`, and past the longest sequence col * PAGE leaves 32 bits
  if (cnt == 0 || col > (len - 1) / PAGE) return;
  const int base = col * PAGE;              // first token of the page
  const int pg = c.table[(size_t)s * c.M + col];
  if (pg < 0 || pg >= c.P || c.refs[pg] != 1) {
    if (tid == 0) flag(c.status, KVCACHE_FLAG_BAD_PAGE);
    return;
  }
  const int r0 = max(0, start - base), r1 = min(PAGE, len - base);   // slots of the new tokens
  const int dv = c.d / 8;                   // vectors per row
  const size_t unit = (size_t)pg * c.Hkv + h;
  float* scales = which ? c.vs : c.ks;
  const float held_scale = r0 > 0 ? scales[unit] : 0.f;
  const __nv_bfloat16* src = (which ? p.v : p.k) + ((size_t)i * c.Hkv + h) * p.rows * c.d;
  uint8_t* dst = (which ? c.v : c.k) + unit * PAGE * c.d;
  // vector n of the page: row n / dv; the new ones are [r0 dv, r1 dv)
  const __nv_bfloat16* from = src + ((long long)base - start) * c.d;   // of the page's slot 0
  uint4 x[kVecs];
  uint32_t m2 = 0;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int n = r0 * dv + tid + u * kThreads;
    x[u] = make_uint4(0, 0, 0, 0);
    if (n < r1 * dv) x[u] = __ldcs(reinterpret_cast<const uint4*>(from + (long long)n * 8));
  }
#pragma unroll
  for (int u = 0; u < kVecs; ++u) m2 = __vmaxu2(m2, largest2(x[u]));
  auto block_max = [&](uint32_t m) {
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) s_max[tid >> 5] = m;
    __syncthreads();
    uint32_t r = s_max[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) r = max(r, s_max[w]);
    __syncthreads();
    return r;
  };
  uint32_t top = block_max(max(m2 & 0xFFFFu, m2 >> 16));
  if (top >= 0x7F80u) {                     // an infinity or not-a-number: the scale is that of the others
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) m = max(m, largest_finite(x[u]));
    top = block_max(m);
    if (tid == 0) flag(c.status, DROPKV_FLAG_NONFINITE);
  }
  const float scale = fmaxf(page_scale(__uint_as_float(top << 16), c.code), held_scale), inv = 1.0f / scale;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int n = r0 * dv + tid + u * kThreads;
    if (n < r1 * dv) *reinterpret_cast<uint2*>(dst + (size_t)n * 8) = codes8(x[u], scale, inv, c.code);
  }
  if (r0 > 0 && scale > held_scale) {       // earlier tokens of the page at the new scale
    const float ratio = held_scale / scale;
    for (int n = tid; n < r0 * dv; n += kThreads) {
      uint2 w = *reinterpret_cast<const uint2*>(dst + (size_t)n * 8);
      w.x = rescale4(w.x, held_scale, scale, ratio, c.code);
      w.y = rescale4(w.y, held_scale, scale, ratio, c.code);
      *reinterpret_cast<uint2*>(dst + (size_t)n * 8) = w;
    }
  }
  if (tid == 0) scales[unit] = scale;
}

}  // namespace

cudaError_t launch_store(const StoreCall& p, cudaStream_t st) {
  const int touched = (int)(((long long)p.rows + p.c.page - 2) / p.c.page) + 1;   // most pages `rows` tokens touch
  const dim3 grid(touched, 2 * p.c.Hkv, p.n);
  switch (p.c.page) {
    case 32: return launch_pdl(store_kernel<32>, grid, dim3(64), 0, st, p);
    case 64: return launch_pdl(store_kernel<64>, grid, dim3(128), 0, st, p);
    case 128: return launch_pdl(store_kernel<128>, grid, dim3(256), 0, st, p);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvcache
