// Internal declarations of the paged 8-bit KV cache: parameter blocks, the
// workspace plan and launchers.
#pragma once
#include <algorithm>
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/kvcache.h"
#include "dropkv_host.cuh"
#include "dropkv_internal.cuh"

namespace kvcache {

constexpr float kScaleMin = 0x1p-120f;      // smallest scale of a page
constexpr int kMaxHeads = 4096;
constexpr int kMaxPages = 1 << 24;

// The cache as the kernels see it.
struct Cache {
  uint8_t *k, *v;                // [layers][P][Hkv][page][d]
  float *ks, *vs;                // [layers][P][Hkv]
  int32_t *refs, *table, *count, *length;
  int layers, Hkv, d, page, P, S, M;
  int page_log2;
  int code;
  uint32_t* status;
};

// Workspace of the page calls (int32 arrays).
struct PagePlan {
  size_t claim;                  // [S] lowest call index that names the sequence
  size_t mark;                   // [S] 1: the sequence is a source of this fork
  size_t from;                   // [S] fork, shared: the page that copy k is made of
  size_t offs;                   // [S + 1] pages taken by entries before i
  size_t entry;                  // [S][4] per entry: what the second kernel needs
  size_t list;                   // [P] pages taken, in order
  size_t rows;                   // [kEarlyRows] old table rows of a compaction
  size_t total;                  // bytes
};
constexpr int kEarlyRows = 1024;            // table entries one CTA rewrites by itself
PagePlan make_page_plan(int S, int P);

struct PageCall {
  Cache c;
  const int32_t *seqs, *other;   // sequences (fork: src and dst)
  int n;
  const int32_t* extra;          // reserve
  int32_t* granted;              // reserve: tokens each entry got, or null
  const int32_t *kept_idx, *kept_len;
  int kept_stride, share;
  int32_t *claim, *mark, *from, *offs, *list, *rows;
  int4* entry;
  int early;                     // compact: the bookkeeping rewrites the tables
};

cudaError_t launch_free(const PageCall& p, cudaStream_t st);
cudaError_t launch_reserve(const PageCall& p, cudaStream_t st);
cudaError_t launch_fork(const PageCall& p, int sms, cudaStream_t st);
cudaError_t launch_compact_pages(const PageCall& p, int sms, cudaStream_t st);

struct StoreCall {
  Cache c;                       // k, v, ks, vs at the layer
  const int32_t* seqs;
  int n, rows;
  const __nv_bfloat16 *k, *v;
  const int32_t* counts;
};
cudaError_t launch_store(const StoreCall& p, cudaStream_t st);

struct AttnCall {
  Cache c;                       // k, v, ks, vs at the layer
  const int32_t* seqs;
  int n, Hq, T, g, R;            // R = g * T query rows per KV head
  int RB, RG;                    // rows per warp (8 or 16), row groups per KV head
  int window, sinks;
  int workers;                   // warps of the grid: run * RG + row group
  int solo;                      // 1: a warp per unit and row group, nothing to join
  int team;                      // > 0: a cluster of that many CTAs per unit, joined in shared memory
  int by_unit;                   // 1: cuts is per unit, 0: per run
  int rowwise;                   // 1: a join CTA takes one row
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* part_o;                 // [workers][2][RB][d]
  float4* part_s;                // [workers][2][RB] (m, l, M, unused)
  int2* cuts;                    // by_unit: [units][RG] (first run or -1, last run); else [workers] (unit or -1, last run)
  float scale_log2;
  const int32_t* from;           // a shared attention's second half: first token of each entry
  float* own_o;                  // and what it leaves of units that no run border cuts: [n * Hq * T][d]
  float4* own_s;                 // [n * Hq * T] (m, l, M, unused)
};
struct AttnPlan {
  int RB, RG, workers, solo, team, by_unit, rowwise;
  size_t part_s, cuts, total;    // byte offsets
};
// false: more tiles than a 32-bit count holds.
bool make_attn_plan(const kvcache_shape& s, int n, int Hq, int T, int window, int sinks, int sms, AttnPlan* a);
// Workspace bytes that hold for every attention call of at most T rows on the cache.
size_t attn_workspace_bound(const kvcache_shape& s, int Hq, int T, int sms);
cudaError_t launch_attention(const AttnCall& p, cudaStream_t st);
cudaError_t launch_own_attention(const AttnCall& p, cudaStream_t st);   // a shared attention's second half

struct WindowCall {
  const __nv_bfloat16* q;        // [B][Hq][n_max][d]
  __nv_bfloat16* out;
  const int32_t* lengths;
  int B, Hq, Hkv, g, d, n_max, window, sinks;
  float scale_log2;
  uint32_t* status;
};
cudaError_t launch_window(const WindowCall& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          int sms, cudaStream_t st);

// What every call on a cache checks; open_cache fills the kernels' view, at the layer.
dropkv_status check_shape(const kvcache_shape* s);
dropkv_status open_cache(const kvcache_shape* s, const kvcache_buffers* b, int32_t layer, int32_t n, uint32_t* status,
                         Cache* c);
inline bool aligned(const void* p, uintptr_t a = 16) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline dropkv_status launched(cudaError_t e) { return e == cudaSuccess ? DROPKV_OK : DROPKV_ERR_CUDA; }

// Allow a kernel its dynamic shared memory on the current device, once per
// device (the setting stays; making it at every launch costs host time).
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};     // devices 0 .. 63
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// ---------------------------------------------------------------- device helpers
__device__ __forceinline__ void flag(uint32_t* status, uint32_t bits) { atomicOr(status, bits); }

// The page scale of values whose largest magnitude is amax (finite, >= 0).
__device__ __forceinline__ float page_scale(float amax, int code) {
  if (code == KVCACHE_INT8) return fmaxf(__fmul_rn(amax, 1.0f / 127.0f), kScaleMin);
  // amax = f 2^E with 1 <= f < 2: 448 = 1.75 * 2^8, so the exponent is E - 8
  // when f <= 1.75, else E - 7 (amax is a bf16 number: below 2^-112 the floor rules)
  const uint32_t b = __float_as_uint(amax);
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(e, -120);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two values already divided by their scale, as two e4m3 codes (round to
// nearest even, saturating; lo in the low byte).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t codes) {
  uint32_t r;
  asm("{.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(r) : "r"(codes));
  return r;
}
__device__ __forceinline__ uint32_t int8_code(float x) {   // x divided by its scale; not-a-number gives 0
  return (uint32_t)min(127, max(-127, __float2int_rn(x))) & 0xFFu;
}

// Two e4m3 codes times a power of two of at most 1, rounded again.  In fp16
// the product is exact, or below 2^-20 and rounds to 0 either way.
__device__ __forceinline__ uint32_t e4m3x2_times(uint32_t codes, uint32_t ratio2) {
  uint32_t h = e4m3x2_to_half2(codes);
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(ratio2));
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}

// Four int8 codes rn(y_i) of numbers y_i that are x_i times a factor, where
// the definition is a division: near[i] = x_i * (rounded factor) is within
// 2^-22 |y_i| < 2^-14 of the definition's value, so both round alike unless
// it lies that close to a half; then `exact(i)` gives the definition's value.
template <typename Exact>
__device__ __forceinline__ uint32_t int8x4_near(const float (&near)[4], Exact exact) {
  constexpr float kMagic = 12582912.f;      // 1.5 2^23: adding it rounds to an integer, in the low bits
  uint32_t w[4];
  bool close = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float t = near[i] + kMagic;
    close |= !(fabsf(near[i] - (t - kMagic)) < 0.4999f) || fabsf(near[i]) > 126.9f;   // (not-a-number too)
    w[i] = __float_as_uint(t);
  }
  if (close) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = int8_code(exact(i));
  }
  return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}

// Four codes (bytes 0..3 of w) as two fp16 pairs (0, 1) and (2, 3).
template <int CODE>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& h01, uint32_t& h23) {
  if constexpr (CODE == KVCACHE_E4M3) {
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(h01), "=r"(h23)
        : "r"(w));
  } else {
    // bytes as the low bits of fp16 1024 + (code + 128), minus 1152: exact
    const uint32_t x = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h01) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h23) : "r"(b), "r"(0x64806480u));
  }
}

// Of 8 bf16 values: the largest bit patterns without sign, low and high
// halves apart; and the largest that is no infinity or not-a-number.
__device__ __forceinline__ uint32_t largest2(const uint4& x) {
  return __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
}
__device__ __forceinline__ uint32_t largest_finite(const uint4& x) {
  const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t lo = w4[q] & 0x7FFFu, hi = (w4[q] >> 16) & 0x7FFFu;
    if (lo < 0x7F80u) m = max(m, lo);
    if (hi < 0x7F80u) m = max(m, hi);
  }
  return m;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// The codes of 8 bf16 values at a scale (inv = 1 / scale: exact for e4m3,
// whose scales are powers of two).
__device__ __forceinline__ uint2 codes8(const uint4& x, float scale, float inv, int code) {
  if (code == KVCACHE_E4M3)
    return make_uint2(e4m3x2(bf_lo(x.x) * inv, bf_hi(x.x) * inv) | (e4m3x2(bf_lo(x.y) * inv, bf_hi(x.y) * inv) << 16),
                      e4m3x2(bf_lo(x.z) * inv, bf_hi(x.z) * inv) | (e4m3x2(bf_lo(x.w) * inv, bf_hi(x.w) * inv) << 16));
  const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
  uint32_t b[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float v[4] = {bf_lo(w4[2 * q]), bf_hi(w4[2 * q]), bf_lo(w4[2 * q + 1]), bf_hi(w4[2 * q + 1])};
    const float near[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
    b[q] = int8x4_near(near, [&](int i) { return __fdiv_rn(v[i], scale); });
  }
  return make_uint2(b[0], b[1]);
}

// Four codes of scale `from` rounded again at scale `to` >= from; ratio =
// from / to.  e4m3 scales are powers of two: their ratio is exact.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float from, float to, float ratio, int code) {
  if (code == KVCACHE_INT8) {
    // a byte as a float: the low bits of 2^23 + (code + 128)
    const uint32_t x = w ^ 0x80808080u;
    float c[4], near[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7650 + i)) - 8388736.f;
      near[i] = c[i] * ratio;
    }
    return int8x4_near(near, [&](int i) { return __fdiv_rn(__fmul_rn(c[i], from), to); });
  }
  const __half2 r2 = __float2half2_rn(ratio);
  const uint32_t r = *reinterpret_cast<const uint32_t*>(&r2);
  return e4m3x2_times(w & 0xFFFFu, r) | (e4m3x2_times(w >> 16, r) << 16);
}

}  // namespace kvcache
