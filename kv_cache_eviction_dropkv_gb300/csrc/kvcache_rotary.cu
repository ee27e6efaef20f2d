// Norm and rotation of queries and keys, alone (rotate_kernel) and with the
// store of the keys and values (rotate_store_kernel).
//
//   y = x rsqrt(mean(x^2) + eps) w,   (y_a, y_b) <- A (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
//
// Both are bound by memory: each row is read once and written once, and the
// rest has to stay under that (a 32K prompt of 32 and 8 heads of 128 in 106 us,
// 6.3 TB/s, 95 % of a copy).  A row of d <= 128 channels belongs to 16 lanes
// (8 where d <= 64), 8 channels to a lane: channels that turn together are
// always one lane's, so the rotation needs no exchange and the norm one sum
// over the row's lanes.  With pairs (i, i + dims / 2) a lane has 4 channels of
// either half and moves 8 bytes at a time, the other channels and the other
// pairing are 8 adjacent ones.
//
// Angles: a position times 2^-64 turns, modulo a turn, is the low 64 bits of
// one integer product, so no position is too far.  The nearest quarter turn
// comes off in integers too; what is left is at most an eighth of a turn and
// goes through the Taylor series of sine and cosine in turns (terms left out
// below 2^-29; the results are within 1.3 2^-24, which the hardware's own sine
// and cosine, 2^-20 off with their argument, are not: with those, five times
// as many keys came out of the rounding to bf16 as a neighbour of the value
// that 64 bits give).
#include "kvcache_step_internal.cuh"
#include "sm103_ptx.cuh"

namespace kvcache {
namespace {

using dropkv::grid_dep_launch;
using dropkv::grid_dep_wait;
using dropkv::f2_fma;
using dropkv::f2_hi;
using dropkv::f2_lo;
using dropkv::f2_mul;
using dropkv::f2_pack;
using dropkv::launch_pdl;

// The 8 channels of a lane, as two runs of 4: [c0, c0 + 4), [c1, c1 + 4).
struct Part {
  int c0, c1;
  bool live, turns;              // it has channels; they turn
};
__device__ __forceinline__ Part part_of(const Turning& how, int lane, bool half) {
  Part a;
  a.live = lane * 8 < how.d;
  a.turns = lane * 8 < how.dims;
  a.c0 = half && a.turns ? 4 * lane : 8 * lane;
  a.c1 = half && a.turns ? how.dims / 2 + 4 * lane : 8 * lane + 4;
  return a;
}
// Cosines and sines, times the amplitude, of a lane's four pairs at a position,
// two by two.
struct Angle {
  uint64_t c[2], s[2];
  bool turns;
};
__device__ __forceinline__ void cos_sin_turns(unsigned long long t, float& c, float& s) {
  const uint32_t top = (uint32_t)(t >> 32), q = (top + 0x20000000u) >> 30;
  const float u = __fmul_rn((float)(int)(top - (q << 30)), 0x1p-32f), z = __fmul_rn(u, u);   // |u| <= 1/8 turn
  // sin(2 pi u) = u (2 pi - (2 pi)^3 u^2 / 6 + ...), 2 pi as a sum of two numbers
  float a = __fmaf_rn(z, 42.058693f, -76.70586f);
  a = __fmaf_rn(z, a, 81.60525f);
  a = __fmaf_rn(z, a, -41.3417f);
  a = __fmaf_rn(z, a, -1.7484555e-7f);
  a = __fmaf_rn(u, 6.2831855f, __fmul_rn(u, a));
  float b = __fmaf_rn(z, -26.426256f, 60.24464f);
  b = __fmaf_rn(z, b, -85.45682f);
  b = __fmaf_rn(z, b, 64.93939f);
  b = __fmaf_rn(z, b, -19.739208f);
  b = __fmaf_rn(z, b, 1.f);
  // quarter turns: (c, s) -> (-s, c)
  const float x = q & 1 ? a : b, y = q & 1 ? b : a;
  c = (q + 1) & 2 ? -x : x;
  s = q & 2 ? -y : y;
}
__device__ __forceinline__ Angle angle_of(const Turning& how, const Part& a, int lane, long long position) {
  Angle r;
  r.turns = a.turns;
  float c[4], s[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c[e] = s[e] = 0.f;
    if (a.turns) cos_sin_turns((unsigned long long)position * __ldg(how.turns + 4 * lane + e), c[e], s[e]);
  }
  const uint64_t amplitude = f2_pack(how.amplitude, how.amplitude);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    r.c[e] = f2_mul(f2_pack(c[2 * e], c[2 * e + 1]), amplitude);
    r.s[e] = f2_mul(f2_pack(s[2 * e], s[2 * e + 1]), amplitude);
  }
  return r;
}
__device__ __forceinline__ long long position_of(const int32_t* positions, int each, int i, int rows, int t, int first) {
  return !positions ? (long long)first + t : each ? positions[(size_t)i * rows + t] : (long long)positions[i] + t;
}

// A lane's 8 numbers two by two, so that packed arithmetic does the rotation:
// first and second members of pairs 0 and 1, then of pairs 2 and 3.
//   half:         (x0, x1), (x4, x5);  (x2, x3), (x6, x7)     of its two runs x0 .. x3, x4 .. x7
//   interleaved:  (x0, x2), (x1, x3);  (x4, x6), (x5, x7)
struct Pairs {
  uint64_t a[2], b[2];
};
template <bool HALF>
__device__ __forceinline__ Pairs pairs_of(const float (&x)[8]) {
  Pairs p;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    p.a[e] = HALF ? f2_pack(x[2 * e], x[2 * e + 1]) : f2_pack(x[4 * e], x[4 * e + 2]);
    p.b[e] = HALF ? f2_pack(x[4 + 2 * e], x[5 + 2 * e]) : f2_pack(x[4 * e + 1], x[4 * e + 3]);
  }
  return p;
}
template <bool HALF>
__device__ __forceinline__ Pairs weight_of(const float* w, const Part& a) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = w && a.live ? __ldg(w + (e < 4 ? a.c0 + e : a.c1 + e - 4)) : 1.f;
  return pairs_of<HALF>(x);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A lane's part of a row through norm and rotation, rounded to bf16 (words in
// the order of its channels).  All L lanes of the row call it.  The operations
// are spelt out so that both kernels round alike, and packed two by two.
template <bool HALF, int L>
__device__ __forceinline__ uint4 turn(const uint4& raw, bool norm, const Pairs& w, const Angle& g, const Turning& how) {
  const uint32_t w4[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf_lo(w4[i]);
    x[2 * i + 1] = bf_hi(w4[i]);
  }
  Pairs y = pairs_of<HALF>(x);
  if (norm) {
    auto sum_squares = [&](const Pairs& v) {
      uint64_t s2 = f2_mul(v.a[0], v.a[0]);
      s2 = f2_fma(v.a[1], v.a[1], s2);
      s2 = f2_fma(v.b[0], v.b[0], s2);
      s2 = f2_fma(v.b[1], v.b[1], s2);
      float ss = __fadd_rn(f2_lo(s2), f2_hi(s2));
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
      return ss;
    };
    const float mean = __fmaf_rn(sum_squares(y), how.inv_d, how.eps);
    float r = rsqrtf(mean);
    // past fp32 (elements above 2^63, or an eps near its end): once more at 2^-80.
    // (All lanes: the row's own sum decides.)
    if (__any_sync(0xffffffffu, mean == INFINITY)) {
      const uint64_t down = f2_pack(0x1p-80f, 0x1p-80f);
      Pairs z;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        z.a[e] = f2_mul(y.a[e], down);
        z.b[e] = f2_mul(y.b[e], down);
      }
      const float small = __fmaf_rn(sum_squares(z), how.inv_d, __fmul_rn(__fmul_rn(how.eps, 0x1p-80f), 0x1p-80f));
      if (mean == INFINITY) r = __fmul_rn(rsqrtf(small), 0x1p-80f);
    }
    const uint64_t r2 = f2_pack(r, r);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      y.a[e] = f2_mul(f2_mul(y.a[e], r2), w.a[e]);
      y.b[e] = f2_mul(f2_mul(y.b[e], r2), w.b[e]);
    }
  }
  if (g.turns) {                              // (0 times an infinity of a channel that does not turn would be none)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint64_t a = y.a[e], b = y.b[e], minus = b ^ 0x8000000080000000ull;
      y.a[e] = f2_fma(a, g.c[e], f2_mul(minus, g.s[e]));
      y.b[e] = f2_fma(b, g.c[e], f2_mul(a, g.s[e]));
    }
  }
  if (HALF)
    return make_uint4(pack_bf16(f2_lo(y.a[0]), f2_hi(y.a[0])), pack_bf16(f2_lo(y.a[1]), f2_hi(y.a[1])),
                      pack_bf16(f2_lo(y.b[0]), f2_hi(y.b[0])), pack_bf16(f2_lo(y.b[1]), f2_hi(y.b[1])));
  return make_uint4(pack_bf16(f2_lo(y.a[0]), f2_lo(y.b[0])), pack_bf16(f2_hi(y.a[0]), f2_hi(y.b[0])),
                    pack_bf16(f2_lo(y.a[1]), f2_lo(y.b[1])), pack_bf16(f2_hi(y.a[1]), f2_hi(y.b[1])));
}

// `at`: the lane's first channel c0; `apart`: c1 - c0.
template <bool HALF>
__device__ __forceinline__ uint4 load_part(const __nv_bfloat16* at, int apart) {
  if (!HALF) return __ldcs(reinterpret_cast<const uint4*>(at));
  const uint2 lo = __ldcs(reinterpret_cast<const uint2*>(at)), hi = __ldcs(reinterpret_cast<const uint2*>(at + apart));
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}
template <bool HALF>
__device__ __forceinline__ void store_part(__nv_bfloat16* at, int apart, const uint4& x) {
  if (!HALF) {
    *reinterpret_cast<uint4*>(at) = x;
  } else {
    *reinterpret_cast<uint2*>(at) = make_uint2(x.x, x.y);
    *reinterpret_cast<uint2*>(at + apart) = make_uint2(x.z, x.w);
  }
}

constexpr int kBatch = 4;                       // heads whose loads are in flight together

// One token's rows of `mine` heads, `from` and `to` the lane's part of the
// first.  All lanes of the warp walk `heads`, the most any has, a batch's loads
// ahead of its work: the first one's are made by load_heads before the angles
// are computed.
// (Addresses go along by a step each: with a product per head and access the
// kernel issued 170 instructions a row of two tokens instead of 132, and was
// bound by that: 32K prompt 117 -> 106 us.)
template <int N>
struct Batch {
  uint4 x[N];
};
template <bool HALF, int N>
__device__ __forceinline__ Batch<N> load_heads(const __nv_bfloat16*& from, long long step, int mine, int apart) {
  Batch<N> b;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    b.x[u] = make_uint4(0, 0, 0, 0);
    if (u < mine) b.x[u] = load_part<HALF>(from, apart);
    from += step;
  }
  return b;
}
template <bool HALF, int L, int N>
__device__ __forceinline__ void turn_heads(Batch<N> x, const __nv_bfloat16* from, long long from_step, __nv_bfloat16* to,
                                           long long to_step, int heads, int mine, bool norm, const Pairs& w,
                                           const Angle& g, int apart, const Turning& how) {
#pragma unroll 1
  for (;;) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (u >= heads) break;
      x.x[u] = turn<HALF, L>(x.x[u], norm, w, g, how);
      if (u < mine) store_part<HALF>(to, apart, x.x[u]);
      to += to_step;
    }
    heads -= N;
    mine -= N;
    if (heads <= 0) break;
    x = load_heads<HALF, N>(from, from_step, mine, apart);
  }
}

// Most heads a CTA of rotate_kernel takes (8 and 16: 32K prompt 117 and 124 us;
// a batch's loads under the work of the one before, which costs a fifth of the
// threads that fit: 127).  In the store, of a chunk's queries, a token's lanes
// take up to 32, eight loads in flight (its CTAs are few to an SM), and a CTA 4
// of the KV heads, one after the other.  Four chunks of up to 8192 tokens with 32
// and 8 heads: 16 and 32 query heads 97 and 92 us, batches of 4 and 8 heads 88 and
// 87, 2, 4 and 8 KV heads 91, 87 and 100.
constexpr int kRotThreads = 256, kMostHeads = 8;
constexpr int kStoreHeads = 32, kStoreBatch = 8, kStoreKvHeads = 4;

// A CTA takes kRotThreads / L tokens (adjacent rows, so that a head's rows are
// one piece of memory) and `chunk` heads of either the queries or the keys:
// angles and weights are computed once per token and chunk.
template <bool HALF, int L>
__global__ void __launch_bounds__(kRotThreads, 5) rotate_kernel(const RotateCall p) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % L;
  const uint32_t token = blockIdx.x * (kRotThreads / L) + threadIdx.x / L;   // (up to 2^31 + 30)
  const int b = token / (uint32_t)p.n, t = token - (uint32_t)b * p.n;
  const int which = (int)blockIdx.y >= p.chunks ? 1 : 0;
  const int h0 = ((int)blockIdx.y - (which ? p.chunks : 0)) * p.chunk;
  const int heads = min(p.chunk, p.heads[which] - h0);
  const Part a = part_of(p.how, lane, HALF);
  const bool norm = p.weight[which] != nullptr;
  bool live = b < p.B;
  if (live && p.lengths) {
    const int len = p.lengths[b];
    if (len < 0 || len > p.n) {
      if (t == 0 && lane == 0 && h0 == 0) flag(p.status, DROPKV_FLAG_BAD_LENGTH);
      live = false;
    } else {
      live = t < len;
    }
  }
  if (!__any_sync(0xffffffffu, live)) return;
  const Rows& in = p.in[which];
  const int mine = live && a.live ? heads : 0, apart = a.c1 - a.c0;
  const __nv_bfloat16* from = in.p + (mine > 0 ? b * in.seq + t * in.row + h0 * in.head + a.c0 : 0);
  const Batch<kBatch> x = load_heads<HALF, kBatch>(from, in.head, mine, apart);
  const Pairs w = weight_of<HALF>(p.weight[which], a);
  const Angle g = angle_of(p.how, a, lane, live ? position_of(p.positions, p.each, b, p.n, t, 0) : 0);
  const long long to_step = (long long)p.n * p.how.d;
  __nv_bfloat16* to =
      p.out[which] + (mine > 0 ? ((long long)b * p.heads[which] + h0) * to_step + (long long)t * p.how.d + a.c0 : 0);
  turn_heads<HALF, L>(x, from, in.head, to, to_step, heads, mine, norm, w, g, apart, p.how);
}

__device__ __forceinline__ void prefetch_l2(const void* at) { asm volatile("prefetch.global.L2 [%0];" ::"l"(at)); }

// As store_kernel: a CTA holds one (page, head) of K or V in registers, so its
// largest magnitude is known before any code is written; the rows are laid out
// over lanes as above, and K goes through norm and rotation on the way in.  Of
// many new tokens it takes several heads one after the other, the angles of its
// rows kept in shared memory (a thread's own; four chunks of up to 8192 tokens
// with 32 and 8 heads of 128: 114 -> 103 us when it came; 87 now, 4.8 TB/s, the
// floor is 62: 18 to 20 warps an SM hide no more of the loads).
// Further CTAs of an entry take its queries: L lanes one token's of q_chunk
// heads, so that the angles (as much work as a row's norm and rotation) are
// computed once for all of them.
// (Four threads per token of the page instead of two, with half the registers
// each: the same 114 us for four chunks of up to 8192 tokens, and 9.1 instead of
// 7.6 for a step of 64 single ones.)
template <int PAGE, bool HALF, int L>
__global__ void __launch_bounds__(PAGE * 2) rotate_store_kernel(const RotateStoreCall p) {
  constexpr int kThreads = PAGE * 2, kWarps = kThreads / 32, kPer = kThreads / L, kPasses = PAGE / kPer;
  grid_dep_wait();
  grid_dep_launch();
  __shared__ uint32_t s_max[kWarps];
  extern __shared__ ulonglong2 s_angle[];   // a thread's own: [pass][cosines, sines][thread]
  const Cache& c = p.c;
  const int tid = threadIdx.x, lane = tid % L, group = tid / L;
  const int i = blockIdx.z;
  const int cnt = p.counts ? p.counts[i] : p.rows;
  const int shares = (c.Hkv + p.kv_heads - 1) / p.kv_heads, store_ctas = p.touched * 2 * shares;
  // the grid covers `rows`: CTAs behind the entry's tokens end on one load (its
  // first CTA tells what is wrong with the entry)
  if (cnt >= 0 && cnt <= p.rows && blockIdx.x > 0) {
    const int x = blockIdx.x, ahead = (x >> 1) / shares;   // pages between the first token's and this CTA's
    if (x < store_ctas ? ahead > 0 && (long long)(ahead - 1) * PAGE + 1 >= cnt
                       : ((x - store_ctas) * kPer) % p.rows >= cnt && (x - store_ctas) * kPer % p.rows + kPer <= p.rows)
      return;
  }
  const int s = p.seqs ? p.seqs[i] : i;
  bool again = false;                       // the sequence was named before: that entry stores it
  if (p.seqs)
    for (int j = tid; j < i; j += kThreads) again |= p.seqs[j] == s;
  const bool dup = p.seqs ? __syncthreads_or(again) : false;
  if (s < 0 || s >= c.S || dup) {
    if (tid == 0) flag(c.status, KVCACHE_FLAG_BAD_SEQ);
    return;
  }
  const int len = c.length[s], held = c.count[s];
  if (cnt < 0 || cnt > p.rows || cnt > len || held < 0 || held > c.M || (long long)len > (long long)held * PAGE) {
    if (tid == 0) flag(c.status, DROPKV_FLAG_BAD_LENGTH);
    return;
  }
  const int start = len - cnt;
  if ((int)blockIdx.x >= store_ctas) {
    const int item = ((int)blockIdx.x - store_ctas) * kPer + group;
    const int row = item % p.rows, h0 = item / p.rows * p.q_chunk;
    const Part a = part_of(p.how, lane, HALF);
    const int own = row < cnt ? max(0, min(p.q_chunk, p.Hq - h0)) : 0, heads = __reduce_max_sync(0xffffffffu, own);
    if (heads == 0) return;
    const int mine = a.live ? own : 0, apart = a.c1 - a.c0;
    const __nv_bfloat16* from = p.q.p + (mine > 0 ? i * p.q.seq + row * p.q.row + h0 * p.q.head + a.c0 : 0);
    const Batch<kStoreBatch> x = load_heads<HALF, kStoreBatch>(from, p.q.head, mine, apart);
    const Pairs w = weight_of<HALF>(p.q_weight, a);
    const Angle g = angle_of(p.how, a, lane, position_of(p.positions, p.each, i, p.rows, row, start));
    const long long to_step = (long long)p.rows * p.how.d;
    __nv_bfloat16* to =
        p.q_out + (mine > 0 ? ((long long)i * p.Hq + h0) * to_step + (long long)row * p.how.d + a.c0 : 0);
    turn_heads<HALF, L>(x, from, p.q.head, to, to_step, heads, mine, p.q_weight != nullptr, w, g, apart, p.how);
    return;
  }
  const int which = blockIdx.x & 1, h0 = ((int)blockIdx.x >> 1) % shares * p.kv_heads, h1 = min(h0 + p.kv_heads, c.Hkv);
  const int col = start / PAGE + ((int)blockIdx.x >> 1) / shares;
  if (cnt == 0 || col > (len - 1) / PAGE) return;
  const int base = col * PAGE;              // first token of the page
  const int r0 = max(0, start - base), r1 = min(PAGE, len - base);   // slots of the new tokens
  const int pg = c.table[(size_t)s * c.M + col];
  // the values' lanes have 8 adjacent channels, which do not turn
  Part a = part_of(p.how, lane, HALF);
  if (which) {
    a.c0 = 8 * lane;
    a.c1 = a.c0 + 4;
    a.turns = false;
  }
  const Rows& in = p.kv[which];
  // the lane's part of the first of its group's rows, and how many of them are new
  const int mine = a.live ? max(0, (r1 - r0 - group + kPer - 1) / kPer) : 0, apart = a.c1 - a.c0;
  const __nv_bfloat16* first =
      in.p + (mine > 0 ? i * in.seq + ((long long)base - start + r0 + group) * in.row + a.c0 : 0);
  // a head's rows on their way to L2 while something else is worked out (four
  // chunks of up to 8192 tokens: 90 -> 86 us)
  auto ahead = [&](int h) {
    const __nv_bfloat16* at = first + h * in.head;
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      if (u < mine) {
        prefetch_l2(at);
        if (HALF) prefetch_l2(at + apart);
      }
      at += kPer * in.row;
    }
  };
  if (!which) {
    ahead(h0);
    // the angles of the thread's rows, for all its heads
#pragma unroll 1
    for (int u = 0; r0 + group + u * kPer < r1; ++u) {
      const Angle g = angle_of(p.how, a, lane, position_of(p.positions, p.each, i, p.rows, base + r0 + group + u * kPer - start, start));
      s_angle[(2 * u) * kThreads + tid] = make_ulonglong2(g.c[0], g.c[1]);
      s_angle[(2 * u + 1) * kThreads + tid] = make_ulonglong2(g.s[0], g.s[1]);
    }
  }
  if (pg < 0 || pg >= c.P || c.refs[pg] != 1) {
    if (tid == 0) flag(c.status, KVCACHE_FLAG_BAD_PAGE);
    return;
  }
  const Pairs w = weight_of<HALF>(which ? nullptr : p.k_weight, a);
  float* scales = which ? c.vs : c.ks;
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    uint4 x[kPasses];
    const __nv_bfloat16* src = first + h * in.head;
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      x[u] = make_uint4(0, 0, 0, 0);
      if (u < mine) x[u] = load_part<HALF>(src, apart);
      src += kPer * in.row;
    }
    if (h + 1 < h1) ahead(h + 1);
    const size_t unit = (size_t)pg * c.Hkv + h;
    const float held_scale = r0 > 0 ? scales[unit] : 0.f;
    uint8_t* dst = (which ? c.v : c.k) + unit * PAGE * c.d;
    if (!which) {
#pragma unroll
      for (int u = 0; u < kPasses; ++u) {
        if (r0 + u * kPer >= r1) break;       // (the same for all threads)
        Angle g;
        g.turns = a.turns;
        if (r0 + group + u * kPer < r1) {
          const ulonglong2 cc = s_angle[(2 * u) * kThreads + tid], ss = s_angle[(2 * u + 1) * kThreads + tid];
          g.c[0] = cc.x;
          g.c[1] = cc.y;
          g.s[0] = ss.x;
          g.s[1] = ss.y;
        } else {
          g.c[0] = g.c[1] = g.s[0] = g.s[1] = 0ull;
        }
        x[u] = turn<HALF, L>(x[u], p.k_weight != nullptr, w, g, p.how);
      }
    }
    uint32_t m2 = 0;
#pragma unroll
    for (int u = 0; u < kPasses; ++u) m2 = __vmaxu2(m2, largest2(x[u]));
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
      for (int u = 0; u < kPasses; ++u) m = max(m, largest_finite(x[u]));
      top = block_max(m);
      if (tid == 0) flag(c.status, DROPKV_FLAG_NONFINITE);
    }
    const float scale = fmaxf(page_scale(__uint_as_float(top << 16), c.code), held_scale), inv = 1.0f / scale;
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      if (u < mine) {
        const uint2 o = codes8(x[u], scale, inv, c.code);
        uint8_t* at = dst + (r0 + group + u * kPer) * c.d + a.c0;
        if (HALF) {
          *reinterpret_cast<uint32_t*>(at) = o.x;
          *reinterpret_cast<uint32_t*>(at + apart) = o.y;
        } else {
          *reinterpret_cast<uint2*>(at) = o;
        }
      }
    }
    if (r0 > 0 && scale > held_scale) {       // earlier tokens of the page at the new scale
      const float ratio = held_scale / scale;
      for (int n = tid; n < r0 * (c.d / 8); n += kThreads) {
        uint2 o = *reinterpret_cast<const uint2*>(dst + (size_t)n * 8);
        o.x = rescale4(o.x, held_scale, scale, ratio, c.code);
        o.y = rescale4(o.y, held_scale, scale, ratio, c.code);
        *reinterpret_cast<uint2*>(dst + (size_t)n * 8) = o;
      }
    }
    if (tid == 0) scales[unit] = scale;
  }
}

}  // namespace

cudaError_t launch_rotate(RotateCall p, int sms, cudaStream_t st) {
  const int L = p.how.d <= 64 ? 8 : 16, tokens = kRotThreads / L;
  const long long groups = ((long long)p.B * p.n + tokens - 1) / tokens;
  const int heads[2] = {p.in[0].p ? p.heads[0] : 0, p.in[1].p ? p.heads[1] : 0};
  // as many heads per CTA as leave every SM a few CTAs
  p.chunk = kMostHeads;
  while (p.chunk > 1 && groups * ((heads[0] + p.chunk - 1) / p.chunk + (heads[1] + p.chunk - 1) / p.chunk) < 8LL * sms)
    p.chunk /= 2;
  p.chunks = (heads[0] + p.chunk - 1) / p.chunk;
  const dim3 grid((unsigned)groups, p.chunks + (heads[1] + p.chunk - 1) / p.chunk);
  auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(kRotThreads), 0, st, p); };
  if (L == 8) return p.how.half ? go(rotate_kernel<true, 8>) : go(rotate_kernel<false, 8>);
  return p.how.half ? go(rotate_kernel<true, 16>) : go(rotate_kernel<false, 16>);
}

namespace {
template <int PAGE>
cudaError_t launch_rs(RotateStoreCall p, cudaStream_t st) {
  const int L = p.how.d <= 64 ? 8 : 16, per = 2 * PAGE / L;
  p.touched = (int)(((long long)p.rows + PAGE - 2) / PAGE) + 1;   // most pages `rows` tokens touch
  p.q_chunk = p.rows >= PAGE ? kStoreHeads : 4;
  p.kv_heads = p.rows >= PAGE ? kStoreKvHeads : 1;
  const int q_ctas = p.q.p ? (int)(((long long)((p.Hq + p.q_chunk - 1) / p.q_chunk) * p.rows + per - 1) / per) : 0;
  const dim3 grid((unsigned)(p.touched * 2 * ((p.c.Hkv + p.kv_heads - 1) / p.kv_heads) + q_ctas), 1, p.n);
  constexpr int kMost = 2 * PAGE * 2 * 8 * 16;   // angles of 8 passes (4 where L is 8)
  auto go = [&](auto kern, cudaError_t e) {
    return e != cudaSuccess ? e : launch_pdl(kern, grid, dim3(2 * PAGE), L == 8 ? kMost / 2 : kMost, st, p);
  };
  if (L == 8)
    return p.how.half ? go(rotate_store_kernel<PAGE, true, 8>, allow_smem<rotate_store_kernel<PAGE, true, 8>>(kMost))
                      : go(rotate_store_kernel<PAGE, false, 8>, allow_smem<rotate_store_kernel<PAGE, false, 8>>(kMost));
  return p.how.half ? go(rotate_store_kernel<PAGE, true, 16>, allow_smem<rotate_store_kernel<PAGE, true, 16>>(kMost))
                    : go(rotate_store_kernel<PAGE, false, 16>, allow_smem<rotate_store_kernel<PAGE, false, 16>>(kMost));
}
}  // namespace

cudaError_t launch_rotate_store(RotateStoreCall p, cudaStream_t st) {
  switch (p.c.page) {
    case 32: return launch_rs<32>(p, st);
    case 64: return launch_rs<64>(p, st);
    case 128: return launch_rs<128>(p, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvcache
