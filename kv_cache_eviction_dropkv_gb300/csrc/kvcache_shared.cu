// Attention over the paged 8-bit cache for entries that share pages.
//
// The tokens of a group's shared pages are seen by all its query rows, so for
// each KV head they are one product of M = members * g * T rows with the
// tokens, read once: o_r = sum_j p_rj v_j over shared j, joined with what the
// row's own tokens give by the softmax states of both.  From some 100 rows on
// the shared part is bound by the tensor cores (4 d operations for each row and
// token against 2 d / M bytes), below by memory.
//
// Four kernels in a row:
//   plan_kernel    one cluster finds each group's common pages by comparing the
//                  page tables, and lays out the work
//   prefix_kernel  the shared tokens, on tcgen05; leaves pieces (O, m, l, M)
//   attention_kernel<SHARED> (kvcache_attn.cuh)  each entry's own tokens
//   final_kernel   joins a row's pieces
//
// prefix_kernel.  A unit is (group, KV head, 128 or 256 of its rows); its
// tokens are cut into tiles of 128, the tiles of all units stand in a row, and
// each CTA (one per SM) takes an equal run of them.  The segment of unit u in
// run w leaves its piece at rows 256 w + 2 (rows of the units before u): borders
// of runs and units only move that up, so no index is stored.
//
// Per tile, K and V codes (a page and head lie in one piece) come by bulk copy
// into a staging buffer, four warps turn them into fp16 tiles (both codes are
// exact in fp16; the scales stay outside), in the swizzled layout that the
// matrix instruction reads, and two softmax groups of four warps, a thread per
// row, work as in the windowed prompt's kernel: S = Q K^T in tensor memory,
// P over it in fp16, O += P V with P read from tensor memory.  Units of more
// than 128 rows: both groups take every tile, each for its 128 rows.  Others:
// the groups take the tiles in turn and leave a piece each, so that the tensor
// cores have two independent chains either way.
#include "kvcache_step_internal.cuh"
#include "sm103_ptx.cuh"

namespace kvcache {
namespace {

using namespace dropkv;

// ------------------------------------------------------------------ the plan
constexpr int kPlanThreads = 512;
constexpr int kCols = 128;                       // table entries a warp compares at a time

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ int tiles_of(int tokens) { return (int)(((uint32_t)tokens + 127u) >> 7); }

// The group of entry i (the last that begins at or before it).
__device__ __forceinline__ int group_of(const int32_t* groups, int G, int i) {
  int lo = 0, hi = G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (groups[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const SharedCall p) {
  grid_dep_wait();
  grid_dep_launch();
  const AttnCall& a = p.own;
  const Cache& c = a.c;
  const int threads = kPlanThreads * cluster_ctas(), me = cluster_rank() * kPlanThreads + threadIdx.x;
  const int lane = threadIdx.x & 31;
  __shared__ uint32_t s_sum[kPlanThreads / 32];
  __shared__ int s_most;
  // groups that cover the entries in order
  bool bad = false;
  for (int j = threadIdx.x; j <= p.G; j += kPlanThreads) {
    const int x = p.groups[j];
    bad |= j == 0 ? x != 0 : x < p.groups[j - 1];
    bad |= j == p.G && x != a.n;
  }
  if (__syncthreads_or(bad)) {
    if (me == 0) {
      flag(c.status, DROPKV_FLAG_BAD_LENGTH);
      p.plan->total = 0;
      p.plan->runs = 1;
      p.plan->unit_rows = 128;
    }
    for (int i = me; i < a.n; i += threads) p.from[i] = 0;
    return;
  }
  for (int j = me; j < p.G; j += threads) {
    p.lead[j] = p.prefix[j] = INT_MAX;
    p.active[j] = 0;
  }
  cluster_sync();
  // sequences that hold a full page before the first row's token take part
  for (int i = me; i < a.n; i += threads) {
    const int s = a.seqs ? a.seqs[i] : i, g = group_of(p.groups, p.G, i);
    int bound = 0;
    if (s >= 0 && s < c.S) {
      const int len = c.length[s], held = c.count[s];
      if (len >= a.T && held >= 0 && held <= c.M && (long long)len <= (long long)held << c.page_log2)
        bound = (len - a.T + 1) >> c.page_log2;
    }
    p.bound[i] = bound;
    p.group[i] = g;
    if (bound > 0) {
      atomicMin(p.lead + g, i);
      atomicAdd(p.active + g, 1);
      atomicMin(p.prefix + g, bound);
    }
  }
  cluster_sync();
  const int chunks = (c.M + kCols - 1) / kCols;
  for (long long item = me >> 5; item < (long long)a.n * chunks; item += threads >> 5) {
    const int i = (int)(item / chunks), col0 = (int)(item - (long long)i * chunks) * kCols;
    const int g = p.group[i], end = min(p.prefix[g], col0 + kCols);   // (others may lower it meanwhile: it stays an end)
    if (p.bound[i] == 0 || p.active[g] < 2 || col0 >= end) continue;
    const int lead = p.lead[g];
    const int32_t* mine = c.table + (size_t)(a.seqs ? a.seqs[i] : i) * c.M;
    const int32_t* other = c.table + (size_t)(a.seqs ? a.seqs[lead] : lead) * c.M;
    int differs = INT_MAX;
#pragma unroll
    for (int u = 0; u < kCols / 32; ++u) {
      const int col = col0 + u * 32 + lane;
      if (col >= end) continue;
      const int x = mine[col];
      if (x != other[col] || x < 0 || x >= c.P) differs = min(differs, col);
    }
    differs = __reduce_min_sync(0xffffffffu, differs);
    if (lane == 0 && differs != INT_MAX) atomicMin(p.prefix + g, differs);
  }
  cluster_sync();
  for (int i = me; i < a.n; i += threads) {
    const int g = p.group[i];
    p.from[i] = p.bound[i] > 0 && p.active[g] >= 2 ? p.prefix[g] << c.page_log2 : 0;
  }
  if (cluster_rank() != 0) return;
  // the widest unit, then tiles before each group
  if (threadIdx.x == 0) s_most = 0;
  __syncthreads();
  for (int j = threadIdx.x; j < p.G; j += kPlanThreads)
    if (p.active[j] >= 2 && p.prefix[j] > 0) atomicMax(&s_most, (p.groups[j + 1] - p.groups[j]) * a.R);
  __syncthreads();
  const int unit_rows = s_most > 128 ? 256 : 128;
  uint32_t before = 0;
  for (int j0 = 0; j0 < p.G; j0 += kPlanThreads) {
    const int j = j0 + threadIdx.x;
    uint32_t tiles = 0;
    if (j < p.G && p.active[j] >= 2 && p.prefix[j] > 0)
      tiles = (uint32_t)tiles_of(p.prefix[j] << c.page_log2) * c.Hkv *
              (((p.groups[j + 1] - p.groups[j]) * a.R + unit_rows - 1) / unit_rows);
    uint32_t sum = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) s_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    uint32_t all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < (int)threadIdx.x >> 5) sum += s_sum[w];
      all += s_sum[w];
    }
    if (j < p.G) p.first[j] = before + sum - tiles;
    before += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    p.first[p.G] = before;
    p.plan->total = before;
    p.plan->runs = max(1u, min((uint32_t)p.sms, before / 2));
    p.plan->unit_rows = unit_rows;
  }
}

// ------------------------------------------------------------------ the layout of the work
// Run w's tiles begin at run_start(w).
__device__ __forceinline__ uint32_t run_start(const SharedPlan& q, uint32_t w) {
  const uint32_t share = q.total / q.runs;
  return w * share + min(w, q.total - share * q.runs);
}
__device__ __forceinline__ uint32_t run_of(const SharedPlan& q, uint32_t x) {
  const uint32_t share = q.total / q.runs, more = q.total - share * q.runs, cut = more * (share + 1);
  return x < cut ? x / (share + 1) : more + (x - cut) / share;
}
// The part of a unit that a run holds.
struct Segment {
  int g, h, row0, rows;                           // group, KV head, its rows [row0, row0 + rows)
  int lead, entry0;                               // a sequence that holds the pages, first entry of the group
  int tokens;                                     // shared tokens of the group
  int k0, n;                                      // first tile and tiles
  long long before;                               // rows of the units before this one
  __device__ __forceinline__ bool wide() const { return rows > 128; }
};
__device__ __forceinline__ Segment segment_at(const SharedCall& p, int unit_rows, uint32_t x, uint32_t end) {
  Segment s;
  int lo = 0, hi = p.G;                           // the group with first[g] <= x < first[g + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (p.first[mid] <= x) lo = mid;
    else hi = mid;
  }
  s.g = lo;
  s.entry0 = p.groups[lo];
  const int M = (p.groups[lo + 1] - s.entry0) * p.own.R, per_head = (M + unit_rows - 1) / unit_rows;
  s.tokens = p.prefix[lo] << p.own.c.page_log2;
  const int tiles = tiles_of(s.tokens);
  const uint32_t rel = x - p.first[lo], u = rel / (uint32_t)tiles;
  s.k0 = (int)(rel - u * tiles);
  s.n = (int)min((uint32_t)(tiles - s.k0), end - x);
  s.h = u / (uint32_t)per_head;
  s.row0 = (int)(u - (uint32_t)s.h * per_head) * unit_rows;
  s.rows = min(unit_rows, M - s.row0);
  s.before = (long long)s.entry0 * p.own.R * p.own.c.Hkv + (long long)s.h * M + s.row0;
  const int lead = p.lead[lo];
  s.lead = p.own.seqs ? p.own.seqs[lead] : lead;
  return s;
}

// ------------------------------------------------------------------ the shared tokens
constexpr int kTile = 128;
constexpr int kConvert = 8, kIssuer = 12, kLoader = 13, kThreads = 32 * 14;   // warps 0 .. 7: softmax
constexpr float kMoveLog2 = 8.0f, kLiftLog2 = 7.0f;   // as in kvcache_attn.cuh: P <= 2^15 in fp16
constexpr float kLowLog2 = -60.0f;                // least exponent of the factor of P: below it P is 0 in fp16 anyway
constexpr uint64_t kDrain = 20000000ull;          // 20 ms to drain copies after an abort
constexpr int kMaxStages = 5, kMeta = 8;           // kMeta >= kMaxStages + 2

template <int DS>
struct Layout {                                   // DS: steps of 16 channels
  static constexpr int kDP = DS <= 4 ? 64 : 128;
  static constexpr int kTileB = kTile * kDP * 2, kBlockB = kTile * 128;   // fp16 tile, its blocks of 64 columns
  static constexpr int kStageB = 2 * kTile * kDP;                          // codes: K, then V
  static constexpr int kStages = DS <= 4 ? 4 : 1;                          // and one more in the place of the second Q
  static constexpr int kQ = 0, kK = 2 * kTileB, kV = 4 * kTileB, kStage = 6 * kTileB;
  static constexpr int kSmall = kStage + kStages * kStageB;
};

struct Scales {                                   // of a tile's four blocks of 32 tokens
  float ks[4], lv[4];                             // K scale, log2 of the V scale
};
struct Small {
  uint64_t sk_full[kMaxStages], sk_empty[kMaxStages], sv_full[kMaxStages], sv_empty[kMaxStages];   // codes
  uint64_t kf_full[2], kf_empty[2], vf_full[2], vf_empty[2];                                       // fp16 tiles
  uint64_t meta_full[kMeta];
  uint64_t q_full[2], q_free;      // group g's Q written; both groups' last S of a segment complete
  uint64_t s_full[2], p_full[2][2], o_done[2], drain;
  Scales meta[kMeta];
  uint32_t tmem_base;
  int abort;
};
template <int DS>
constexpr int kSmem = Layout<DS>::kSmall + (int)sizeof(Small) + 1024;
static_assert(kSmem<8> <= 232448 && kSmem<4> <= 232448, "shared memory exceeds the per-CTA limit");

__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(pred));
  return pred != 0;
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 0; it < (1u << 26) && !mbar_try_wait(bar, parity); ++it)
    if (global_timer_ns() - t0 > kDrain) break;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
constexpr uint32_t idesc_f16(uint32_t N, uint32_t b_mn) {   // both operands fp16 (format 0), fp32 accumulators, M = 128
  return (1u << 4) | (b_mn << 16) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}

// Codes of a tile (row pitch d bytes) as fp16 in the swizzled layout; rows from
// `tokens` on are zero.  128 threads, t of them.
template <int CODE, int DS>
__device__ __forceinline__ void convert_tile(const uint8_t* from, uint8_t* to, int d, int tokens, int t) {
  constexpr int kBlockB = Layout<DS>::kBlockB;
  auto chunk = [&](int r, int ch) {               // 16-byte chunk ch of row r
    return reinterpret_cast<uint4*>(to + (ch >> 3) * kBlockB + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
  };
  if (d == 16 * DS) {
    constexpr int kBatch = DS % 4 == 0 ? 4 : 3;
#pragma unroll
    for (int it0 = 0; it0 < DS; it0 += kBatch) {
      uint4 w[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int x = t + 128 * (it0 + u);
        w[u] = x / DS < tokens ? *reinterpret_cast<const uint4*>(from + 16 * x) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int x = t + 128 * (it0 + u), r = x / DS, c = x % DS;
        uint4 lo, hi;
        codes_to_half<CODE>(w[u].x, lo.x, lo.y);
        codes_to_half<CODE>(w[u].y, lo.z, lo.w);
        codes_to_half<CODE>(w[u].z, hi.x, hi.y);
        codes_to_half<CODE>(w[u].w, hi.z, hi.w);
        // lanes of the second block of columns begin with the odd chunk: all banks at once
        const bool swap = c & 4;
        *chunk(r, 2 * c + swap) = swap ? hi : lo;
        *chunk(r, 2 * c + !swap) = swap ? lo : hi;
      }
    }
  } else {
    const int per = d >> 3;
    for (int x = t; x < kTile * per; x += 128) {
      const int r = x / per, c = x - r * per;
      const uint2 w = r < tokens ? *reinterpret_cast<const uint2*>(from + 8 * x) : make_uint2(0, 0);
      uint4 v;
      codes_to_half<CODE>(w.x, v.x, v.y);
      codes_to_half<CODE>(w.y, v.z, v.w);
      *chunk(r, c) = v;
    }
  }
}

// 32 columns of the thread's row; read them behind wait_ld32.
__device__ __forceinline__ void ld32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
// (The values pass through, so that nothing that uses them comes before.)
__device__ __forceinline__ void wait_ld32(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                 "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}

// A thread's row of a tile: S in its columns of tensor memory becomes P.
//   x_c = s f_c (base-2 logits; f_c: the row's factor times block c's K scale),
//   P = 2^(x - m + e_c), e_c = lv_c + m - M + 7,  l += sum of 2^(x - m)
// m and M are references of the sums and of the outputs (which carry the V
// scales); they move only when a tile's maximum is 2^8 above, so P <= 2^15.
// follow(factor) lets O follow M, half() says that P's first half is stored.
template <typename Follow, typename Half>
__device__ __forceinline__ void softmax_tile(uint32_t tS, const Scales& scales, int blocks, float fq, float& m, float& M,
                                             float& l, Follow follow, Half half) {
  float f[4], lv[4], v[2][32];
  float mt = -INFINITY, Mt = -INFINITY;
  ld32(tS, v[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    f[c] = fmaxf(fq * scales.ks[c], 0x1p-126f);
    lv[c] = scales.lv[c];
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    wait_ld32(v[c & 1]);
    ld32(tS + 32 * ((c + 1) & 3), v[(c + 1) & 1]);         // (after the last block, the first again)
    float m4[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) m4[u] = v[c & 1][u];
#pragma unroll
    for (int u = 4; u < 32; ++u) m4[u & 3] = fmaxf(m4[u & 3], v[c & 1][u]);
    if (c < blocks) {
      const float x = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * f[c];
      mt = fmaxf(mt, x);
      Mt = fmaxf(Mt, x + lv[c]);
    }
  }
  const bool need = mt > m + kMoveLog2 || Mt > M + kMoveLog2;
  if (__any_sync(0xffffffffu, need)) {
    const float mn = mt > m + kMoveLog2 ? mt : m, Mn = Mt > M + kMoveLog2 ? Mt : M;
    l *= m == mn ? 1.f : ex2_approx(m - mn);               // (from nothing: 0 times 0)
    const float factor = M == Mn ? 1.f : ex2_approx(M - Mn);
    m = mn;
    M = Mn;
    // the first block waits in registers meanwhile
    wait_ld32(v[0]);
    follow(factor);
  }
  float hw[32];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    wait_ld32(v[c & 1]);
    if (c < 3) ld32(tS + 32 * (c + 1), v[(c + 1) & 1]);
    const float e = fmaxf(lv[c] + m - M + kLiftLog2, kLowLog2);
    const uint64_t f2 = f2_pack(f[c], f[c]), n2 = f2_pack(e - m, e - m);
    uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
    for (int u = 0; u < 32; u += 2) {
      uint64_t y = f2_fma(f2_pack(v[c & 1][u], v[c & 1][u + 1]), f2, n2);
      if (c >= blocks) y = f2_pack(-INFINITY, -INFINITY);
      const float a = ex2_approx(f2_lo(y)), b = ex2_approx(f2_hi(y));
      sum2[(u >> 1) & 1] = f2_add(sum2[(u >> 1) & 1], f2_pack(a, b));
      hw[(c & 1) * 16 + u / 2] = __uint_as_float(pack_half2(a, b));
    }
    const uint64_t sum = f2_add(sum2[0], sum2[1]);
    l += (f2_lo(sum) + f2_hi(sum)) * ex2_approx(-e);
    tmem_st16(tS + 16 * c, hw + (c & 1) * 16);
    if (c == 1) half();
  }
}

// A value all lanes of the converged warp hold, in a uniform register.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

template <int DS>
__device__ __forceinline__ void softmax_group(const SharedCall& p, Small& S, uint8_t* sm, uint32_t tmem, int warp,
                                              int lane, int unit_rows, uint32_t x0, uint32_t x1) {
  using L = Layout<DS>;
  const AttnCall& a = p.own;
  const int gi = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane, d = a.c.d;
  const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
  const uint32_t tS = tmem + lane_base + 128 * gi, tO = tmem + lane_base + 256 + 128 * gi;
  auto give_up = [&]() {
    if (lane == 0) {
      S.abort = 1;
      atomicOr(a.c.status, DROPKV_FLAG_TIMEOUT);
    }
  };
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, &S.abort));
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    __syncwarp();
  };
  // The thread's query row as fp16 into its place in shared memory (`write`),
  // times a power of two that brings its largest element to [2^14, 2^15);
  // returns the factor of its logits.
  auto load_q = [&](const Segment& s, bool write) {
    const int r = (s.wide() ? gi * 128 : 0) + row;
    uint4 w[2 * DS];
#pragma unroll
    for (int u = 0; u < 2 * DS; ++u) w[u] = make_uint4(0, 0, 0, 0);
    if (r < s.rows) {
      const int y = s.row0 + r, member = y / a.R, rr = y - member * a.R;
      const __nv_bfloat16* q = a.q + (((size_t)(s.entry0 + member) * a.Hq + (size_t)s.h * a.g) * a.T + rr) * d;
#pragma unroll
      for (int u = 0; u < 2 * DS; ++u)
        if (8 * u < d) w[u] = *reinterpret_cast<const uint4*>(q + 8 * u);
    }
    uint32_t m2 = 0;
#pragma unroll
    for (int u = 0; u < 2 * DS; ++u) m2 = __vmaxu2(m2, largest2(w[u]));
    const int e = min(126, max(-113, 14 - ((int)(max(m2 & 0xFFFFu, m2 >> 16) >> 7) - 127)));
    const float up = __uint_as_float((uint32_t)(e + 127) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
    if (write) {
      uint8_t* to = sm + L::kQ + (s.wide() ? gi * L::kTileB : 0) + row * 128;
#pragma unroll
      for (int u = 0; u < 2 * DS; ++u)
        *reinterpret_cast<uint4*>(to + (u >> 3) * L::kBlockB + (((u & 7) ^ (row & 7)) << 4)) =
            make_uint4(pack_half2(bf_lo(w[u].x) * up, bf_hi(w[u].x) * up), pack_half2(bf_lo(w[u].y) * up, bf_hi(w[u].y) * up),
                       pack_half2(bf_lo(w[u].z) * up, bf_hi(w[u].z) * up), pack_half2(bf_lo(w[u].w) * up, bf_hi(w[u].w) * up));
      fence_proxy_async_smem();
      arrive(&S.q_full[gi]);
    }
    return down * a.scale_log2;
  };

  uint32_t tile0 = 0, mine = 0, outputs = 0, segments = 0;
  Segment s = segment_at(p, unit_rows, x0, x1);
  float fq = load_q(s, gi == 0 || s.wide());
  for (uint32_t x = x0;;) {
    const int n = uniform(s.n), step = s.wide() ? 1 : 2, start = s.wide() ? 0 : gi;
    float m = -INFINITY, M = -INFINITY, l = 0.f;
    if (start >= n) {
      // no tile for this group; its word still counts for this segment's Q, so
      // it waits for that (a group that ran ahead would give the next one's)
      if (!wait(&S.q_full[0], segments)) { give_up(); return; }
      arrive(&S.q_free);
    }
#pragma unroll 1
    for (int j = start; j < n; j += step) {
      if (!wait(&S.s_full[gi], mine)) { give_up(); return; }
      tc_fence_after();
      if (j + step >= n) arrive(&S.q_free);
      const uint32_t i = tile0 + j;
      if (!wait(&S.meta_full[i % kMeta], i / kMeta)) { give_up(); return; }
      auto written = [&](int h) {
        tmem_wait_st();
        tc_fence_before();
        arrive(&S.p_full[gi][h]);
      };
      const int blocks = min(4, (s.tokens - (s.k0 + j) * kTile + 31) / 32);
      softmax_tile(tS, S.meta[i % kMeta], blocks, fq, m, M, l,
                   [&](float factor) {
                     // the group's P V of its tile before is complete: the
                     // commit that its S signalled came behind it
                     if (j == start) return;
#pragma unroll 1
                     for (int c = 0; c < DS; ++c) {
                       float o[16];
                       tmem_ld16(tO + 16 * c, o);
                       tmem_wait_ld();
#pragma unroll
                       for (int u = 0; u < 16; ++u) o[u] *= factor;
                       tmem_st16(tO + 16 * c, o);
                     }
                   },
                   [&]() { written(0); });
      written(1);
      ++mine;
    }
    tile0 += n;
    x += n;
    const bool more = x < x1;
    // the next segment's queries, once no S of this one is to come
    Segment next;
    float fq_next = 0.f;
    if (more) {
      next = segment_at(p, unit_rows, x, x1);
      const bool write = gi == 0 || next.wide();
      if (write && !wait(&S.q_free, segments)) { give_up(); return; }
      fq_next = load_q(next, write);
    }
    ++segments;
    const int r = (s.wide() ? gi * 128 : 0) + row;
    const size_t at = (size_t)blockIdx.x * 256 + 2 * s.before + (s.wide() ? r : gi * s.rows + row);
    if (start < n) {
      if (!wait(&S.o_done[gi], outputs)) { give_up(); return; }
      ++outputs;
      tc_fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < d; c0 += 16) {
        float o[16];
        __syncwarp();
        tmem_ld16(tO + c0, o);
        tmem_wait_ld();
        if (r < s.rows) {
#pragma unroll
          for (int u = 0; u < 16; u += 4)
            if (c0 + u < d)
              *reinterpret_cast<float4*>(p.piece_o + at * d + c0 + u) = make_float4(o[u], o[u + 1], o[u + 2], o[u + 3]);
        }
      }
      tc_fence_before();
    }
    if (r < s.rows) p.piece_s[at] = make_float4(m, l, M, 0.f);
    if (!more) return;
    s = next;
    fq = fq_next;
  }
}

template <int CODE, int DS>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ SharedCall p) {
  using L = Layout<DS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Small& S = *reinterpret_cast<Small*>(sm + L::kSmall);
  const Cache& c = p.own.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&S.sk_full[i], 1); mbar_init(&S.sk_empty[i], 4);
      mbar_init(&S.sv_full[i], 1); mbar_init(&S.sv_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.kf_full[i], 4); mbar_init(&S.kf_empty[i], 1);
      mbar_init(&S.vf_full[i], 4); mbar_init(&S.vf_empty[i], 1);
      mbar_init(&S.q_full[i], 4); mbar_init(&S.s_full[i], 1); mbar_init(&S.o_done[i], 1);
      mbar_init(&S.p_full[i][0], 4); mbar_init(&S.p_full[i][1], 4);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(&S.meta_full[i], 1);
    mbar_init(&S.q_free, 8);
    mbar_init(&S.drain, 1);
    S.abort = 0;
    fence_mbar_init();
  }
  if (c.d < 16 * DS) {                            // K's columns past d: zero, and never written
    for (int u = tid; u < 2 * L::kTileB / 16; u += kThreads)
      reinterpret_cast<uint4*>(sm + L::kK)[u] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (warp == kIssuer) tmem_alloc(&S.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  grid_dep_wait();
  grid_dep_launch();
  const SharedPlan plan = *p.plan;
  const int unit_rows = plan.unit_rows, stages = L::kStages + (unit_rows == 128 ? 1 : 0);
  const bool work = plan.total > 0 && blockIdx.x < plan.runs;
  const uint32_t x0 = work ? run_start(plan, blockIdx.x) : 0, x1 = work ? run_start(plan, blockIdx.x + 1) : 0;
  auto stage = [&](int s) { return sm + (s < L::kStages ? L::kStage + s * L::kStageB : L::kQ + L::kTileB); };
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, &S.abort)) != 0;
  };
  auto give_up = [&]() {
    if (lane == 0) {
      S.abort = 1;
      atomicOr(c.status, DROPKV_FLAG_TIMEOUT);
    }
  };

  if (x0 >= x1) {
    // (no more runs than work: nothing to do)
  } else if (warp == kLoader) {
    // Lane l describes page l % per of tile l / per of the batch: two
    // dependent loads, a batch ahead of their use.
    const int per = kTile >> c.page_log2, tiles = 32 / per, j = lane % per;
    Segment s;
    uint32_t from = 0, to = 0;                    // tiles of the run the lane's segment spans
    int pg[2], head[2];
    float ks[2], vs[2];
    auto describe = [&](uint32_t x, int w) {
      pg[w] = -1;
      if (x >= x1) return;
      if (x >= to) {
        s = segment_at(p, unit_rows, x, x1);
        from = x;
        to = x + s.n;
      }
      const int tok = (s.k0 + (int)(x - from)) * kTile + (j << c.page_log2);
      if (tok >= s.tokens) return;
      head[w] = s.h;
      pg[w] = c.table[(size_t)s.lead * c.M + (tok >> c.page_log2)];
      const size_t unit = (size_t)pg[w] * c.Hkv + s.h;
      ks[w] = c.ks[unit];
      vs[w] = c.vs[unit];
    };
    describe(x0 + lane / per, 0);
    const uint32_t bytes = (uint32_t)c.page * c.d;
    bool ok = true;
    uint32_t i = 0, n = x1 - x0;
    for (; ok && i < n; ++i) {
      const int t = i % tiles;
      if (t == 0) {
        if (i > 0) {
          pg[0] = pg[1];
          head[0] = head[1];
          ks[0] = ks[1];
          vs[0] = vs[1];
        }
        describe(x0 + i + tiles + lane / per, 1);
      }
      const bool here = lane / per == t, mine = here && pg[0] >= 0;
      const uint32_t pages = __popc(__ballot_sync(0xffffffffu, mine));
      const uint32_t slot = i % stages, round = i / stages;
      const size_t at = mine ? ((size_t)pg[0] * c.Hkv + head[0]) * bytes : 0;
      uint8_t* dst = stage(slot) + j * bytes;
      if (round > 0 && !(ok = wait(&S.sk_empty[slot], round - 1))) break;
      if (lane == 0) mbar_arrive_expect_tx(&S.sk_full[slot], pages * bytes);
      __syncwarp();
      if (mine) bulk_load(dst, c.k + at, bytes, &S.sk_full[slot]);
      if (round > 0 && !(ok = wait(&S.sv_empty[slot], round - 1))) { ++i; break; }
      // V of tile i - stages is converted, so P V of tile i - stages - 2 is
      // complete, and the softmax of tile i - kMeta long before
      if (here) {
        const int first = j << (c.page_log2 - 5), blocks = 1 << (c.page_log2 - 5);
        for (int b = first; b < first + blocks; ++b) {
          S.meta[i % kMeta].ks[b] = mine ? ks[0] : 0.f;
          S.meta[i % kMeta].lv[b] = mine ? __log2f(fmaxf(vs[0], 0x1p-126f)) : 0.f;
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&S.meta_full[i % kMeta]);
        mbar_arrive_expect_tx(&S.sv_full[slot], pages * bytes);
      }
      __syncwarp();
      if (mine) bulk_load(dst + L::kStageB / 2, c.v + at, bytes, &S.sv_full[slot]);
    }
    if (!ok) give_up();
    // every copy has landed before the CTA can leave
    for (uint32_t u = i > (uint32_t)stages ? i - stages : 0; u < i; ++u) {
      drain_wait(&S.sk_full[u % stages], (u / stages) & 1);
      drain_wait(&S.sv_full[u % stages], (u / stages) & 1);
    }
    __syncwarp();
  } else if (warp >= kConvert && warp < kIssuer) {
    const int t = tid - 32 * kConvert;
    bool ok = true;
    uint32_t i = 0;
    auto arrive = [&](uint64_t* bar, uint64_t* bar2) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar);
        mbar_arrive(bar2);
      }
      __syncwarp();
    };
    for (uint32_t x = x0; ok && x < x1;) {
      const Segment s = segment_at(p, unit_rows, x, x1);
      for (int k = 0; ok && k < s.n; ++k, ++i) {
        const int tokens = min(kTile, s.tokens - (s.k0 + k) * kTile);
        const uint32_t slot = i % stages, round = i / stages;
        uint8_t* from = stage(slot);
        ok = wait(&S.sk_full[slot], round) && (i < 2 || wait(&S.kf_empty[i & 1], (i >> 1) - 1));
        if (!ok) break;
        convert_tile<CODE, DS>(from, sm + L::kK + (i & 1) * L::kTileB, c.d, tokens, t);
        arrive(&S.kf_full[i & 1], &S.sk_empty[slot]);
        ok = wait(&S.sv_full[slot], round) && (i < 2 || wait(&S.vf_empty[i & 1], (i >> 1) - 1));
        if (!ok) break;
        convert_tile<CODE, DS>(from + L::kStageB / 2, sm + L::kV + (i & 1) * L::kTileB, c.d, tokens, t);
        arrive(&S.vf_full[i & 1], &S.sv_empty[slot]);
      }
      x += s.n;
    }
    if (!ok) give_up();
    __syncwarp();
  } else if (warp == kIssuer) {
    // The warp walks the tiles, one elected lane issues (descriptors stay in
    // uniform registers).  A group's next S follows its P V: it goes over the
    // P that this has read.
    const bool leader = elect_one();
    const uint64_t qd = desc_kmajor_sw128(smem_addr(sm + L::kQ), kTile, 0);
    const uint64_t kd = desc_kmajor_sw128(smem_addr(sm + L::kK), kTile, 0);
    const uint64_t vd = desc_mnmajor_sw128(smem_addr(sm + L::kV), kTile, 0);
    constexpr uint32_t idS = idesc_f16(128, 0), idO = idesc_f16(L::kDP, 1);
    // The products S stand in the order of the tiles (both groups' of a tile in
    // a wide segment); the next is issued when its group's P V before it is.
    struct {
      uint32_t x, i;                              // the segment's first tile of the call, of the run
      int n, j, g;                                // its tiles (0: no more), the next S
      bool wide;
    } next;
    auto enter = [&](uint32_t x, uint32_t i) {
      next.x = x;
      next.i = i;
      next.n = next.j = next.g = 0;
      next.wide = false;
      if (x >= x1) return;
      const Segment s = segment_at(p, unit_rows, x, x1);
      next.n = uniform(s.n);
      next.wide = uniform(s.wide()) != 0;
    };
    bool busy0 = false, busy1 = false;
    uint32_t q0 = 0, q1 = 0;                      // segments begun, wide ones among them
    auto pump = [&]() {                           // false: a wait gave up
      while (next.n > 0) {
        const int g = next.g;
        if (g ? busy1 : busy0) return true;
        if (next.j == 0 && g == 0 && !wait(&S.q_full[0], q0++)) return false;
        if (next.j == 0 && g == 1 && next.wide && !wait(&S.q_full[1], q1++)) return false;
        const uint32_t i = next.i + next.j, slot = i & 1;
        if (!next.wide || g == 0) {
          if (!wait(&S.kf_full[slot], i >> 1)) return false;
        }
        tc_fence_after();
        const uint64_t qg = qd + ((next.wide ? g * L::kTileB : 0) >> 4), kg = kd + ((slot * L::kTileB) >> 4);
        if (leader) {
#pragma unroll
          for (int s = 0; s < DS; ++s) {
            const uint64_t at = ((s >> 2) * L::kBlockB + (s & 3) * 32) >> 4;
            umma_bf16(128 * g, qg + at, kg + at, idS, s > 0);
          }
          umma_commit(&S.s_full[g]);
          if (!next.wide || g == 1) umma_commit(&S.kf_empty[slot]);
        }
        __syncwarp();
        if (g) busy1 = true;
        else busy0 = true;
        if (next.wide && g == 0) {
          next.g = 1;
        } else {
          ++next.j;
          next.g = next.wide ? 0 : next.j & 1;
          if (next.j == next.n) enter(next.x + next.n, next.i + next.n);
        }
      }
      return true;
    };
    enter(x0, 0);
    bool ok = pump();
    uint32_t i = 0, seen0 = 0, seen1 = 0;
    for (uint32_t x = x0; ok && x < x1;) {
      const Segment s = segment_at(p, unit_rows, x, x1);
      const int n = uniform(s.n);
      const bool wide = uniform(s.wide()) != 0;
      for (int j = 0; ok && j < n; ++j, ++i) {
        const uint32_t slot = i & 1;
        const uint64_t vg = vd + ((slot * L::kTileB) >> 4);
        if (!(ok = wait(&S.vf_full[slot], i >> 1))) break;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (!wide && (j & 1) != g) continue;
          uint32_t& seen = g ? seen1 : seen0;
          const bool first = j == (wide ? 0 : g), last = j + (wide ? 1 : 2) >= n;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!(ok = wait(&S.p_full[g][h], seen))) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int k = 4 * h; k < 4 * h + 4; ++k)
                umma_bf16_tmem_a(256 + 128 * g, 128 * g + 8 * k, vg + ((k * 16 * 128) >> 4), idO, !first || k > 0);
            }
            __syncwarp();
          }
          if (!ok) break;
          ++seen;
          if (leader) {
            if (!wide || g == 1) umma_commit(&S.vf_empty[slot]);
            if (last) umma_commit(&S.o_done[g]);
          }
          __syncwarp();
          if (g) busy1 = false;
          else busy0 = false;
          if (!(ok = pump())) break;
        }
      }
      x += n;
    }
    if (!ok) give_up();
    // no MMA may still be writing tensor memory when it is released
    if (leader) {
      umma_commit(&S.drain);
      drain_wait(&S.drain, 0);
    }
    __syncwarp();
  } else if (warp < kConvert) {
    softmax_group<DS>(p, S, sm, tmem, warp, lane, unit_rows, x0, x1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ the join
constexpr int kJoinWarps = 4, kJoinBatch = 8;
// A warp joins the pieces of a row: those of the shared tokens, in run order,
// and those of its own (one, or where its unit was cut, one per run).
__global__ void __launch_bounds__(32 * kJoinWarps) final_kernel(const SharedCall p) {
  grid_dep_wait();
  grid_dep_launch();
  const AttnCall& a = p.own;
  const int lane = threadIdx.x & 31, d = a.c.d;
  const long long row = (long long)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (row >= (long long)a.n * a.Hq * a.T) return;
  const int b = (int)(row / (a.Hq * a.T)), in = (int)(row - (long long)b * a.Hq * a.T), h = in / a.R, r = in - h * a.R;
  const bool cols = lane * 4 < d;
  float m = -INFINITY, M = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto join = [&](const float4& st, const float4& x) {
    if (st.x == -INFINITY && st.y == 0.f) return; // nothing there, perhaps no outputs either
    const float mn = fmaxf(m, st.x), Mn = fmaxf(M, st.z);
    const float fa = m == mn ? 1.f : ex2_approx(m - mn), fb = st.x == mn ? 1.f : ex2_approx(st.x - mn);
    const float Fa = M == Mn ? 1.f : ex2_approx(M - Mn), Fb = st.z == Mn ? 1.f : ex2_approx(st.z - Mn);
    l = l * fa + st.y * fb;
    o.x = o.x * Fa + x.x * Fb;
    o.y = o.y * Fa + x.y * Fb;
    o.z = o.z * Fa + x.z * Fb;
    o.w = o.w * Fa + x.w * Fb;
    m = mn;
    M = Mn;
  };
  // pieces at rows at(0), at(1), ..., at(n - 1) of a pair of arrays
  auto take = [&](const float4* states, const float* outputs, int n, auto at) {
    for (int k0 = 0; k0 < n; k0 += kJoinBatch) {
      float4 st[kJoinBatch], x[kJoinBatch];
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u) {
        st[u] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
        x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + u < n) {
          const size_t y = at(k0 + u);
          st[u] = states[y];
          if (cols) x[u] = *reinterpret_cast<const float4*>(outputs + y * d + lane * 4);
        }
      }
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u) join(st[u], x[u]);
    }
  };
  const int from = p.from[b];
  if (from > 0) {
    const SharedPlan plan = *p.plan;
    const int g = p.group[b], entry0 = p.groups[g], Mg = (p.groups[g + 1] - entry0) * a.R;
    const int per_head = (Mg + plan.unit_rows - 1) / plan.unit_rows, tiles = tiles_of(from);
    const int y = (b - entry0) * a.R + r, part = y / plan.unit_rows, rows = min(plan.unit_rows, Mg - part * plan.unit_rows);
    const uint32_t t0 = p.first[g] + ((uint32_t)h * per_head + part) * tiles;
    const int w0 = run_of(plan, t0), w1 = run_of(plan, t0 + tiles - 1), k = y - part * plan.unit_rows;
    const size_t before = 2 * ((size_t)entry0 * a.R * a.c.Hkv + (size_t)h * Mg + (size_t)part * plan.unit_rows) + k;
    if (rows > 128)
      take(p.piece_s, p.piece_o, w1 - w0 + 1, [&](int u) { return (size_t)(w0 + u) * 256 + before; });
    else                                          // two pieces per run, one of either group
      take(p.piece_s, p.piece_o, 2 * (w1 - w0 + 1),
           [&](int u) { return (size_t)(w0 + (u >> 1)) * 256 + before + (size_t)(u & 1) * rows; });
  }
  int2 cut = make_int2(-1, 0);
  const int rg = r / a.RB;
  if (p.by_runs) cut = a.cuts[((size_t)b * a.c.Hkv + h) * a.RG + rg];
  if (cut.x < 0)
    take(a.own_s, a.own_o, 1, [&](int) { return (size_t)row; });
  else
    take(a.part_s, a.part_o, cut.y - cut.x + 1, [&](int u) {
      return (((size_t)(cut.x + u) * a.RG + rg) * 2 + (u == 0 ? 1 : 0)) * a.RB + (r - rg * a.RB);
    });
  if (!cols) return;
  // o stands for o 2^(M - m - 7); a row that saw nothing has l = 0
  const float f = l == 0.f ? 0.f : ex2_approx(M - m) / l, unlift = 0x1p-7f;
  const __nv_bfloat162 h0 = __floats2bfloat162_rn(o.x * unlift * f, o.y * unlift * f),
                       h1 = __floats2bfloat162_rn(o.z * unlift * f, o.w * unlift * f);
  uint2 w = make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
  if (l == 0.f) w = make_uint2(0u, 0u);
  *reinterpret_cast<uint2*>(a.out + row * d + lane * 4) = w;
}

cudaError_t launch_plan(const SharedCall& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  // more CTAs only where there is much to compare
  const unsigned ctas = (long long)p.own.n * p.own.c.M > 8192 || p.own.n > 4 * kPlanThreads ? 8 : 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, plan_kernel, p);
}

template <int CODE, int DS>
cudaError_t launch_prefix(const SharedCall& p, cudaStream_t st) {
  const cudaError_t e = allow_smem<prefix_kernel<CODE, DS>>(kSmem<DS>);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefix_kernel<CODE, DS>, dim3(p.sms), dim3(kThreads), kSmem<DS>, st, p);
}
template <int CODE>
cudaError_t launch_prefix(const SharedCall& p, cudaStream_t st) {
  const int d = p.own.c.d;
  return d <= 64 ? launch_prefix<CODE, 4>(p, st) : d <= 96 ? launch_prefix<CODE, 6>(p, st) : launch_prefix<CODE, 8>(p, st);
}

}  // namespace

cudaError_t launch_shared(const SharedCall& p, cudaStream_t st) {
  cudaError_t e = launch_plan(p, st);
  if (e == cudaSuccess)
    e = p.own.c.code == KVCACHE_INT8 ? launch_prefix<KVCACHE_INT8>(p, st) : launch_prefix<KVCACHE_E4M3>(p, st);
  if (e == cudaSuccess) e = launch_own_attention(p.own, st);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)p.own.n * p.own.Hq * p.own.T;
  return launch_pdl(final_kernel, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)), dim3(32 * kJoinWarps), 0, st, p);
}

}  // namespace kvcache
