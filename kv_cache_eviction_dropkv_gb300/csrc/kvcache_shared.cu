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
//   attention_kernel<SHARED> (kvcache_attn.cuh)  each entry's own tokens
//   prefix_kernel  the shared tokens, on tcgen05; leaves pieces (O, m, l, M)
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
constexpr int kPlanEntries = 1024;

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

// (The passes between two calls of this kernel sweep its code out of every
// cache: what it takes is mostly the fetching of its instructions, so its loops
// are short and little is unrolled.  The comparing unrolled over 8 entries took
// 9.6 us of 15, for 64 sequences with 512 shared pages.)
// Up to kPlanEntries entries: every CTA of the cluster works out the groups by
// itself, in shared memory, and the CTAs share out the comparing only.  More:
// the entries are shared out too, and the groups stand in global memory.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const SharedCall p) {
  __shared__ int s_start[kPlanEntries + 1], s_seq[kPlanEntries], s_bound[kPlanEntries], s_group[kPlanEntries];
  __shared__ int s_lead[kPlanEntries], s_active[kPlanEntries], s_prefix[kPlanEntries], s_found[kPlanEntries];
  __shared__ uint32_t s_first[kPlanEntries], s_sum[kPlanThreads / 32];
  __shared__ int s_most;
  grid_dep_wait();
  grid_dep_launch();
  const AttnCall& a = p.own;
  const Cache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, rank = cluster_rank(), ctas = cluster_ctas();
  const int threads = kPlanThreads * ctas, me = rank * kPlanThreads + tid;
  const bool small = a.n <= kPlanEntries;
  const int first = small ? tid : me, step = small ? kPlanThreads : threads;   // of entries and groups
  const int32_t* start = small ? s_start : p.groups;
  int *bound = small ? s_bound : p.bound, *group = small ? s_group : p.group;
  int *lead = small ? s_lead : p.lead, *active = small ? s_active : p.active, *prefix = small ? s_prefix : p.prefix;
  auto seq_of = [&](int i) { return small ? s_seq[i] : a.seqs ? a.seqs[i] : i; };
  // groups that cover the entries in order
  bool bad = false;
  for (int j = tid; j <= p.G; j += kPlanThreads) {
    const int x = p.groups[j], y = j > 0 ? p.groups[j - 1] : 0;
    if (small) s_start[j] = x;
    bad |= x < y || (j == 0 && x != 0) || (j == p.G && x != a.n);
  }
  if (small)
    for (int i = tid; i < a.n; i += kPlanThreads) s_seq[i] = a.seqs ? a.seqs[i] : i;
  for (int j = first; j < p.G; j += step) {
    lead[j] = prefix[j] = INT_MAX;
    active[j] = 0;
    if (small) s_found[j] = INT_MAX;
  }
  if (tid == 0) s_most = 0;
  if (__syncthreads_or(bad)) {
    if (me == 0) {
      flag(c.status, DROPKV_FLAG_BAD_LENGTH);
      p.plan->total = 0;
      p.plan->runs = 1;
      p.plan->unit_rows = 128;
    }
    for (int i = me; i < a.n; i += threads) {
      p.from[i] = 0;
      p.info[i] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  // (small: what the others add to the first CTA's s_found comes behind its
  // start; they wait for that only then)
  if (small) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  else cluster_sync();
  // sequences that hold a full page before the first row's token take part
  for (int i = first; i < a.n; i += step) {
    const int s = seq_of(i), g = group_of(start, p.G, i);
    int full = 0;
    if (s >= 0 && s < c.S) {
      const int len = c.length[s], held = c.count[s];
      if (len >= a.T && held >= 0 && held <= c.M && (long long)len <= (long long)held << c.page_log2)
        full = (len - a.T + 1) >> c.page_log2;
    }
    bound[i] = full;
    group[i] = g;
    if (full > 0) {
      atomicMin(lead + g, i);
      atomicAdd(active + g, 1);
      atomicMin(prefix + g, full);
    }
  }
  if (small) __syncthreads();
  else cluster_sync();
  // `parts` warps compare an entry's columns with those of its group's first
  int* found = small ? s_found : p.prefix;
  const int warps = threads >> 5, parts = max(1, warps / a.n);
  for (long long item = me >> 5; item < (long long)a.n * parts; item += warps) {
    const int i = (uint32_t)item % (uint32_t)a.n, part = (uint32_t)item / (uint32_t)a.n, g = group[i];
    if (bound[i] == 0 || active[g] < 2) continue;
    const int32_t* mine = c.table + (size_t)seq_of(i) * c.M;
    const int32_t* other = c.table + (size_t)seq_of(lead[g]) * c.M;
    const int end = prefix[g];                    // (others may lower it meanwhile: it stays an end)
    int differs = INT_MAX;
#pragma unroll 4
    for (int col = part * 32 + lane; col < end; col += 32 * parts) {
      const int x = mine[col], y = other[col];
      if (x != y || (uint32_t)x >= (uint32_t)c.P) differs = min(differs, col);
    }
    differs = __reduce_min_sync(0xffffffffu, differs);
    if (lane == 0 && differs != INT_MAX) atomicMin(found + g, differs);
  }
  if (small) {
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (rank > 0)
      for (int j = tid; j < p.G; j += kPlanThreads)
        if (s_found[j] != INT_MAX) {
          uint32_t at;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(s_found + j)), "r"(0));
          asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;" ::"r"(at), "r"(s_found[j]) : "memory");
        }
  }
  cluster_sync();
  if (rank != 0) return;
  if (small) {
    for (int j = tid; j < p.G; j += kPlanThreads) prefix[j] = min(prefix[j], s_found[j]);
    __syncthreads();
  }
  // the widest unit, then tiles before each group, then what the kernels behind need
  for (int j = tid; j < p.G; j += kPlanThreads)
    if (active[j] >= 2 && prefix[j] > 0) atomicMax(&s_most, (start[j + 1] - start[j]) * a.R);
  __syncthreads();
  const int unit_rows = s_most > 128 ? 256 : 128;
  uint32_t before = 0;
  for (int j0 = 0; j0 < p.G; j0 += kPlanThreads) {
    const int j = j0 + tid;
    uint32_t tiles = 0;
    if (j < p.G && active[j] >= 2 && prefix[j] > 0)
      tiles = (uint32_t)tiles_of(prefix[j] << c.page_log2) * c.Hkv *
              (((start[j + 1] - start[j]) * a.R + unit_rows - 1) / unit_rows);
    uint32_t sum = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) s_sum[tid >> 5] = sum;
    __syncthreads();
    uint32_t all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < tid >> 5) sum += s_sum[w];
      all += s_sum[w];
    }
    if (j < p.G) {
      p.first[j] = before + sum - tiles;
      if (small) {
        s_first[j] = before + sum - tiles;
        p.lead[j] = lead[j];
        p.prefix[j] = prefix[j];
      }
    }
    before += all;
    __syncthreads();
  }
  if (tid == 0) {
    p.first[p.G] = before;
    p.plan->total = before;
    p.plan->runs = max(1u, min((uint32_t)p.sms, before / 2));
    p.plan->unit_rows = unit_rows;
  }
  for (int i = tid; i < a.n; i += kPlanThreads) {
    const int g = group[i], from = bound[i] > 0 && active[g] >= 2 ? prefix[g] << c.page_log2 : 0;
    p.from[i] = from;
    p.info[i] = make_int4(from, start[g], (start[g + 1] - start[g]) * a.R, from > 0 ? (int)(small ? s_first[g] : p.first[g]) : 0);
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
// (Out of line, as everything here that runs once per segment: the roles of the
// kernel below share an instruction cache, and 110 KB of code left each waiting
// for its next instruction most of the time.)
__device__ __noinline__ Segment segment_at(const SharedCall& p, int unit_rows, uint32_t x, uint32_t end) {
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
// Warps 0 .. 7: softmax; two for K's codes, two for V's, one that issues, one
// that loads (128 registers a thread).
constexpr int kConvert = 8, kIssuer = 12, kLoader = 13, kThreads = 32 * 14;
// P enters the product times 2^7 and the references are rounded down, so a row's
// largest P (times its V scale) is 2^7 at least, and what fp16 drops of a token
// is at most 2^-32 of it, as in kvcache_attention: what is far below the
// references must not be missing from the outputs while the sum counts it.
// (Times 2^4, with references rounded up, they move less often, each time for a
// tile's time and a half: 64 sequences behind 32768 shared tokens 113 instead of
// 115 us, 16 behind 131072 114 instead of 117; but behind dominant keys 2^20
// tokens of 2^-27.6 of their weight came out 37 % too large.)
constexpr float kLiftLog2 = 7.0f;
constexpr float kMost = 65504.f;                  // most that P of a row and 32 tokens may sum up to: what fp16 holds
constexpr float kLowLog2 = -60.0f;                // least exponent of the factor of P
constexpr float kMostLow = 0x1p-26f;              // the most such a block's P may sum up to: all are 0 in fp16 then
constexpr uint64_t kDrain = 20000000ull;          // 20 ms to drain copies after an abort
constexpr int kAhead = 6;                         // below 8, the fewest tiles of a batch of descriptions
constexpr int kMaxStages = 5, kMeta = 16;          // kMeta >= kMaxStages + 4

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
  int tokens;                                     // tokens of the tile
};
struct Small {
  uint64_t sk_full[kMaxStages], sk_empty[kMaxStages], sv_full[kMaxStages], sv_empty[kMaxStages];   // codes
  uint64_t kf_full[2], kf_empty[2], vf_full[2], vf_empty[2];                                       // fp16 tiles
  uint64_t q_full[2], q_free;      // group g's Q written; both groups' last S of a segment complete
  uint64_t s_full[2], p_full[2], o_done[2], drain;
  Scales meta[kMeta];
  uint32_t tmem_base;
  int abort;
};
template <int DS>
__device__ __forceinline__ uint8_t* stage_of(uint8_t* sm, int s) {   // one more in the place of the second Q
  using L = Layout<DS>;
  return sm + (s < L::kStages ? L::kStage + s * L::kStageB : L::kQ + L::kTileB);
}
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
// A wait whose first look fails.
__device__ __noinline__ bool slow_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_wait(bar, parity, abort);
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t phase, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase & 1))) return true;
  return __all_sync(0xffffffffu, slow_wait(bar, phase & 1, abort)) != 0;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {   // 16-byte aligned, a multiple of 16
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
constexpr uint32_t idesc_f16(uint32_t N, uint32_t b_mn) {   // both operands fp16 (format 0), fp32 accumulators, M = 128
  return (1u << 4) | (b_mn << 16) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}

// 16 bytes of a swizzled tile: chunk ch of row r.
__device__ __forceinline__ uint8_t* chunk_of(uint8_t* tile, int r, int ch) {
  return tile + (ch >> 3) * (kTile * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
}
// 16 codes as two chunks.
template <int CODE>
__device__ __forceinline__ void convert16(const uint4& w, uint8_t* lo, uint8_t* hi) {
  uint4 a, b;
  codes_to_half<CODE>(w.x, a.x, a.y);
  codes_to_half<CODE>(w.y, a.z, a.w);
  codes_to_half<CODE>(w.z, b.x, b.y);
  codes_to_half<CODE>(w.w, b.z, b.w);
  *reinterpret_cast<uint4*>(lo) = a;
  *reinterpret_cast<uint4*>(hi) = b;
}
// Codes of a tile (row pitch d bytes) as fp16 in the swizzled layout, rows from
// `tokens` on zero: rows [row0, row0 + 64), by a warp (t: the lane).  V codes at a
// time, V = 16 where d is a multiple of 16, else 8: the rows lie one behind the
// other, so the lanes read them as they come, and where a piece belongs is counted
// along.  (Divided out, 8 codes at a time: 10 groups of 4 to 7 sequences behind 64000
// to 96000 tokens, one head of 112, 186 us instead of 132.)
template <int CODE, int V>
__device__ __noinline__ void convert_odd(const uint8_t* from, uint8_t* to, int d, int tokens, int row0, int t) {
  constexpr int kBatch = 4;
  const int per = d / V, n = 64 * per, step_r = 32 / per, step_c = 32 - step_r * per;
  const uint8_t* src = from + row0 * d;
  const int r0 = t / per;
  int r = row0 + r0, c = t - r0 * per;
#pragma unroll 1
  for (int x0 = t; x0 < n; x0 += 32 * kBatch) {
    uint4 w[kBatch];
    int rows[kBatch], cols[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      rows[u] = r;
      cols[u] = c;
      r += step_r;
      c += step_c;
      if (c >= per) {
        c -= per;
        ++r;
      }
      w[u] = make_uint4(0, 0, 0, 0);
      const int x = x0 + 32 * u;
      if (x < n && rows[u] < tokens) {
        if (V == 16) {
          w[u] = *reinterpret_cast<const uint4*>(src + 16 * x);
        } else {
          const uint2 y = *reinterpret_cast<const uint2*>(src + 8 * x);
          w[u].x = y.x;
          w[u].y = y.y;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (x0 + 32 * u >= n) break;
      if (V == 16) {
        convert16<CODE>(w[u], chunk_of(to, rows[u], 2 * cols[u]), chunk_of(to, rows[u], 2 * cols[u] + 1));
      } else {
        uint4 v;
        codes_to_half<CODE>(w[u].x, v.x, v.y);
        codes_to_half<CODE>(w[u].y, v.z, v.w);
        *reinterpret_cast<uint4*>(chunk_of(to, rows[u], cols[u])) = v;
      }
    }
  }
}
// The same for d = 16 DS.  Eight lanes take 4 pieces of 16 codes of two
// adjacent rows, one row's from the first block of 64 columns, the other's from
// the second, so that their 128-bit accesses touch all banks once, reading and
// writing.
template <int CODE, int DS>
__device__ __forceinline__ void convert_tile(const uint8_t* from, uint8_t* to, int tokens, int row0, int t) {
  constexpr int kPitch = 16 * DS, kBlockB = kTile * 128, kBatch = 4;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int u = t & 3, r7 = t >> 2;
  const int first = DS == 8 ? r7 & 1 : 0;                  // the block that comes first
  const uint8_t* src = from + (row0 + r7) * kPitch + 16 * u;
  uint8_t* lo = to + (row0 + r7) * 128 + (((2 * u) ^ r7) << 4);
  uint8_t* hi = to + (row0 + r7) * 128 + (((2 * u + 1) ^ r7) << 4);
  constexpr int kBlocks = DS == 8 ? 2 : 1;
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) {
    const int block = b ? 1 - first : first;
#pragma unroll 1
    for (int k0 = 0; k0 < 64; k0 += 8 * kBatch) {
      uint4 w[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        w[k] = row0 + r7 + k0 + 8 * k < tokens
                   ? *reinterpret_cast<const uint4*>(src + (k0 + 8 * k) * kPitch + 64 * block)
                   : zero;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        convert16<CODE>(w[k], lo + (k0 + 8 * k) * 128 + block * kBlockB, hi + (k0 + 8 * k) * 128 + block * kBlockB);
    }
  }
  if (DS == 6) {                                           // columns 64 to 95
#pragma unroll 2
    for (int r = row0 + (t >> 1); r < row0 + 64; r += 16) {
      const uint4 w = r < tokens ? *reinterpret_cast<const uint4*>(from + r * kPitch + 64 + 16 * (t & 1)) : zero;
      convert16<CODE>(w, chunk_of(to, r, 8 + 2 * (t & 1)), chunk_of(to, r, 9 + 2 * (t & 1)));
    }
  }
}

// Values of loads from tensor memory pass through here behind the wait for
// them, so that nothing that uses them comes before it.
__device__ __forceinline__ void pin16(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void ld64(uint32_t taddr, float (&v)[64]) {
#pragma unroll
  for (int u = 0; u < 64; u += 16) tmem_ld16(taddr + u, v + u);
}
__device__ __forceinline__ void wait_ld64(float (&v)[64]) {
  tmem_wait_ld();
#pragma unroll
  for (int u = 0; u < 64; u += 16) pin16(v + u);
}
// Packed halves in `columns` columns of tensor memory, times `factor`.
__device__ __noinline__ void scale_halves(uint32_t taddr, int columns, float factor) {
  for (int c = 0; c < columns; c += 8) {
    float w[8];
    tmem_ld8(taddr + c, w);
    tmem_wait_ld();
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      asm volatile("" : "+f"(w[u]));
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[u]));
      w[u] = __uint_as_float(pack_half2(h.x * factor, h.y * factor));
    }
    tmem_st8(taddr + c, w);
  }
  tmem_wait_st();
}

// A thread's row of a tile: S in its columns of tensor memory becomes P.
//   x_c = s f_c (base-2 logits; f_c: the row's factor times block c's K scale),
//   P = 2^(x - m + e_c), e_c = lv_c + m - M + 7,  l += sum of 2^(x - m)
// m and M are references of the sums and of the outputs (which carry the V
// scales).  No maximum is looked for: P is made on the references as they are,
// and only where the sum of a block of 32 shows that some P is too large for
// fp16 the references move (to whole numbers, at most 1 below the maxima of the
// half row at hand) and the half row is made again from S, which its P has not yet
// replaced.  follow(factor) lets O follow M, and P of the first half follows
// too.  A row's first tile always takes that way.
// A block whose V scale is so far below the others' that e_c would pass under
// kLowLog2 is made with that instead, so that P does not vanish from l; as its P
// is then larger than it should be, the references move as soon as any of it
// would show in fp16.
template <typename Follow>
__device__ __forceinline__ void softmax_tile(uint32_t tS, const Scales& scales, int blocks, float fq, float& m, float& M,
                                             float& l, Follow follow) {
  float v[64], hw[32];
  ld64(tS, v);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    float s[2], e[2], most[2];
    for (int round = 0;; ++round) {
      wait_ld64(v);
      uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull}, f2[2], n2[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int c = 2 * h + b;
        const float f = fmaxf(fq * scales.ks[c], 0x1p-126f);
        e[b] = scales.lv[c] + m - M + kLiftLog2;
        most[b] = e[b] < kLowLog2 ? kMostLow : kMost;
        e[b] = fmaxf(e[b], kLowLog2);
        const float n = c < blocks ? e[b] - m : -INFINITY;   // (no tokens: P = 0)
        f2[b] = f2_pack(f, f);
        n2[b] = f2_pack(n, n);
      }
      // 16 columns at a time: while the exponentials of one run, those before
      // are summed and packed, and make room for the next half row
#pragma unroll
      for (int k = 0; k <= 4; ++k) {
        if (k < 4) {
#pragma unroll
          for (int u = 16 * k; u < 16 * k + 16; u += 2) {
            const uint64_t y = f2_fma(f2_pack(v[u], v[u + 1]), f2[k >> 1], n2[k >> 1]);
            v[u] = ex2_approx(f2_lo(y));
            v[u + 1] = ex2_approx(f2_hi(y));
          }
        }
        if (k > 0) {
#pragma unroll
          for (int u = 16 * k - 16; u < 16 * k; u += 2) {
            uint64_t& a = sum2[((k - 1) & 2) + ((u >> 1) & 1)];
            a = f2_add(a, f2_pack(v[u], v[u + 1]));
            hw[u / 2] = __uint_as_float(pack_half2(v[u], v[u + 1]));
          }
          if (h == 0) tmem_ld16(tS + 64 + 16 * (k - 1), v + 16 * (k - 1));
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint64_t a = f2_add(sum2[2 * b], sum2[2 * b + 1]);
        s[b] = f2_lo(a) + f2_hi(a);
      }
      const bool over = s[0] > most[0] || s[1] > most[1];
      if (round == 1 || !__any_sync(0xffffffffu, over)) break;
      // What is loaded, scaled and stored again below (O, the first half of P) may
      // just have been stored, and loads do not wait for stores by themselves.
      tmem_wait_st();
      if (h == 0) wait_ld64(v);                            // (what came for the next half row is loaded again)
      ld64(tS + 64 * h, v);
      wait_ld64(v);
      float mt = -INFINITY, Mt = -INFINITY;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int c = 2 * h + b;
        float x = v[32 * b], z = v[32 * b + 1];
#pragma unroll
        for (int u = 2; u < 32; u += 2) {
          x = fmaxf(x, v[32 * b + u]);
          z = fmaxf(z, v[32 * b + u + 1]);
        }
        x = fmaxf(x, z) * fmaxf(fq * scales.ks[c], 0x1p-126f);
        if (c < blocks) {
          mt = fmaxf(mt, x);
          Mt = fmaxf(Mt, x + scales.lv[c]);
        }
      }
      const float mn = over ? fmaxf(m, floorf(mt)) : m, Mn = over ? fmaxf(M, floorf(Mt)) : M;
      l *= m == mn ? 1.f : ex2_approx(m - mn);             // (from nothing: 0 times 0)
      const float factor = M == Mn ? 1.f : ex2_approx(M - Mn);
      m = mn;
      M = Mn;
      follow(factor);
      if (h == 1) scale_halves(tS, 32, factor);
    }
    l += s[0] * ex2_approx(-e[0]) + s[1] * ex2_approx(-e[1]);
    tmem_st16(tS + 32 * h, hw);
    tmem_st16(tS + 32 * h + 16, hw + 16);
  }
}

// A value all lanes of the converged warp hold, in a uniform register.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

// A thread's query row as fp16 to `to` (a row of a swizzled tile, or null),
// times a power of two that brings its largest element to [2^14, 2^15);
// returns the factor of its logits.
template <int DS>
__device__ __noinline__ float load_query(const AttnCall& a, const Segment& s, int gi, int row, uint8_t* to) {
  const int r = (s.wide() ? gi * 128 : 0) + row, d = a.c.d;
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
  if (to) {
#pragma unroll
    for (int u = 0; u < 2 * DS; ++u)
      *reinterpret_cast<uint4*>(to + (u >> 3) * (kTile * 128) + (((u & 7) ^ (row & 7)) << 4)) =
          make_uint4(pack_half2(bf_lo(w[u].x) * up, bf_hi(w[u].x) * up), pack_half2(bf_lo(w[u].y) * up, bf_hi(w[u].y) * up),
                     pack_half2(bf_lo(w[u].z) * up, bf_hi(w[u].z) * up), pack_half2(bf_lo(w[u].w) * up, bf_hi(w[u].w) * up));
  }
  return down * a.scale_log2;
}

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
  auto wait = [&](uint64_t* bar, uint32_t phase) { return wait_phase(bar, phase, &S.abort); };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    __syncwarp();
  };
  auto load_q = [&](const Segment& s, bool write) {
    const float f = load_query<DS>(a, s, gi, row, write ? sm + L::kQ + (s.wide() ? gi * L::kTileB : 0) + row * 128 : nullptr);
    if (write) {
      fence_proxy_async_smem();
      arrive(&S.q_full[gi]);
    }
    return f;
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
      const uint32_t i = tile0 + j;
      if (!wait(&S.s_full[gi], mine)) { give_up(); return; }
      tc_fence_after();
      if (j + step >= n) arrive(&S.q_free);
      softmax_tile(tS, S.meta[i % kMeta], S.meta[i % kMeta].tokens / 32, fq, m, M, l,
                   [&](float factor) {
                     // the group's P V of its tile before is complete: the
                     // commit that its S signalled came behind it
                     if (j == start) return;
#pragma unroll 1
                     for (int c = 0; c < DS; ++c) {
                       float o[16];
                       tmem_ld16(tO + 16 * c, o);
                       tmem_wait_ld();
                       pin16(o);
#pragma unroll
                       for (int u = 0; u < 16; ++u) o[u] *= factor;
                       tmem_st16(tO + 16 * c, o);
                     }
                   });
      tmem_wait_st();
      tc_fence_before();
      arrive(&S.p_full[gi]);
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
        pin16(o);
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

#ifdef DROPKV_TEST_HOOKS
__device__ int g_test_skip_load[2] = {-1, -1};    // CTA and load that the test build leaves out
#endif

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
      mbar_init(&S.sk_full[i], 1); mbar_init(&S.sk_empty[i], 2);
      mbar_init(&S.sv_full[i], 1); mbar_init(&S.sv_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.kf_full[i], 2); mbar_init(&S.kf_empty[i], 1);
      mbar_init(&S.vf_full[i], 2); mbar_init(&S.vf_empty[i], 1);
      mbar_init(&S.q_full[i], 4); mbar_init(&S.s_full[i], 1); mbar_init(&S.o_done[i], 1);
      mbar_init(&S.p_full[i], 4);
    }
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
  auto wait = [&](uint64_t* bar, uint32_t phase) { return wait_phase(bar, phase, &S.abort); };
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
    // The stages hold one or two tiles, which is less than memory's latency:
    // tiles up to kAhead further on are on their way to L2.
    auto ahead = [&](int w, bool take) {
      if (!take || pg[w] < 0) return;
      const size_t at = ((size_t)pg[w] * c.Hkv + head[w]) * bytes;
      prefetch_l2(c.k + at, bytes);
      prefetch_l2(c.v + at, bytes);
    };
    ahead(0, lane / per < kAhead);
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
      ahead(t + kAhead < tiles ? 0 : 1, lane / per == (t + kAhead) % tiles);
      const bool here = lane / per == t, mine = here && pg[0] >= 0;
      const uint32_t pages = __popc(__ballot_sync(0xffffffffu, mine));
      const uint32_t slot = i % stages, round = i / stages;
      const size_t at = mine ? ((size_t)pg[0] * c.Hkv + head[0]) * bytes : 0;
      uint8_t* dst = stage_of<DS>(sm, slot) + j * bytes;
      if (round > 0 && !(ok = wait(&S.sk_empty[slot], round - 1))) break;
      // K of tile i - stages is converted, so S of tile i - stages - 2 is
      // complete and the softmax of tile i - kMeta long done
      if (here) {
        const int first = j << (c.page_log2 - 5), blocks = 1 << (c.page_log2 - 5);
        for (int b = first; b < first + blocks; ++b) {
          S.meta[i % kMeta].ks[b] = mine ? ks[0] : 0.f;
          S.meta[i % kMeta].lv[b] = mine ? __log2f(fmaxf(vs[0], 0x1p-126f)) : 0.f;
        }
      }
      if (lane == 0) S.meta[i % kMeta].tokens = pages << c.page_log2;
      __syncwarp();
      bool load[2] = {true, true};
#ifdef DROPKV_TEST_HOOKS
      if ((int)blockIdx.x == g_test_skip_load[0] && (int)i == g_test_skip_load[1] >> 1) load[g_test_skip_load[1] & 1] = false;
#endif
      if (lane == 0 && load[0]) mbar_arrive_expect_tx(&S.sk_full[slot], pages * bytes);
      __syncwarp();
      if (mine && load[0]) bulk_load(dst, c.k + at, bytes, &S.sk_full[slot]);
      if (round > 0 && !(ok = wait(&S.sv_empty[slot], round - 1))) { ++i; break; }
      if (lane == 0 && load[1]) mbar_arrive_expect_tx(&S.sv_full[slot], pages * bytes);
      __syncwarp();
      if (mine && load[1]) bulk_load(dst + L::kStageB / 2, c.v + at, bytes, &S.sv_full[slot]);
    }
    if (!ok) give_up();
    // every copy has landed before the CTA can leave
    for (uint32_t u = i > (uint32_t)stages ? i - stages : 0; u < i; ++u) {
      drain_wait(&S.sk_full[u % stages], (u / stages) & 1);
      drain_wait(&S.sv_full[u % stages], (u / stages) & 1);
    }
    __syncwarp();
  } else if (warp >= kConvert && warp < kIssuer) {
    const int v = (warp - kConvert) >> 1, row0 = 64 * (warp & 1);   // K's or V's, half a tile
    uint64_t *coded = v ? S.sv_full : S.sk_full, *read = v ? S.sv_empty : S.sk_empty;
    uint64_t *made = v ? S.vf_full : S.kf_full, *used = v ? S.vf_empty : S.kf_empty;
    bool ok = true;
#pragma unroll 1
    for (uint32_t i = 0; i < x1 - x0; ++i) {
      const uint32_t slot = i % stages;
      ok = wait(coded + slot, i / stages) && (i < 2 || wait(used + (i & 1), (i >> 1) - 1));
      if (!ok) break;
      const uint8_t* from = stage_of<DS>(sm, slot) + v * (L::kStageB / 2);
      uint8_t* to = sm + (v ? L::kV : L::kK) + (i & 1) * L::kTileB;
      const int tokens = S.meta[i % kMeta].tokens;
      if (c.d == 16 * DS) convert_tile<CODE, DS>(from, to, tokens, row0, lane);
      else if (c.d % 16 == 0) convert_odd<CODE, 16>(from, to, c.d, tokens, row0, lane);
      else convert_odd<CODE, 8>(from, to, c.d, tokens, row0, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(made + (i & 1));
        mbar_arrive(read + slot);
      }
      __syncwarp();
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
    bool ok = true;
    uint32_t tile0 = 0, seen0 = 0, seen1 = 0;
    for (uint32_t x = x0; ok && x < x1;) {
      const Segment s = segment_at(p, unit_rows, x, x1);
      const int n = uniform(s.n);
      const bool wide = uniform(s.wide()) != 0;
      const int products = wide ? 2 * n : n;      // P V of the segment: tile by tile, in a wide one both groups'
#pragma unroll 1
      for (int y = 0; ok && y < products; ++y) {
        if (!(ok = pump())) break;
        const int j = wide ? y >> 1 : y, g = y & 1;
        const uint32_t i = tile0 + j, slot = i & 1, seen = g ? seen1 : seen0;
        const bool first = j == (wide ? 0 : g), last = j + (wide ? 1 : 2) >= n;
        const uint64_t vg = vd + ((slot * L::kTileB) >> 4);
        if ((!wide || g == 0) && !(ok = wait(&S.vf_full[slot], i >> 1))) break;
        if (!(ok = wait(&S.p_full[g], seen))) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_bf16_tmem_a(256 + 128 * g, 128 * g + 8 * k, vg + ((k * 16 * 128) >> 4), idO, !first || k > 0);
        }
        __syncwarp();
        if (g) ++seen1;
        else ++seen0;
        if (leader) {
          if (!wide || g == 1) umma_commit(&S.vf_empty[slot]);
          if (last) umma_commit(&S.o_done[g]);
        }
        __syncwarp();
        if (g) busy1 = false;
        else busy0 = false;
      }
      tile0 += n;
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
// The pieces of a row are joined in an order that does not depend on timing:
// those of the shared tokens, in run order, then those of its own (one, or
// where its unit was cut, one per run).  A lane holds the state of a piece and
// works out its factor; then the warp adds up the outputs, 4 channels a lane,
// the factors handed round.  (Short code here too: see plan_kernel.)
struct Joined {
  float m, M, l;
  float4 o;
};
// The factor of the lane's piece with state st (m, l, M), when 32 pieces join j;
// l and the references of j follow, o has to be multiplied by *follow.
__device__ __forceinline__ float join_state(Joined& j, const float4& st, float* follow) {
  float mn = fmaxf(j.m, st.x), Mn = fmaxf(j.M, st.z);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    Mn = fmaxf(Mn, __shfl_xor_sync(0xffffffffu, Mn, o));
  }
  const float m0 = mn == -INFINITY ? 0.f : mn, M0 = Mn == -INFINITY ? 0.f : Mn;   // (nothing yet: all factors 0)
  float sum = st.y * ex2_approx(st.x - m0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  j.l = j.l * ex2_approx(j.m - m0) + sum;
  *follow = ex2_approx(j.M - M0);
  j.m = mn;
  j.M = Mn;
  // of nothing perhaps no outputs were written either: they are passed over
  return st.x == -INFINITY && st.y == 0.f ? 0.f : ex2_approx(st.z - M0);
}
__device__ __forceinline__ void scale4(float4& o, float f) {
  o.x *= f;
  o.y *= f;
  o.z *= f;
  o.w *= f;
}
__device__ __forceinline__ void add4(float4& o, const float4& x, float f) {
  if (f == 0.f) return;                           // (the same for all lanes)
  o.x = fmaf(x.x, f, o.x);
  o.y = fmaf(x.y, f, o.y);
  o.z = fmaf(x.z, f, o.z);
  o.w = fmaf(x.w, f, o.w);
}
// W > 1: a CTA of W warps joins one row, of up to some 300 pieces, a warp every
// W-th; else a warp each joins a row (4 to a CTA).  Whole calls with 1, 4 and 8
// warps a row, when P was lifted by 2^4: 512 rows of 39 pieces 124, 117, 112 us;
// 1456 rows 90.6, 88.5, 95.2; 2048 rows of 20 pieces 110.7, 114.6, 119.5; 20 rows to
// an SM 69.8, 76.4, 86.4.  The launch bounds leave 40 registers (W > 1) and 64, and
// the eight loads in flight spill 268 and 116 bytes: 8 to 12 us where the bytes
// take 4.
template <int W>
__global__ void __launch_bounds__(32 * (W > 1 ? W : 4), W > 1 ? 48 / W : 8) final_kernel(const SharedCall p) {
  constexpr bool WHOLE = W > 1;
  constexpr int kBatch = 8, kJoinWarps = WHOLE ? W : 4, kStep = WHOLE ? W : 1;
  __shared__ float4 s_o[kJoinWarps][32], s_s[kJoinWarps];
  grid_dep_wait();
  grid_dep_launch();
  const AttnCall& a = p.own;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = a.c.d, b = blockIdx.y;
  const uint32_t in = WHOLE ? blockIdx.x : blockIdx.x * kJoinWarps + warp, h = in / (uint32_t)a.R, r = in - h * a.R;
  if (!WHOLE && in >= (uint32_t)a.Hq * a.T) return;
  const size_t row = (size_t)b * a.Hq * a.T + in;
  const uint32_t rg = a.RB == 8 ? r >> 3 : r >> 4;
  const bool cols = lane * 4 < d;
  const int4 info = p.info[b];                    // shared tokens, first entry of the group, its rows, its first tile
  const SharedPlan plan = *p.plan;
  const int2 cut = p.by_runs ? a.cuts[((size_t)b * a.c.Hkv + h) * a.RG + rg] : make_int2(-1, 0);
  // its pieces of the shared tokens, in runs w0 .. w1, two each where the groups
  // of warps took turns, and of its own
  int shared = 0, both = 0, rows = 0;
  uint32_t at = 0;
  if (info.x > 0) {
    const int shift = plan.unit_rows == 256 ? 8 : 7, per_head = (info.z + plan.unit_rows - 1) >> shift;
    const int y = (b - info.y) * a.R + r, part = y >> shift;
    rows = min(plan.unit_rows, info.z - (part << shift));
    both = rows > 128 ? 0 : 1;
    const int tiles = tiles_of(info.x);
    const uint32_t t0 = (uint32_t)info.w + (h * per_head + part) * tiles;
    const uint32_t w0 = run_of(plan, t0), w1 = run_of(plan, t0 + tiles - 1);
    shared = (w1 - w0 + 1) << both;
    at = w0 * 256 + 2 * ((uint32_t)info.y * a.R * a.c.Hkv + h * info.z + (part << shift)) + (y - (part << shift));
  }
  const bool whole = cut.x < 0;
  const uint32_t first = whole ? (uint32_t)row : (((uint32_t)cut.x * a.RG + rg) * 2) * a.RB + (r - rg * a.RB);
  const uint32_t pitch = 2 * a.RB * a.RG;
  const float4* own_s = whole ? a.own_s : a.part_s;
  const float* own_o = whole ? a.own_o : a.part_o;
  const int pieces = shared + (whole ? 1 : cut.y - cut.x + 1);
  Joined j;
  j.m = j.M = -INFINITY;
  j.l = 0.f;
  j.o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k0 = WHOLE ? warp : 0; k0 < pieces; k0 += 32 * kStep) {
    const int k = k0 + lane * kStep, q = k - shared, n = min(32, (pieces - k0 + kStep - 1) / kStep);
    const uint32_t y = q < 0 ? at + (k >> both) * 256 + (both & k ? rows : 0)
                             : whole ? first : first + q * pitch + (q == 0 ? a.RB : 0);
    float4 st = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    if (k < pieces) st = (q < 0 ? p.piece_s : own_s)[y];
    float G = 0.f;
#pragma unroll 1
    for (int u0 = 0; u0 < n; u0 += kBatch) {
      float4 x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const uint32_t yu = __shfl_sync(0xffffffffu, y, u0 + u);
        x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (cols && u0 + u < n)
          x[u] = *reinterpret_cast<const float4*>((k0 + (u0 + u) * kStep < shared ? p.piece_o : own_o) + (size_t)yu * d + lane * 4);
      }
      if (u0 == 0) {                              // (behind the loads)
        float follow;
        G = join_state(j, st, &follow);
        scale4(j.o, follow);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) add4(j.o, x[u], __shfl_sync(0xffffffffu, G, u0 + u));
    }
  }
  if (WHOLE) {
    s_o[warp][lane] = j.o;
    if (lane == 0) s_s[warp] = make_float4(j.m, j.l, j.M, 0.f);
    __syncthreads();
    if (warp > 0) return;
    const float4 st = lane < kJoinWarps ? s_s[lane] : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    j.m = j.M = -INFINITY;
    j.l = 0.f;
    j.o = make_float4(0.f, 0.f, 0.f, 0.f);
    float follow;
    const float G = join_state(j, st, &follow);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) add4(j.o, s_o[w][lane], __shfl_sync(0xffffffffu, G, w));
  }
  if (!cols) return;
  // o stands for o 2^(M - m - 7); a row that saw nothing has l = 0
  const float f = j.l == 0.f ? 0.f : ex2_approx(j.M - j.m) / j.l, unlift = 0x1p-7f;
  const __nv_bfloat162 h0 = __floats2bfloat162_rn(j.o.x * unlift * f, j.o.y * unlift * f),
                       h1 = __floats2bfloat162_rn(j.o.z * unlift * f, j.o.w * unlift * f);
  uint2 w = make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
  if (j.l == 0.f) w = make_uint2(0u, 0u);
  *reinterpret_cast<uint2*>(a.out + row * d + lane * 4) = w;
}

cudaError_t launch_plan(const SharedCall& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  // more CTAs only where there is much to compare
  const unsigned ctas = (long long)p.own.n * p.own.c.M > 8192 || p.own.n > kPlanEntries ? 8 : 1;
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
  // (own tokens first: the shared tokens' pieces, some 20 MB, are then still in
  // the L2 cache when they are joined)
  if (e == cudaSuccess) e = launch_own_attention(p.own, st);
  if (e == cudaSuccess)
    e = p.own.c.code == KVCACHE_INT8 ? launch_prefix<KVCACHE_INT8>(p, st) : launch_prefix<KVCACHE_E4M3>(p, st);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)p.own.n * p.own.Hq * p.own.T;
  const unsigned per = (unsigned)(p.own.Hq * p.own.T);
  if (rows <= 4LL * p.sms) return launch_pdl(final_kernel<8>, dim3(per, p.own.n), dim3(256), 0, st, p);
  if (rows <= 12LL * p.sms) return launch_pdl(final_kernel<4>, dim3(per, p.own.n), dim3(128), 0, st, p);
  return launch_pdl(final_kernel<1>, dim3((per + 3) / 4, p.own.n), dim3(128), 0, st, p);
}

}  // namespace kvcache

#ifdef DROPKV_TEST_HOOKS
#include "../../include/kvcache_step_test_hooks.h"
extern "C" dropkv_status kvcache_test_skip_shared_load(int32_t cta, int32_t load) {
  const int v[2] = {cta, load};
  return cudaMemcpyToSymbol(kvcache::g_test_skip_load, v, sizeof v) == cudaSuccess ? DROPKV_OK : DROPKV_ERR_CUDA;
}
#endif
