// Pages of the paged 8-bit cache: taking, sharing, copying, compacting and
// releasing them.
//
// A page is free when its reference count is 0, and the lowest free pages are
// taken in order: there is no free list whose order would depend on the order
// of atomics, and results depend on the state alone.  The integer bookkeeping
// of a call (who wants how many pages, which pages those are) is one CTA's
// work: block scans over the call's entries and over the reference counts, 16
// counts a thread at a time, loaded before anything that waits for them.
// What grows with the cache (page bytes, table rows, reference counts of
// shared pages) is a second kernel's, spread over the GPU and launched with
// programmatic dependent launch.  (One cluster of 16 CTAs doing both in one
// launch was slower even for a few hundred kilobytes: 16 against 10 us.)
#include "kvcache_internal.cuh"
#include "sm103_ptx.cuh"

namespace kvcache {
namespace {

using dropkv::grid_dep_launch;
using dropkv::grid_dep_wait;
using dropkv::launch_pdl;
using dropkv::named_bar;

constexpr int kBook = 1024;                // threads of a bookkeeping CTA
constexpr int kBookWarps = kBook / 32;

__device__ __forceinline__ int seq_of(const int32_t* seqs, int i) { return seqs ? seqs[i] : i; }
__device__ __forceinline__ int pages_for(const Cache& c, int tokens) {
  return (int)(((unsigned)tokens + (unsigned)c.page - 1u) >> c.page_log2);
}

// Exclusive sum over the block's threads; *total gets the sum of all.  `turn`
// counts the calls (it picks one of two buffers, so a call needs one barrier).
// 64 bits: the pages a call wants may be many times those there are.
__device__ __forceinline__ long long block_scan(long long x, long long* total, int& turn) {
  __shared__ long long warp_sum[2][kBookWarps];
  long long* sums = warp_sum[turn++ & 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  long long w = sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return (warp > 0 ? before : 0) + inc - x;
}

// Which entries are the first to name their sequence.  Up to kSmall entries
// are compared in shared memory; more go through claim[s] = lowest index that
// names s.
constexpr int kSmall = 128;
struct Names {
  int mine[kSmall], other[kSmall];
};
__device__ __forceinline__ void claim_seqs(const PageCall& p, const int32_t* seqs, Names& names) {
  if (p.n <= kSmall) {
    for (int i = threadIdx.x; i < p.n; i += kBook) names.mine[i] = seqs[i];
  } else {
    for (int i = threadIdx.x; i < p.n; i += kBook) {
      const int s = seqs[i];
      if (s >= 0 && s < p.c.S) p.claim[s] = INT32_MAX;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += kBook) {
      const int s = seqs[i];
      if (s >= 0 && s < p.c.S) atomicMin(&p.claim[s], i);
    }
  }
  __syncthreads();
}
__device__ __forceinline__ bool first_named(const PageCall& p, const Names& names, int i, int s) {
  if (p.n > kSmall) return p.claim[s] == i;
  int before = 0;
#pragma unroll 8
  for (int j = 0; j < i; ++j) before |= names.mine[j] == s;
  return before == 0;
}

// 16 reference counts a thread, of the pages from `base` on.
constexpr int kPer = 16;
struct Counts {
  int4 r[kPer / 4];
};
__device__ __forceinline__ Counts load_counts(const Cache& c, int base) {
  Counts k;
  const int first = base + threadIdx.x * kPer;
#pragma unroll
  for (int u = 0; u < kPer / 4; ++u) {
    const int a = first + 4 * u;
    if (a + 4 <= c.P) {
      k.r[u] = *reinterpret_cast<const int4*>(c.refs + a);
    } else {
      k.r[u] = make_int4(1, 1, 1, 1);
      if (a < c.P) k.r[u].x = c.refs[a];
      if (a + 1 < c.P) k.r[u].y = c.refs[a + 1];
      if (a + 2 < c.P) k.r[u].z = c.refs[a + 2];
    }
  }
  return k;
}

// The `want` lowest free pages into p.list; false (and a flag) if there are
// fewer.  k: the counts of the first pages.
__device__ __forceinline__ bool find_pages(const PageCall& p, long long want, Counts k, int& turn) {
  int found = 0;
  if (want > p.c.P) {
    if (threadIdx.x == 0) flag(p.c.status, KVCACHE_FLAG_NO_PAGES);
    return false;
  }
  for (int base = 0; base < p.c.P && found < want; base += kBook * kPer) {
    if (base > 0) k = load_counts(p.c, base);
    uint32_t free_bits = 0;
#pragma unroll
    for (int u = 0; u < kPer / 4; ++u) {
      free_bits |= (k.r[u].x == 0 ? 1u : 0u) << (4 * u) | (k.r[u].y == 0 ? 2u : 0u) << (4 * u) |
                   (k.r[u].z == 0 ? 4u : 0u) << (4 * u) | (k.r[u].w == 0 ? 8u : 0u) << (4 * u);
    }
    long long total;
    int at = found + (int)block_scan(__popc(free_bits), &total, turn);
    const int first = base + threadIdx.x * kPer;
    while (free_bits && at < want) {
      const int bit = __ffs(free_bits) - 1;
      free_bits &= free_bits - 1;
      p.list[at++] = first + bit;
    }
    found += (int)total;
  }
  __syncthreads();
  if (found < want && threadIdx.x == 0) flag(p.c.status, KVCACHE_FLAG_NO_PAGES);
  return found >= want;
}

// Index of the entry that takes page k of the list: the last i with offs[i] <= k.
__device__ __forceinline__ int entry_of(const int32_t* offs, int n, int k) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offs[mid] <= k) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ============================================================== free
// One CTA per entry.  The exchange gives a sequence named twice to one of
// them; either way its pages lose one reference.
__global__ void __launch_bounds__(256) free_kernel(const PageCall p) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int held;
  const int s = seq_of(p.seqs, blockIdx.x);
  if (s < 0 || s >= p.c.S) {
    if (threadIdx.x == 0) flag(p.c.status, KVCACHE_FLAG_BAD_SEQ);
    return;
  }
  int32_t* row = p.c.table + (size_t)s * p.c.M;
  // read before it is known how many pages are held: a round trip less
  const int mine = threadIdx.x < p.c.M ? row[threadIdx.x] : -1;
  if (threadIdx.x == 0) {
    held = atomicExch(&p.c.count[s], 0);
    if (held < 0 || held > p.c.M) {
      flag(p.c.status, DROPKV_FLAG_BAD_LENGTH);
      held = min(max(held, 0), p.c.M);
    }
    if (held > 0) p.c.length[s] = 0;
  }
  __syncthreads();
  for (int col = threadIdx.x; col < held; col += 256) {
    const int pg = col < 256 ? mine : row[col];
    row[col] = -1;
    if (pg < 0 || pg >= p.c.P) {
      flag(p.c.status, KVCACHE_FLAG_BAD_PAGE);
    } else if (atomicSub(&p.c.refs[pg], 1) <= 0) {
      atomicAdd(&p.c.refs[pg], 1);
      flag(p.c.status, KVCACHE_FLAG_BAD_PAGE);
    }
  }
}

// ============================================================== reserve
__global__ void __launch_bounds__(kBook) reserve_kernel(const PageCall p) {
  __shared__ Names names;
  grid_dep_wait();
  const Cache& c = p.c;
  const Counts counts = load_counts(c, 0);
  if (p.seqs) claim_seqs(p, p.seqs, names);
  long long sum = 0;                        // pages wanted
  int turn = 0;
  for (int base = 0; base < p.n; base += kBook) {
    const int i = base + threadIdx.x;
    int need = 0, pages = 0, extra = 0;
    long long tokens = -1;                  // new length, -1: the entry is left out
    if (i < p.n) {
      const int s = seq_of(p.seqs, i);
      if (s < 0 || s >= c.S || (p.seqs && !first_named(p, names, i, s))) {
        flag(c.status, KVCACHE_FLAG_BAD_SEQ);
      } else {
        const int len = c.length[s], have = c.count[s];
        extra = p.extra[i];
        if (extra < 0 || len < 0 || have < 0 || have > c.M || have != pages_for(c, len)) {
          flag(c.status, DROPKV_FLAG_BAD_LENGTH);
        } else if ((long long)len + extra > (long long)c.M * c.page) {
          flag(c.status, DROPKV_FLAG_OVERFLOW);
        } else {
          tokens = (long long)len + extra;
          pages = pages_for(c, (int)tokens);
          need = pages - have;
        }
      }
    }
    long long total;
    const long long at = sum + block_scan(need, &total, turn);
    if (i < p.n) {
      p.offs[i] = (int)at;                  // (read only where the sum fits)
      p.entry[i] = make_int4((int)tokens, pages, need, extra);
    }
    sum += total;
  }
  __syncthreads();
  if (!find_pages(p, sum, counts, turn)) {
    if (p.granted)
      for (int i = threadIdx.x; i < p.n; i += kBook) p.granted[i] = 0;
    return;
  }
  grid_dep_launch();
  for (int k = threadIdx.x; k < sum; k += kBook) {
    const int i = entry_of(p.offs, p.n, k);
    const int4 e = p.entry[i];
    const int pg = p.list[k];
    c.table[(size_t)seq_of(p.seqs, i) * c.M + (e.y - e.z) + (k - p.offs[i])] = pg;
    c.refs[pg] = 1;
  }
  for (int i = threadIdx.x; i < p.n; i += kBook) {
    const int4 e = p.entry[i];
    if (p.granted) p.granted[i] = e.x < 0 ? 0 : e.w;
    if (e.x < 0) continue;
    const int s = seq_of(p.seqs, i);
    c.length[s] = e.x;
    c.count[s] = e.y;
  }
}

// ============================================================== fork
// entry: (source, destination or -1, pages held by both, pages of the
// branch); the list holds the pages of each entry's own copies in order.
__device__ __forceinline__ void fork_book(const PageCall& p, Names& names) {
  const Cache& c = p.c;
  const Counts counts = load_counts(c, 0);
  const int32_t *src = p.seqs, *dst = p.other;
  if (p.n <= kSmall) {
    for (int i = threadIdx.x; i < p.n; i += kBook) names.other[i] = src[i];
  } else {
    for (int i = threadIdx.x; i < p.n; i += kBook) {
      const int d = dst[i];
      if (d >= 0 && d < c.S) p.mark[d] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += kBook) {
      const int s = src[i];
      if (s >= 0 && s < c.S) p.mark[s] = 1;
    }
  }
  claim_seqs(p, dst, names);
  auto is_source = [&](int d) {
    if (p.n > kSmall) return p.mark[d] == 1;
    int any = 0;
#pragma unroll 8
    for (int j = 0; j < p.n; ++j) any |= names.other[j] == d;
    return any != 0;
  };
  long long sum = 0;                        // pages wanted
  int turn = 0;
  for (int base = 0; base < p.n; base += kBook) {
    const int i = base + threadIdx.x;
    int need = 0, len = 0, last = -1;       // (a sharing branch copies one page at most)
    int4 e = make_int4(0, -1, 0, 0);
    if (i < p.n) {
      const int s = src[i], d = dst[i];
      if (s < 0 || s >= c.S || d < 0 || d >= c.S) {
        flag(c.status, KVCACHE_FLAG_BAD_SEQ);
      } else {
        len = c.length[s];
        const int pages = c.count[s], d_len = c.length[d], d_pages = c.count[d];
        if (!first_named(p, names, i, d) || is_source(d) || d_pages != 0 || d_len != 0) {
          flag(c.status, KVCACHE_FLAG_BAD_SEQ);
        } else if (len < 0 || pages < 0 || pages > c.M || pages != pages_for(c, len)) {
          flag(c.status, DROPKV_FLAG_BAD_LENGTH);
        } else {
          const int both = p.share ? len >> c.page_log2 : 0;
          need = pages - both;
          e = make_int4(s, d, both, pages);
          if (p.share && need > 0) last = c.table[(size_t)s * c.M + both];
        }
      }
    }
    long long total;
    const long long at = sum + block_scan(need, &total, turn);
    if (i < p.n) {
      p.offs[i] = (int)at;                  // (read only where the sum fits)
      p.entry[i] = e;
      if (p.share && need > 0) p.from[at] = last;   // (at < n)
    }
    sum += total;
  }
  const bool ok = find_pages(p, sum, counts, turn);
  if (threadIdx.x == 0) p.offs[p.n] = ok ? (int)sum : -1;   // -1: nothing to do
  if (!ok) return;
  for (int k = threadIdx.x; k < sum; k += kBook) c.refs[p.list[k]] = 1;
  for (int i = threadIdx.x; i < p.n; i += kBook) {
    const int4 e = p.entry[i];
    if (e.y < 0) continue;
    c.length[e.y] = c.length[e.x];
    c.count[e.y] = e.w;
  }
}

constexpr int kCopyTeam = 256, kCopyUnroll = 4;
constexpr int kCopyChunk = kCopyTeam * kCopyUnroll * 16;   // bytes a CTA moves at a time

// CTA `team` of `teams` (kCopyTeam threads each): its share of two lists,
// table rows of the branches in pieces of kCopyTeam entries, then page bytes
// (page copy, layer, K or V, chunk).
__device__ __forceinline__ void fork_move(const PageCall& p, int row_pieces, int chunks, int team, int teams, int tid) {
  const Cache& c = p.c;
  const int copies = p.offs[p.n];
  if (copies < 0) return;
  for (int w = team; w < p.n * row_pieces; w += teams) {
    const int i = w / row_pieces, col = (w - i * row_pieces) * kCopyTeam + tid;
    const int4 e = p.entry[i];
    if (e.y < 0 || col >= e.w) continue;
    int pg;
    if (col < e.z) {
      pg = c.table[(size_t)e.x * c.M + col];
      if (pg >= 0 && pg < c.P) atomicAdd(&c.refs[pg], 1);
      else flag(c.status, KVCACHE_FLAG_BAD_PAGE);
    } else {
      pg = p.list[p.offs[i] + col - e.z];
    }
    c.table[(size_t)e.y * c.M + col] = pg;
  }
  const size_t page_bytes = (size_t)c.Hkv * c.page * c.d;
  const long long pieces = (long long)copies * c.layers * 2 * chunks;
  for (long long w = team; w < pieces; w += teams) {
    const int chunk = (int)(w % chunks);
    const long long x = w / chunks;
    const int which = (int)(x & 1);
    const int layer = (int)((x >> 1) % c.layers), k = (int)((x >> 1) / c.layers);
    const int to = p.list[k];
    int from;
    if (p.share) {
      from = p.from[k];
    } else {
      const int i = entry_of(p.offs, p.n, k);
      from = c.table[(size_t)p.entry[i].x * c.M + (k - p.offs[i])];   // (none is shared)
    }
    if (from < 0 || from >= c.P) {
      if (tid == 0) flag(c.status, KVCACHE_FLAG_BAD_PAGE);
      continue;
    }
    uint8_t* pool = which ? c.v : c.k;
    const uint8_t* a = pool + ((size_t)layer * c.P + from) * page_bytes;
    uint8_t* b = pool + ((size_t)layer * c.P + to) * page_bytes;
    const size_t at = (size_t)chunk * kCopyChunk + (size_t)tid * 16;
    uint4 r[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (at + u * kCopyTeam * 16 < page_bytes)
        r[u] = __ldcs(reinterpret_cast<const uint4*>(a + at + u * kCopyTeam * 16));
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (at + u * kCopyTeam * 16 < page_bytes)
        __stcs(reinterpret_cast<uint4*>(b + at + u * kCopyTeam * 16), r[u]);
    if (chunk == 0) {
      float* sc = which ? c.vs : c.ks;
      for (int h = tid; h < c.Hkv; h += kCopyTeam)
        sc[((size_t)layer * c.P + to) * c.Hkv + h] = sc[((size_t)layer * c.P + from) * c.Hkv + h];
    }
  }
}

__global__ void __launch_bounds__(kBook) fork_book_kernel(const PageCall p) {
  __shared__ Names names;
  grid_dep_wait();
  grid_dep_launch();
  fork_book(p, names);
}
// Both in one CTA, where little can be wanted: a launch less.
__global__ void __launch_bounds__(kBook) fork_one_kernel(const PageCall p, int row_pieces, int chunks) {
  __shared__ Names names;
  grid_dep_wait();
  grid_dep_launch();
  fork_book(p, names);
  __syncthreads();
  fork_move(p, row_pieces, chunks, threadIdx.x / kCopyTeam, kBook / kCopyTeam, threadIdx.x % kCopyTeam);
}
// Most copies (page, layer, K or V, chunk) and table entries of the one-CTA
// form: two rounds of its teams take as long as the second launch.
constexpr int kOnePieces = 2 * kBook / kCopyTeam, kOneRows = 1024;

__global__ void __launch_bounds__(kCopyTeam) fork_move_kernel(const PageCall p, int row_pieces, int chunks) {
  grid_dep_wait();
  grid_dep_launch();
  fork_move(p, row_pieces, chunks, blockIdx.x, gridDim.x, threadIdx.x);
}
// ============================================================== compact
// entry: (sequence or -1, old length, old pages, kept tokens).
// The table rows of the evicted sequences: old pages lose a reference, the
// new ones take their place.  Either the bookkeeping does it at once, leaving
// the old rows in p.rows for the gather (early: rows of up to kEarlyRows
// entries in all), or a third kernel after the gather (which then reads the
// table).
__device__ __forceinline__ void compact_row(const PageCall& p, int i, int col) {
  const Cache& c = p.c;
  const int4 e = p.entry[i];
  if (e.x < 0 || col >= e.z) return;
  int32_t* at = c.table + (size_t)e.x * c.M + col;
  const int pg = *at;
  if (p.early) p.rows[(size_t)i * c.M + col] = pg;
  if (pg < 0 || pg >= c.P) {
    flag(c.status, KVCACHE_FLAG_BAD_PAGE);
  } else if (atomicSub(&c.refs[pg], 1) <= 0) {
    atomicAdd(&c.refs[pg], 1);
    flag(c.status, KVCACHE_FLAG_BAD_PAGE);
  }
  *at = col < pages_for(c, e.w) ? p.list[p.offs[i] + col] : -1;
}

__device__ __forceinline__ void compact_book(const PageCall& p, Names& names) {
  const Cache& c = p.c;
  const Counts counts = load_counts(c, 0);
  if (p.seqs) claim_seqs(p, p.seqs, names);
  long long sum = 0;                        // pages wanted
  int turn = 0;
  for (int base = 0; base < p.n; base += kBook) {
    const int i = base + threadIdx.x;
    int need = 0;
    int4 e = make_int4(-1, 0, 0, 0);
    if (i < p.n) {
      const int s = seq_of(p.seqs, i), kept = p.kept_len[i];
      if (s < 0 || s >= c.S || (p.seqs && !first_named(p, names, i, s))) {
        flag(c.status, KVCACHE_FLAG_BAD_SEQ);
      } else {
        const int len = c.length[s], have = c.count[s];
        if (len < 0 || have < 0 || have > c.M || have != pages_for(c, len)) {
          flag(c.status, DROPKV_FLAG_BAD_LENGTH);
        } else if (kept < 0 || kept > len || kept > p.kept_stride) {
          flag(c.status, DROPKV_FLAG_BAD_K);
        } else {
          need = pages_for(c, kept);
          e = make_int4(s, len, have, kept);
        }
      }
    }
    long long total;
    const long long at = sum + block_scan(need, &total, turn);
    if (i < p.n) {
      p.offs[i] = (int)at;                  // (read only where the sum fits)
      p.entry[i] = e;
    }
    sum += total;
  }
  const bool ok = find_pages(p, sum, counts, turn);
  if (threadIdx.x == 0) p.offs[p.n] = ok ? (int)sum : -1;
  if (!ok) return;
  for (int k = threadIdx.x; k < sum; k += kBook) c.refs[p.list[k]] = 1;
  for (int i = threadIdx.x; i < p.n; i += kBook) {
    const int4 e = p.entry[i];
    if (e.x < 0) continue;
    c.length[e.x] = e.w;
    c.count[e.x] = pages_for(c, e.w);
  }
  if (p.early)
    for (int x = threadIdx.x; x < p.n * c.M; x += kBook) compact_row(p, x / c.M, x % c.M);
}

constexpr int kGatherTeam = 128, kGatherCtas = 12;   // threads of a CTA, CTAs per SM
constexpr int kGatherWaves = 8;
constexpr int kMaxPage = 128;
static_assert(kMaxPage <= kGatherTeam, "a thread looks up one row of a page");
struct Gather {
  size_t row[kMaxPage];                         // source row, ~0: none
  float scale[2][kMaxPage];
  float top[2][kGatherTeam / 32];
  int offs[kSmall + 1];                         // the call's entries, where they fit
  int4 entry[kSmall];
};

// Team `team` of `teams` (kGatherTeam threads, barrier `bar`) fills one (new
// page, layer, head) at a time: the kept positions give each row's source, then the first
// vectors of the rows and the scales are on their way together; the new scale
// is the largest, and codes of other scales are rounded again.  Bound by the
// chain position -> table -> row, so the CTAs are many and small.
template <int VB, int CODE>
__device__ __forceinline__ void compact_move(const PageCall& p, Gather& g, int team, int teams, int tid, uint32_t bar) {
  using Vec = typename std::conditional<VB == 16, uint4, uint2>::type;
  constexpr int kBatch = 2;
  const Cache& c = p.c;
  const int taken = p.offs[p.n];
  if (taken < 0) return;
  const int lane = tid & 31, warp = tid >> 5;
  const int units = c.d / VB;                   // at most 16
  const uint32_t per = (65536 + units - 1) / units;   // u / units == u * per >> 16 for u < 2048
  const int* offs = p.offs;
  const int4* entry = p.entry;
  if (p.n <= kSmall) {
    for (int i = tid; i < p.n; i += kGatherTeam) {
      g.offs[i] = p.offs[i];
      g.entry[i] = p.entry[i];
    }
    offs = g.offs;
    entry = g.entry;
    named_bar(bar, kGatherTeam);
  }
  const long long work = (long long)taken * c.layers * c.Hkv;
  for (long long w = team; w < work; w += teams) {
    const int h = (int)(w % c.Hkv);
    const long long x = w / c.Hkv;
    const int layer = (int)(x % c.layers), k = (int)(x / c.layers);
    const int i = entry_of(offs, p.n, k);
    const int4 e = entry[i];
    const int first = (k - offs[i]) << c.page_log2;
    const int rows = min(c.page, e.w - first), to = p.list[k];
    float ks = 0.f, vs = 0.f;
    if (tid < rows) {
      const int idx = p.kept_idx[(((size_t)layer * p.n + i) * c.Hkv + h) * p.kept_stride + first + tid];
      size_t row = ~(size_t)0;
      if (idx < 0 || idx >= e.y) {
        flag(c.status, DROPKV_FLAG_BAD_K);
      } else {
        const int col = idx >> c.page_log2;
        const int pg = p.early ? p.rows[(size_t)i * c.M + col] : c.table[(size_t)e.x * c.M + col];
        if (pg < 0 || pg >= c.P) {
          flag(c.status, KVCACHE_FLAG_BAD_PAGE);
        } else {
          const size_t u = ((size_t)layer * c.P + pg) * c.Hkv + h;
          row = u * c.page + (idx & (c.page - 1));
          ks = c.ks[u];
          vs = c.vs[u];
        }
      }
      g.row[tid] = row;
    }
    named_bar(bar, kGatherTeam);
    const int vecs = rows * units;
    Vec val[kBatch][2];
    auto load = [&](int base) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int u = base + b * kGatherTeam + tid;
        val[b][0] = val[b][1] = Vec{};
        if (u >= vecs) continue;
        const int r = (int)((uint32_t)u * per >> 16), off = (u - r * units) * VB;
        const size_t row = g.row[r];
        if (row != ~(size_t)0) {
          val[b][0] = *reinterpret_cast<const Vec*>(c.k + row * c.d + off);
          val[b][1] = *reinterpret_cast<const Vec*>(c.v + row * c.d + off);
        }
      }
    };
    load(0);
    if (tid < rows) {
      g.scale[0][tid] = ks;
      g.scale[1][tid] = vs;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ks = fmaxf(ks, __shfl_xor_sync(0xffffffffu, ks, o));
      vs = fmaxf(vs, __shfl_xor_sync(0xffffffffu, vs, o));
    }
    if (lane == 0) {
      g.top[0][warp] = ks;
      g.top[1][warp] = vs;
    }
    named_bar(bar, kGatherTeam);
    float top[2] = {kScaleMin, kScaleMin};
#pragma unroll
    for (int q = 0; q < kGatherTeam / 32; ++q) {
      top[0] = fmaxf(top[0], g.top[0][q]);
      top[1] = fmaxf(top[1], g.top[1][q]);
    }
    const size_t ut = ((size_t)layer * c.P + to) * c.Hkv + h;
    if (tid == 0) {
      c.ks[ut] = top[0];
      c.vs[ut] = top[1];
    }
    for (int base = 0; base < vecs; base += kBatch * kGatherTeam) {
      if (base > 0) load(base);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int u = base + b * kGatherTeam + tid;
        if (u >= vecs) continue;
        const int r = (int)((uint32_t)u * per >> 16), off = (u - r * units) * VB;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float from = g.scale[q][r];
          if (from != top[q]) {
            const float ratio = from / top[q];
            uint32_t* wv = reinterpret_cast<uint32_t*>(&val[b][q]);
#pragma unroll
            for (int s = 0; s < VB / 4; ++s) wv[s] = rescale4(wv[s], from, top[q], ratio, CODE);
          }
        }
        const size_t dst = (ut * c.page + r) * c.d + off;
        *reinterpret_cast<Vec*>(c.k + dst) = val[b][0];
        *reinterpret_cast<Vec*>(c.v + dst) = val[b][1];
      }
    }
    named_bar(bar, kGatherTeam);                        // the rows are rewritten next
  }
}

__global__ void __launch_bounds__(kBook) compact_book_kernel(const PageCall p) {
  __shared__ Names names;
  grid_dep_wait();
  grid_dep_launch();
  compact_book(p, names);
}
template <int VB, int CODE>
__global__ void __launch_bounds__(kGatherTeam, kGatherCtas) compact_move_kernel(const PageCall p) {
  __shared__ Gather g;
  grid_dep_wait();
  grid_dep_launch();
  compact_move<VB, CODE>(p, g, blockIdx.x, gridDim.x, threadIdx.x, 1);
}
// Both in one CTA, where no team has more than one to fill (1 x 100 tokens, 2
// heads: a launch less, 16.8 -> 14.5 us with the fork and the free before it;
// two each would lose).
template <int VB, int CODE>
__global__ void __launch_bounds__(kBook) compact_one_kernel(const PageCall p) {
  __shared__ Names names;
  __shared__ Gather g[kBook / kGatherTeam];
  grid_dep_wait();
  grid_dep_launch();
  compact_book(p, names);
  __syncthreads();
  const int team = threadIdx.x / kGatherTeam;
  compact_move<VB, CODE>(p, g[team], team, kBook / kGatherTeam, threadIdx.x % kGatherTeam, 1 + team);
}
__global__ void __launch_bounds__(kCopyTeam) compact_commit_kernel(const PageCall p, int row_pieces) {
  grid_dep_wait();
  grid_dep_launch();
  if (p.offs[p.n] < 0) return;
  for (int w = blockIdx.x; w < p.n * row_pieces; w += gridDim.x) {
    const int i = w / row_pieces;
    compact_row(p, i, (w - i * row_pieces) * kCopyTeam + threadIdx.x);
  }
}
}  // namespace

PagePlan make_page_plan(int S, int P) {
  PagePlan w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  w.claim = take((size_t)S * 4);
  w.from = take((size_t)S * 4);
  w.mark = take((size_t)S * 4);
  w.offs = take(((size_t)S + 1) * 4);
  w.entry = take((size_t)S * 16);
  w.list = take((size_t)P * 4);
  w.rows = take((size_t)kEarlyRows * 4);
  w.total = off;
  return w;
}

cudaError_t launch_free(const PageCall& p, cudaStream_t st) {
  return launch_pdl(free_kernel, dim3(p.n), dim3(256), 0, st, p);
}

cudaError_t launch_reserve(const PageCall& p, cudaStream_t st) {
  return launch_pdl(reserve_kernel, dim3(1), dim3(kBook), 0, st, p);
}

cudaError_t launch_fork(const PageCall& p, int sms, cudaStream_t st) {
  const Cache& c = p.c;
  const int row_pieces = (c.M + kCopyTeam - 1) / kCopyTeam;
  const int chunks = (int)(((size_t)c.Hkv * c.page * c.d + kCopyChunk - 1) / kCopyChunk);
  const long long pages = (long long)p.n * (p.share ? 1 : c.M);   // that can be copied
  if (pages * c.layers * 2 * chunks <= kOnePieces && (long long)p.n * c.M <= kOneRows)
    return launch_pdl(fork_one_kernel, dim3(1), dim3(kBook), 0, st, p, row_pieces, chunks);
  const cudaError_t e = launch_pdl(fork_book_kernel, dim3(1), dim3(kBook), 0, st, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(fork_move_kernel, dim3(sms * 16), dim3(kCopyTeam), 0, st, p, row_pieces, chunks);
}

cudaError_t launch_compact_pages(const PageCall& p, int sms, cudaStream_t st) {
  const Cache& c = p.c;
  const int row_pieces = (c.M + kCopyTeam - 1) / kCopyTeam;
  const bool int8 = c.code == KVCACHE_INT8;
  // (new page, layer, head)s there can be
  const long long most =
      std::min<long long>(c.P, p.n * (((long long)p.kept_stride + c.page - 1) / c.page)) * c.layers * c.Hkv;
  if (most <= kBook / kGatherTeam && p.early) {
    auto one = c.d % 16 == 0 ? (int8 ? compact_one_kernel<16, KVCACHE_INT8> : compact_one_kernel<16, KVCACHE_E4M3>)
                             : (int8 ? compact_one_kernel<8, KVCACHE_INT8> : compact_one_kernel<8, KVCACHE_E4M3>);
    return launch_pdl(one, dim3(1), dim3(kBook), 0, st, p);
  }
  cudaError_t e = launch_pdl(compact_book_kernel, dim3(1), dim3(kBook), 0, st, p);
  if (e != cudaSuccess) return e;
  auto move = c.d % 16 == 0 ? (int8 ? compact_move_kernel<16, KVCACHE_INT8> : compact_move_kernel<16, KVCACHE_E4M3>)
                            : (int8 ? compact_move_kernel<8, KVCACHE_INT8> : compact_move_kernel<8, KVCACHE_E4M3>);
  // a CTA for each (page, layer, head) there can be, up to kGatherWaves full
  // loads of the GPU: those with nothing to do leave at once, and the others
  // need not come out even over the resident CTAs
  const unsigned grid = (unsigned)std::max(1LL, std::min<long long>(most, (long long)sms * kGatherCtas * kGatherWaves));
  e = launch_pdl(move, dim3(grid), dim3(kGatherTeam), 0, st, p);
  if (e != cudaSuccess || p.early) return e;
  const long long pieces = (long long)p.n * row_pieces;
  return launch_pdl(compact_commit_kernel, dim3((unsigned)std::min<long long>(pieces, sms * 8)), dim3(kCopyTeam), 0, st,
                    p, row_pieces);
}

}  // namespace kvcache
