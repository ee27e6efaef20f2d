// Pages of the paged 8-bit cache: taking, sharing, copying, compacting and
// releasing them.
//
// A page is free when its reference count is 0, and the lowest free pages are
// taken in order: there is no free list whose order would depend on the order
// of atomics, and results depend on the state alone.  The integer bookkeeping
// of a call (who wants how many pages, which pages those are) is one CTA's
// work: block scans over the call's entries and over the reference counts,
// 16 counts a thread at a time.  What grows with the cache (page bytes, table
// rows, reference counts of shared pages) is a second kernel's, spread over
// the GPU and launched with programmatic dependent launch.
#include "kvcache_internal.cuh"
#include "sm103_ptx.cuh"

namespace kvcache {
namespace {

using dropkv::grid_dep_launch;
using dropkv::grid_dep_wait;
using dropkv::launch_pdl;

constexpr int kBook = 1024;                // threads of a bookkeeping CTA
constexpr int kBookWarps = kBook / 32;

__device__ __forceinline__ int seq_of(const int32_t* seqs, int i) { return seqs ? seqs[i] : i; }
__device__ __forceinline__ int pages_for(const Cache& c, int tokens) {
  return (int)(((unsigned)tokens + (unsigned)c.page - 1u) >> c.page_log2);
}

// Exclusive sum over the block's threads; *total gets the sum of all.
__device__ __forceinline__ int block_scan(int x, int* total) {
  __shared__ int warp_sum[kBookWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();                         // the last use of warp_sum is over
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int w = warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
  return before + inc - x;
}

// The block marks the call's sequences: claim[s] = lowest index that names s.
__device__ __forceinline__ void claim_seqs(const PageCall& p, const int32_t* seqs) {
  for (int i = threadIdx.x; i < p.n; i += kBook) {
    const int s = seqs[i];
    if (s >= 0 && s < p.c.S) p.claim[s] = INT32_MAX;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += kBook) {
    const int s = seqs[i];
    if (s >= 0 && s < p.c.S) atomicMin(&p.claim[s], i);
  }
  __syncthreads();
}

// The `want` lowest free pages into p.list; false (and a flag) if there are fewer.
__device__ __forceinline__ bool find_pages(const PageCall& p, int want) {
  constexpr int kPer = 16;
  int found = 0;
  for (int base = 0; base < p.c.P && found < want; base += kBook * kPer) {
    const int first = base + threadIdx.x * kPer;
    int4 r[kPer / 4];
#pragma unroll
    for (int u = 0; u < kPer / 4; ++u) {
      const int a = first + 4 * u;
      if (a + 4 <= p.c.P) {
        r[u] = *reinterpret_cast<const int4*>(p.c.refs + a);
      } else {
        r[u] = make_int4(1, 1, 1, 1);
        if (a < p.c.P) r[u].x = p.c.refs[a];
        if (a + 1 < p.c.P) r[u].y = p.c.refs[a + 1];
        if (a + 2 < p.c.P) r[u].z = p.c.refs[a + 2];
      }
    }
    uint32_t free_bits = 0;
#pragma unroll
    for (int u = 0; u < kPer / 4; ++u) {
      free_bits |= (r[u].x == 0 ? 1u : 0u) << (4 * u) | (r[u].y == 0 ? 2u : 0u) << (4 * u) |
                   (r[u].z == 0 ? 4u : 0u) << (4 * u) | (r[u].w == 0 ? 8u : 0u) << (4 * u);
    }
    int total;
    int at = found + block_scan(__popc(free_bits), &total);
    while (free_bits && at < want) {
      const int bit = __ffs(free_bits) - 1;
      free_bits &= free_bits - 1;
      p.list[at++] = first + bit;
    }
    found += total;
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
  if (threadIdx.x == 0) {
    held = atomicExch(&p.c.count[s], 0);
    if (held < 0 || held > p.c.M) {
      flag(p.c.status, DROPKV_FLAG_BAD_LENGTH);
      held = min(max(held, 0), p.c.M);
    }
    if (held > 0) p.c.length[s] = 0;
  }
  __syncthreads();
  int32_t* row = p.c.table + (size_t)s * p.c.M;
  for (int col = threadIdx.x; col < held; col += 256) {
    const int pg = row[col];
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
  grid_dep_wait();
  const Cache& c = p.c;
  if (p.seqs) claim_seqs(p, p.seqs);
  int sum = 0;
  for (int base = 0; base < p.n; base += kBook) {
    const int i = base + threadIdx.x;
    int need = 0, pages = 0;
    long long tokens = -1;                  // new length, -1: the entry is left out
    if (i < p.n) {
      const int s = seq_of(p.seqs, i);
      if (s < 0 || s >= c.S || (p.seqs && p.claim[s] != i)) {
        flag(c.status, KVCACHE_FLAG_BAD_SEQ);
      } else {
        const int extra = p.extra[i], len = c.length[s], have = c.count[s];
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
    int total;
    const int at = sum + block_scan(need, &total);
    if (i < p.n) {
      p.offs[i] = at;
      p.entry[i] = make_int4((int)tokens, pages, need, 0);
    }
    sum += total;
  }
  __syncthreads();
  if (!find_pages(p, sum)) return;
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
    if (e.x < 0) continue;
    const int s = seq_of(p.seqs, i);
    c.length[s] = e.x;
    c.count[s] = e.y;
  }
}

// ============================================================== fork
// entry: (source, destination or -1, pages held by both, pages of the
// branch); the list holds the pages of each entry's own copies in order.
__global__ void __launch_bounds__(kBook) fork_book_kernel(const PageCall p) {
  grid_dep_wait();
  const Cache& c = p.c;
  const int32_t *src = p.seqs, *dst = p.other;
  claim_seqs(p, dst);
  for (int i = threadIdx.x; i < p.n; i += kBook) {
    const int d = dst[i];
    if (d >= 0 && d < c.S) p.mark[d] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += kBook) {
    const int s = src[i];
    if (s >= 0 && s < c.S) p.mark[s] = 1;
  }
  __syncthreads();
  int sum = 0;
  for (int base = 0; base < p.n; base += kBook) {
    const int i = base + threadIdx.x;
    int need = 0;
    int4 e = make_int4(0, -1, 0, 0);
    if (i < p.n) {
      const int s = src[i], d = dst[i];
      if (s < 0 || s >= c.S || d < 0 || d >= c.S || p.claim[d] != i || p.mark[d] == 1 || c.count[d] != 0 ||
          c.length[d] != 0) {
        flag(c.status, KVCACHE_FLAG_BAD_SEQ);
      } else {
        const int len = c.length[s], pages = c.count[s];
        if (len < 0 || pages < 0 || pages > c.M || pages != pages_for(c, len)) {
          flag(c.status, DROPKV_FLAG_BAD_LENGTH);
        } else {
          const int both = p.share ? len >> c.page_log2 : 0;
          need = pages - both;
          e = make_int4(s, d, both, pages);
        }
      }
    }
    int total;
    const int at = sum + block_scan(need, &total);
    if (i < p.n) {
      p.offs[i] = at;
      p.entry[i] = e;
    }
    sum += total;
  }
  __syncthreads();
  const bool ok = find_pages(p, sum);
  if (threadIdx.x == 0) p.offs[p.n] = ok ? sum : -1;   // -1: nothing to do
  if (!ok) return;
  for (int k = threadIdx.x; k < sum; k += kBook) c.refs[p.list[k]] = 1;
  for (int i = threadIdx.x; i < p.n; i += kBook) {
    const int4 e = p.entry[i];
    if (e.y < 0) continue;
    c.length[e.y] = c.length[e.x];
    c.count[e.y] = e.w;
  }
}

constexpr int kCopyThreads = 256, kCopyUnroll = 4;
constexpr int kCopyChunk = kCopyThreads * kCopyUnroll * 16;   // bytes a CTA moves at a time

// The blocks share out two lists: table rows of the branches in pieces of
// kCopyThreads entries, then page bytes (page copy, layer, K or V, chunk).
__global__ void __launch_bounds__(kCopyThreads) fork_move_kernel(const PageCall p, int row_pieces, int chunks) {
  grid_dep_wait();
  grid_dep_launch();
  const Cache& c = p.c;
  const int copies = p.offs[p.n];
  if (copies < 0) return;
  const int tid = threadIdx.x;
  for (int w = blockIdx.x; w < p.n * row_pieces; w += gridDim.x) {
    const int i = w / row_pieces, col = (w - i * row_pieces) * kCopyThreads + tid;
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
  for (long long w = blockIdx.x; w < pieces; w += gridDim.x) {
    const int chunk = (int)(w % chunks);
    const long long x = w / chunks;
    const int which = (int)(x & 1);
    const int layer = (int)((x >> 1) % c.layers), k = (int)((x >> 1) / c.layers);
    const int i = entry_of(p.offs, p.n, k);
    const int4 e = p.entry[i];
    const int from = c.table[(size_t)e.x * c.M + e.z + (k - p.offs[i])], to = p.list[k];
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
      if (at + u * kCopyThreads * 16 < page_bytes)
        r[u] = __ldcs(reinterpret_cast<const uint4*>(a + at + u * kCopyThreads * 16));
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (at + u * kCopyThreads * 16 < page_bytes)
        __stcs(reinterpret_cast<uint4*>(b + at + u * kCopyThreads * 16), r[u]);
    if (chunk == 0) {
      float* sc = which ? c.vs : c.ks;
      for (int h = tid; h < c.Hkv; h += kCopyThreads)
        sc[((size_t)layer * c.P + to) * c.Hkv + h] = sc[((size_t)layer * c.P + from) * c.Hkv + h];
    }
  }
}

// ============================================================== compact
// entry: (sequence or -1, old length, old pages, kept tokens).
__global__ void __launch_bounds__(kBook) compact_book_kernel(const PageCall p) {
  grid_dep_wait();
  const Cache& c = p.c;
  if (p.seqs) claim_seqs(p, p.seqs);
  int sum = 0;
  for (int base = 0; base < p.n; base += kBook) {
    const int i = base + threadIdx.x;
    int need = 0;
    int4 e = make_int4(-1, 0, 0, 0);
    if (i < p.n) {
      const int s = seq_of(p.seqs, i);
      if (s < 0 || s >= c.S || (p.seqs && p.claim[s] != i)) {
        flag(c.status, KVCACHE_FLAG_BAD_SEQ);
      } else {
        const int len = c.length[s], have = c.count[s], kept = p.kept_len[i];
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
    int total;
    const int at = sum + block_scan(need, &total);
    if (i < p.n) {
      p.offs[i] = at;
      p.entry[i] = e;
    }
    sum += total;
  }
  __syncthreads();
  const bool ok = find_pages(p, sum);
  if (threadIdx.x == 0) p.offs[p.n] = ok ? sum : -1;
  if (!ok) return;
  for (int k = threadIdx.x; k < sum; k += kBook) c.refs[p.list[k]] = 1;
  for (int i = threadIdx.x; i < p.n; i += kBook) {
    const int4 e = p.entry[i];
    if (e.x < 0) continue;
    c.length[e.x] = e.w;
    c.count[e.x] = pages_for(c, e.w);
  }
}

constexpr int kGatherThreads = 128;
constexpr int kMaxPage = 128;

// A CTA fills one (new page, layer, head) at a time: the kept positions give
// each row's source and its scales, the new scale is their largest, then the
// rows are moved VB bytes at a time.
template <int VB>
__global__ void __launch_bounds__(kGatherThreads) compact_move_kernel(const PageCall p) {
  grid_dep_wait();
  grid_dep_launch();
  const Cache& c = p.c;
  const int taken = p.offs[p.n];
  if (taken < 0) return;
  __shared__ size_t s_row[kMaxPage];            // source row, ~0: none
  __shared__ float s_scale[2][kMaxPage];
  __shared__ float s_max[2][kGatherThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = c.d / VB;
  const long long work = (long long)taken * c.layers * c.Hkv;
  for (long long w = blockIdx.x; w < work; w += gridDim.x) {
    const int h = (int)(w % c.Hkv);
    const long long x = w / c.Hkv;
    const int layer = (int)(x % c.layers), k = (int)(x / c.layers);
    const int i = entry_of(p.offs, p.n, k);
    const int4 e = p.entry[i];
    const int first = (k - p.offs[i]) << c.page_log2;
    const int rows = min(c.page, e.w - first), to = p.list[k];
    float ks = 0.f, vs = 0.f;
    if (tid < rows) {
      const int idx = p.kept_idx[(((size_t)layer * p.n + i) * c.Hkv + h) * p.kept_stride + first + tid];
      size_t row = ~(size_t)0;
      if (idx < 0 || idx >= e.y) {
        flag(c.status, DROPKV_FLAG_BAD_K);
      } else {
        const int pg = c.table[(size_t)e.x * c.M + (idx >> c.page_log2)];
        if (pg < 0 || pg >= c.P) {
          flag(c.status, KVCACHE_FLAG_BAD_PAGE);
        } else {
          const size_t u = ((size_t)layer * c.P + pg) * c.Hkv + h;
          row = u * c.page + (idx & (c.page - 1));
          ks = c.ks[u];
          vs = c.vs[u];
        }
      }
      s_row[tid] = row;
      s_scale[0][tid] = ks;
      s_scale[1][tid] = vs;
    }
    float km = ks, vm = vs;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, o));
      vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
    }
    if (lane == 0) {
      s_max[0][warp] = km;
      s_max[1][warp] = vm;
    }
    __syncthreads();
    float top[2] = {kScaleMin, kScaleMin};
#pragma unroll
    for (int q = 0; q < kGatherThreads / 32; ++q) {
      top[0] = fmaxf(top[0], s_max[0][q]);
      top[1] = fmaxf(top[1], s_max[1][q]);
    }
    const size_t ut = ((size_t)layer * c.P + to) * c.Hkv + h;
    if (tid == 0) {
      c.ks[ut] = top[0];
      c.vs[ut] = top[1];
    }
    using Vec = typename std::conditional<VB == 16, uint4, uint2>::type;
    for (int u = tid; u < rows * units; u += kGatherThreads) {
      const int r = u / units, off = (u - r * units) * VB;
      const size_t row = s_row[r];
      Vec val[2] = {};
      if (row != ~(size_t)0) {
        val[0] = *reinterpret_cast<const Vec*>(c.k + row * c.d + off);
        val[1] = *reinterpret_cast<const Vec*>(c.v + row * c.d + off);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float from = s_scale[q][r];
        if (from != top[q]) {
          const float ratio = from / top[q];
          uint32_t* wv = reinterpret_cast<uint32_t*>(&val[q]);
#pragma unroll
          for (int b = 0; b < VB / 4; ++b) wv[b] = rescale4(wv[b], from, top[q], ratio, c.code);
        }
      }
      const size_t dst = (ut * c.page + r) * c.d + off;
      *reinterpret_cast<Vec*>(c.k + dst) = val[0];
      *reinterpret_cast<Vec*>(c.v + dst) = val[1];
    }
    __syncthreads();                        // the shared rows are rewritten next
  }
}

// The table rows of the evicted sequences: old pages lose a reference, the
// new ones take their place (after every row has been gathered).
__global__ void __launch_bounds__(kCopyThreads) compact_commit_kernel(const PageCall p, int row_pieces) {
  grid_dep_wait();
  grid_dep_launch();
  const Cache& c = p.c;
  if (p.offs[p.n] < 0) return;
  for (int w = blockIdx.x; w < p.n * row_pieces; w += gridDim.x) {
    const int i = w / row_pieces, col = (w - i * row_pieces) * kCopyThreads + threadIdx.x;
    const int4 e = p.entry[i];
    if (e.x < 0 || col >= e.z) continue;
    int32_t* at = c.table + (size_t)e.x * c.M + col;
    const int pg = *at;
    if (pg < 0 || pg >= c.P) {
      flag(c.status, KVCACHE_FLAG_BAD_PAGE);
    } else if (atomicSub(&c.refs[pg], 1) <= 0) {
      atomicAdd(&c.refs[pg], 1);
      flag(c.status, KVCACHE_FLAG_BAD_PAGE);
    }
    *at = col < pages_for(c, e.w) ? p.list[p.offs[i] + col] : -1;
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
  w.mark = take((size_t)S * 4);
  w.offs = take(((size_t)S + 1) * 4);
  w.entry = take((size_t)S * 16);
  w.list = take((size_t)P * 4);
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
  const cudaError_t e = launch_pdl(fork_book_kernel, dim3(1), dim3(kBook), 0, st, p);
  if (e != cudaSuccess) return e;
  const int row_pieces = (p.c.M + kCopyThreads - 1) / kCopyThreads;
  const int chunks = (int)(((size_t)p.c.Hkv * p.c.page * p.c.d + kCopyChunk - 1) / kCopyChunk);
  return launch_pdl(fork_move_kernel, dim3(sms * 8), dim3(kCopyThreads), 0, st, p, row_pieces, chunks);
}

cudaError_t launch_compact_pages(const PageCall& p, int sms, cudaStream_t st) {
  cudaError_t e = launch_pdl(compact_book_kernel, dim3(1), dim3(kBook), 0, st, p);
  if (e != cudaSuccess) return e;
  const dim3 grid(sms * 12);
  if (p.c.d % 16 == 0) e = launch_pdl(compact_move_kernel<16>, grid, dim3(kGatherThreads), 0, st, p);
  else e = launch_pdl(compact_move_kernel<8>, grid, dim3(kGatherThreads), 0, st, p);
  if (e != cudaSuccess) return e;
  const int row_pieces = (p.c.M + kCopyThreads - 1) / kCopyThreads;
  const long long pieces = (long long)p.n * row_pieces;
  return launch_pdl(compact_commit_kernel, dim3((unsigned)std::min<long long>(pieces, sms * 8)), dim3(kCopyThreads), 0,
                    st, p, row_pieces);
}

}  // namespace kvcache
