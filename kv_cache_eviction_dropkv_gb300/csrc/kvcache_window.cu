// A prompt's causal attention over a sliding window with the first tokens
// kept visible: row i sees keys j <= i with j > i - W or j < S.
//
//   o_i = sum_j exp(x_ij - m_i) v_j / sum_j exp(x_ij - m_i),  x_ij = q_i . k_j / sqrt(d)
//
// 4 d operations for each visible (row, key): for windows of a few hundred
// tokens and more it is bound by the tensor cores (and, one step behind, by
// the exponentials: 128 x 128 of them against 2 x 128^3 multiply-adds per
// tile), so the tiles go through tcgen05 with TMEM accumulators.
//
// One CTA per SM works through items: two 128-row query tiles of one head, t
// and t + 1, one per softmax group of four warps; thread r of a group owns
// TMEM lane r, the whole of its row, so a row's maximum and sum need no
// exchange between threads.  Both walk one list of 128-key tiles: those with
// first tokens, then those the two windows reach.  Per key tile and group:
// S = Q K^T into the group's TMEM columns; P = 2^(x - ref), with a reference
// that moves only when it must, written back over S as bf16 pairs; O += P V
// with P read from tensor memory.  The MMA warp alternates between the groups,
// so one group's products run under the other's softmax.  Issuing is what
// bounds the kernel (an MMA of 128 x 128 x 16 is issued about as fast as it
// runs, and S = Q K^T reads both operands from shared memory at its full
// rate), so the MMA warp is spared everything else: the items' lists
// follow one another as one row of entries, K of an entry comes with V of the
// entry before as one pair on one barrier, and the softmax groups release a
// pair when their S of it is complete, which every product issued before it
// then is too.  The next item's Q, K and first S so come in under the last
// one's softmax and output.  A group skips tiles outside its own window; only
// tiles that cut the diagonal or a window's edge are masked, and a tile of
// which only the first kNarrow keys are first tokens is taken kNarrow keys wide.
#include "kvcache_internal.cuh"
#include "sm103_ptx.cuh"

namespace kvcache {
namespace {

using namespace dropkv;

constexpr int kQT = 128;                          // rows of a query tile, keys of a key tile
constexpr int kTileB = kQT * kDPad * 2;           // 32 KB: two SW128 blocks of 64 columns
constexpr int kHalfB = kTileB / 2;
constexpr int kProducer = 8, kIssuer = 9, kWalker = 10, kWinThreads = 32 * 12;   // warp 11 idle (register shares)
constexpr int kOffQ = 0, kOffK = 2 * kTileB, kOffV = 4 * kTileB, kOffSmall = 6 * kTileB;
constexpr uint32_t kCols = 512;                   // group g: S / P at [128 g, +128), O at [256 + 128 g, +128)
constexpr float kMove = 24.0f;                    // base-2 logarithm by which a maximum may pass its reference
constexpr uint64_t kDrain = 20000000ull;          // 20 ms to drain copies after an abort

constexpr int kNarrow = 32;
constexpr int kSplitWindow = 1536;                // windows from which on P goes in halves

// The key tiles of an item: list entry i is key tile tile(i).  Group 0 (query
// tile t[0], -1: none) takes all entries but the last, group 1 (t[1] = t[0] +
// 1) all but `skip`, the one tile that only group 0's window may reach.
struct List {
  int t[2];
  int ns, s2, n;                                  // tiles [0, ns), then s2, s2 + 1, ...: n entries
  int skip;
  int narrow;                                     // entry that is taken kNarrow keys wide (-1: none)
  __device__ __forceinline__ int tile(int i) const { return i < ns ? i : s2 + (i - ns); }
  __device__ __forceinline__ bool takes(int g, int i) const {
    return g ? i < n && i != skip : t[0] >= 0 && i < n - 1;
  }
};
__device__ __forceinline__ List make_list(const WindowCall& p, int t0, int t1) {
  List l;
  l.t[0] = t0;
  l.t[1] = t1;
  // first key tiles the groups' windows reach, and the tiles that hold first tokens
  const int lo1 = p.window > 0 ? max(0, t1 * kQT - p.window + 1) / kQT : 0;
  const int lo = t0 >= 0 && p.window > 0 ? max(0, t0 * kQT - p.window + 1) / kQT : lo1;
  const int sink_tiles = p.window > 0 ? (min(p.sinks, p.n_max) + kQT - 1) / kQT : 0;
  l.ns = min(sink_tiles, lo);                     // those before both windows
  l.s2 = lo;
  l.n = l.ns + (t1 + 1 - l.s2);
  l.skip = lo < lo1 && lo >= sink_tiles ? l.ns : -1;
  l.narrow = l.ns > 0 && l.ns == sink_tiles && p.sinks - (l.ns - 1) * kQT <= kNarrow ? l.ns - 1 : -1;
  return l;
}

// The items of the call in order: chunks of 32 sequences, in a chunk by
// position, the last pair of query tiles first (the last tile of a sequence is
// group 1's), there sequence by sequence, heads innermost.  Round r gives every
// CTA one item, odd rounds from the last CTA to the first: costs fall along
// the order, so that evens them out (causal, 8192 tokens, 32 heads: the longest
// CTA has 1.02 instead of 1.14 of the mean, 385 -> 347 us; eight sequences of 2
// to 4096 tokens 119 -> 88).  One warp walks the order and hands the items to
// the others through a ring.
__device__ __forceinline__ int length_of(const WindowCall& p, int b) {
  const int nb = p.lengths ? p.lengths[b] : p.n_max;
  return nb < 0 || nb > p.n_max ? 0 : nb;
}
struct Item {
  int b, hq, nb;
  List list;
};
// Ring slots.  The softmax warps hold the item they are at; the MMA warp looks
// one item ahead and may be three before a group that passes over items.
constexpr int kItems = 8;
constexpr int kWalkerWaits = 3600;                // waits (of 1 s) for a slot
constexpr int kTakers = 10;                       // softmax warps, MMA warp, producer
struct Ring {
  uint64_t full[kItems], empty[kItems];
  int4 item[kItems];                              // sequence (-1: no more), head, length, last query tile
};
enum Got { kGaveUp = -1, kEnd = 0, kItem = 1 };

// Item `k` for a taker; wait(barrier, phase) waits, arrive(barrier) arrives once for it.
template <typename Wait, typename Arrive>
__device__ __forceinline__ Got take_item(const WindowCall& p, Ring& ring, uint32_t k, Item* w, Wait wait,
                                         Arrive arrive) {
  const uint32_t slot = k % kItems;
  if (!wait(&ring.full[slot], k / kItems)) return kGaveUp;
  const int4 x = ring.item[slot];
  arrive(&ring.empty[slot]);
  if (x.x < 0) return kEnd;
  w->b = x.x;
  w->hq = x.y;
  w->nb = x.z;
  w->list = make_list(p, x.w - 1, x.w);
  return kItem;
}

// The walking warp: false if a wait gave up.
template <typename Wait>
__device__ __forceinline__ bool walk_items(const WindowCall& p, Ring& ring, int lane, Wait wait) {
  long long first = 0, width = 0;                 // items before the level, items of it
  int b0 = -32, nb = 0, pairs = 0;                // the lane's sequence: b0 + lane
  int level = 0;                                  // pair of query tiles, from the sequence's start
  uint32_t at_level = 0;                          // lanes whose sequences have it
  for (uint32_t r = 0;; ++r) {
    const long long it = (long long)r * gridDim.x + (r & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    bool more = true;
    while (more && it >= first + width) {
      first += width;
      width = 0;
      if (--level < 0) {
        b0 += 32;
        more = b0 < p.B;
        nb = b0 + lane < p.B ? length_of(p, b0 + lane) : 0;
        pairs = (nb + 2 * kQT - 1) / (2 * kQT);
        level = __reduce_max_sync(0xffffffffu, pairs) - 1;
      }
      at_level = __ballot_sync(0xffffffffu, pairs > level && level >= 0);
      width = (long long)__popc(at_level) * p.Hq;
    }
    int4 x = make_int4(-1, 0, 0, 0);
    if (more) {
      const int y = (int)(it - first), k = y / p.Hq;
      uint32_t left = at_level;
      for (int u = 0; u < k; ++u) left &= left - 1;
      const int l = __ffs(left) - 1;
      x.x = b0 + l;
      x.y = y - k * p.Hq;
      x.z = __shfl_sync(0xffffffffu, nb, l);
      x.w = (x.z + kQT - 1) / kQT - 1 - 2 * (__shfl_sync(0xffffffffu, pairs, l) - 1 - level);
    }
    const uint32_t slot = r % kItems;
    if (r >= kItems && !wait(&ring.empty[slot], r / kItems - 1)) return false;
    if (lane == 0) {
      ring.item[slot] = x;
      mbar_arrive(&ring.full[slot]);
    }
    __syncwarp();
    if (!more) return true;
  }
}

struct Small {
  uint64_t qfull[2], qempty[2];   // group g's Q: landed; its last S of the item complete
  uint64_t full[2], empty[2];     // K and V pairs: landed; released by the groups (one arrival each)
  uint64_t sfull[2];   // group g: its next S, and every MMA issued before it, complete
  uint64_t pfull[2][2];   // group g: the first and the second half of its P written by the group's four warps
  uint64_t odone[2];   // group g: its last P V of the item complete
  uint64_t drain;
  Ring ring;           // the items to come
  uint32_t tmem_base;
  int abort;
};
constexpr int kWinSmem = kOffSmall + (int)sizeof(Small) + 1024;
static_assert(kWinSmem <= 232448, "shared memory exceeds the per-CTA limit");

// One lane of a converged warp.
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

// One row against its 128 columns of S: moves the reference, turns S into P in
// place (P is rounded to bf16, which the product with V takes and which holds
// 2^24 above the reference as well as any value below; its sum, in fp32, is of
// the unrounded values).  Columns [from, to) and [0, first) are seen.  follow(factor) lets O
// follow the reference (l does here); SPLIT: before half(), which is called
// when the first half of P is stored, else at the end, when x is dead.  The masked path is
// kept short: this code runs four warps wide from a small instruction cache,
// and a cold branch of a few hundred instructions costs more than the
// exponentials.
template <bool SPLIT, typename Follow, typename Half>
__device__ __forceinline__ void softmax_tile(const WindowCall& p, uint32_t tS, bool mask, int from, int to, int first,
                                             float& ref, float& l, Follow follow, Half half) {
  const float scale = p.scale_log2;
  float x[kQT];
#pragma unroll
  for (int c = 0; c < 8; ++c) tmem_ld16(tS + 16 * c, x + 16 * c);
  tmem_wait_ld();
  if (mask) {
    auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };   // bits [0, n)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t seen = (below(to - 32 * c) & ~below(from - 32 * c)) | below(first - 32 * c);
      if (__all_sync(0xffffffffu, seen == ~0u)) continue;
#pragma unroll
      for (int u = 0; u < 32; ++u)
        if (!(seen & (1u << u))) x[32 * c + u] = -INFINITY;
    }
  }
  float m8[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) m8[u] = x[u];
#pragma unroll
  for (int u = 8; u < kQT; ++u) m8[u & 7] = fmaxf(m8[u & 7], x[u]);
  const float mt = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                         fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7]))) * scale;
  const bool need = mt > ref + kMove;
  float factor = 1.f;
  if (need) {
    factor = ref == -INFINITY ? 0.f : ex2_approx(ref - mt);
    ref = mt;
    l *= factor;
  }
  if (SPLIT && __any_sync(0xffffffffu, need)) follow(factor);
  // a row that has seen nothing yet keeps P = 0
  const float r0 = ref == -INFINITY ? 0.f : ref;
  // P = 2^(x scale - ref), 16 columns at a time: while the exponentials of
  // one block run, the block before is summed, packed and stored
  const uint64_t sc2 = f2_pack(scale, scale), nr2 = f2_pack(-r0, -r0);
  uint64_t ls2[4] = {0ull, 0ull, 0ull, 0ull};
  float hw[16];
#pragma unroll
  for (int c = 0; c <= 8; ++c) {
    if (c < 8) {
#pragma unroll
      for (int u = 16 * c; u < 16 * c + 16; u += 2) {
        const uint64_t y = f2_fma(f2_pack(x[u], x[u + 1]), sc2, nr2);
        x[u] = ex2_approx(f2_lo(y));
        x[u + 1] = ex2_approx(f2_hi(y));
      }
    }
    if (c > 0) {
#pragma unroll
      for (int u = 16 * c - 16; u < 16 * c; u += 2) {
        ls2[(u >> 1) & 3] = f2_add(ls2[(u >> 1) & 3], f2_pack(x[u], x[u + 1]));
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(x[u], x[u + 1]);
        hw[(u >> 1) & 15] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&h2));
      }
      if (c % 2 == 0) tmem_st16(tS + 16 * (c / 2 - 1), hw);
      if (SPLIT && c == 5) half();
    }
  }
  const uint64_t lsum = f2_add(f2_add(ls2[0], ls2[1]), f2_add(ls2[2], ls2[3]));
  l += f2_lo(lsum) + f2_hi(lsum);
  if (!SPLIT && __any_sync(0xffffffffu, need)) follow(factor);
}

// A value all lanes of the converged warp hold, where the compiler knows that
// they do: in a uniform register.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

template <bool SPLIT, int DS>
__device__ __forceinline__ void softmax_group(const WindowCall& p, Small& S, uint8_t* sm, uint32_t tmem, int warp,
                                              int lane) {
  const int g = warp >> 2, quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
  const uint32_t tS = tmem + lane_base + 128 * g, tO = tmem + lane_base + 256 + 128 * g;
  const bool speaks = quarter == 0 && lane == 0;
  uint32_t pair0 = 0, seen = 0, done = 0;         // entries, the group's tiles and items so far
  // A wait this warp gave up on raises the timeout flag and the CTA's abort
  // flag, which ends every other wait of the CTA; the warp stops.
  auto give_up = [&]() {
    if (lane == 0) {
      S.abort = 1;
      atomicOr(p.status, DROPKV_FLAG_TIMEOUT);
    }
  };
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, &S.abort));
  };
  // The pair of the item's entry j (with V of the entry before) is needed no
  // more by this group.
  auto release = [&](int j) {
    if (speaks) mbar_arrive(&S.empty[(pair0 + j) & 1]);
    __syncwarp();
  };
  // The same for an entry this group does not take: only once it has landed,
  // so that the release counts for it and not for the pair before in its slot.
  // The warp that releases is the only one to wait: once it has, the slot's
  // next pair may land, and a warp that came to look only then would find the
  // barrier one phase on, at the parity of the phase before, and wait for a
  // pair that cannot come until its own P has.
  auto pass = [&](int j) {
    if (quarter != 0) return true;
    if (!wait(&S.full[(pair0 + j) & 1], (pair0 + j) >> 1)) return false;
    release(j);
    return true;
  };
  for (uint32_t k = 0;; ++k) {
    if (!wait(&S.ring.full[k % kItems], k / kItems)) { give_up(); return; }
    // The item stays in the ring until its output is written: what only that
    // needs is read again there.  In uniform registers its list leaves the
    // tile loop more of the others (32768 tokens, window 4096: 1.44 -> 1.34
    // ms); with both numbers so, the short form without SPLIT spills (50 -> 55 us).
    const int4 item = S.ring.item[k % kItems];
    if (item.x < 0) return;
    const int nb = SPLIT ? uniform(item.z) : item.z, t1 = uniform(item.w);
    const List list = make_list(p, t1 - 1, t1);
    auto leave_item = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.ring.empty[k % kItems]);
      __syncwarp();
    };
    const int n = list.n, tg = list.t[g], pos = tg * kQT + row;
    if (tg < 0) {
      for (int j = 0; j < n; ++j)
        if (!pass(j)) { give_up(); return; }
      pair0 += n;
      leave_item();
      continue;
    }
    float ref = -INFINITY, l = 0.f;
    bool first = true;
    for (int i = 0; i < n; ++i) {
      if (!list.takes(g, i)) continue;
      const int kt = list.tile(i), j0 = kt * kQT;
      if (!wait(&S.sfull[g], seen)) { give_up(); return; }
      tc_fence_after();
      if (g == 1 && list.skip >= 0 && i == list.skip + 1) release(list.skip);
      release(i);                                 // S is complete, and the P V issued before it
      if (speaks && kt == tg) mbar_arrive(&S.qempty[g]);
      // the last row of the tile reaches back to tg 128 + 127 - W + 1
      const bool edge = p.window > 0 && j0 <= tg * kQT + 127 - p.window && j0 + kQT > p.sinks;
      // the sequence's last key tile (group 1's alone): rows past the end may
      // hold anything; zero them so that 0 * NaN never reaches O
      auto zero_tail = [&]() {
        if (j0 + kQT <= nb) return true;
        const uint32_t pr = pair0 + i + 1;
        if (!wait(&S.full[pr & 1], pr >> 1)) return false;
        if (j0 + row >= nb) {
          uint8_t* vrow = sm + kOffV + (pr & 1) * kTileB + row * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            *reinterpret_cast<uint4*>(vrow + c * 16) = make_uint4(0, 0, 0, 0);
            if (DS > 4) *reinterpret_cast<uint4*>(vrow + kHalfB + c * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        return true;
      };
      if (SPLIT && !zero_tail()) { give_up(); return; }
      auto written = [&](int h) {                 // half h of P, and all before it
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.pfull[g][h]);
      };
      // keys j <= pos with j > pos - window or j < sinks; past a narrow tile's
      // kNarrow columns S holds anything
      softmax_tile<SPLIT>(
          p, tS, kt == tg || edge || i == list.narrow, p.window > 0 ? pos - p.window + 1 - j0 : 0, pos + 1 - j0,
          p.window > 0 ? min(p.sinks, pos + 1) - j0 : 0, ref, l,
          [&](float factor) {
            // the group's P V of its tile before is complete (the commit its S
            // signalled came after it): O follows the reference
            if (first) return;
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
      first = false;
      if (!SPLIT && !zero_tail()) { give_up(); return; }
      written(1);
      ++seen;
    }
    if (!wait(&S.odone[g], done)) { give_up(); return; }
    ++done;
    tc_fence_after();
    // group 0 does not take the last entry, but its last V came with it
    if (g == 0 && !pass(n - 1)) { give_up(); return; }
    pair0 += n;
    const float inv_l = 1.0f / l;                 // a row sees itself at least
    const int4 x = S.ring.item[k % kItems];
    __nv_bfloat16* orow = p.out + (((size_t)x.x * p.Hq + x.y) * p.n_max + pos) * p.d;
    leave_item();
#pragma unroll 1
    for (int c0 = 0; c0 < p.d; c0 += 32) {
      float o[32];
      __syncwarp();                               // rows past the end stored nothing
      tmem_ld16(tO + c0, o);
      tmem_ld16(tO + c0 + 16, o + 16);
      tmem_wait_ld();
      if (pos < nb) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w4[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(o[8 * q + 2 * u] * inv_l, o[8 * q + 2 * u + 1] * inv_l);
            w4[u] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          if (c0 + 8 * q < p.d)
            *reinterpret_cast<uint4*>(orow + c0 + 8 * q) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
      }
    }
  }
}

#ifdef DROPKV_TEST_HOOKS
__device__ int g_test_skip_pair[2] = {-1, -1};    // CTA and pair that the test build leaves out
#endif

// SPLIT: P V of a tile begins on the first half of P while the softmax is at
// the second.  With many tiles per item it shortens the chain softmax -> P V ->
// S that bounds the kernel (32768 tokens, window 4096: 1.45 -> 1.36 ms when it
// came); with few, most of them masked, the extra barrier costs more (now:
// 2051 tokens, window 333 50 -> 55 us; 8192 tokens, window 1024 137 -> 141).
//
// DS: steps of 16 channels, 4, 6 or 8.  A head of up to 64 channels takes one
// block of 64 columns of Q, K and V, and N = 64 in P V; up to 96 takes six
// steps for S (P V stays at N = 128: V's columns come in swizzled blocks of
// 64).  Against eight steps for all: d 64, 8192 tokens, window 2048 197 -> 179
// us, d 96 202 -> 196; a ragged batch of short prompts 54.7 -> 48.8 and 58.1
// -> 56.8.
template <bool SPLIT, int DS>
__global__ void __launch_bounds__(kWinThreads, 1)
    window_prefill_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                          const __grid_constant__ CUtensorMap tmv, const WindowCall p) {
  constexpr int kLoadB = DS <= 4 ? kHalfB : kTileB;   // bytes of a tile that are loaded
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Small& S = *reinterpret_cast<Small*>(sm + kOffSmall);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.qfull[i], 1); mbar_init(&S.qempty[i], 1);
      mbar_init(&S.full[i], 1); mbar_init(&S.empty[i], 2);
      mbar_init(&S.sfull[i], 1); mbar_init(&S.pfull[i][0], 4); mbar_init(&S.pfull[i][1], 4);
      mbar_init(&S.odone[i], 1);
    }
    mbar_init(&S.drain, 1);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&S.ring.full[i], 1);
      mbar_init(&S.ring.empty[i], kTakers);
    }
    S.abort = 0;
    fence_mbar_init();
  }
  if (warp == kIssuer) tmem_alloc(&S.tmem_base, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0)                            // lengths that cannot be served are left out
    for (int b = tid; b < p.B; b += kWinThreads)
      if (p.lengths && (p.lengths[b] < 0 || p.lengths[b] > p.n_max)) atomicOr(p.status, DROPKV_FLAG_BAD_LENGTH);

  if (warp == kProducer) {
    if (lane == 0) {
      uint32_t pair = 0, used[2] = {0, 0};        // pairs issued, items of group g
      int v_tile = -1, v_unit = 0;                // the entry before: its V comes with this one's K
      auto put = [&](int k_tile, int k_unit) {    // k_tile -1: the last V alone
        const uint32_t slot = pair & 1;
        if (pair >= 2 && !mbar_wait(&S.empty[slot], ((pair >> 1) + 1) & 1, &S.abort)) return false;
        bool load = true;
#ifdef DROPKV_TEST_HOOKS
        load = (int)blockIdx.x != g_test_skip_pair[0] || (int)pair != g_test_skip_pair[1];
#endif
        if (load) mbar_arrive_expect_tx(&S.full[slot], (k_tile >= 0 ? kLoadB : 0) + (v_tile >= 0 ? kLoadB : 0));
        if (load && v_tile >= 0) {                // needed first
          uint8_t* dst = sm + kOffV + slot * kTileB;
          tma_load_3d(dst, &tmv, &S.full[slot], 0, v_tile * kQT, v_unit);
          if (DS > 4) tma_load_3d(dst + kHalfB, &tmv, &S.full[slot], 64, v_tile * kQT, v_unit);
        }
        if (load && k_tile >= 0) {
          uint8_t* dst = sm + kOffK + slot * kTileB;
          tma_load_3d(dst, &tmk, &S.full[slot], 0, k_tile * kQT, k_unit);
          if (DS > 4) tma_load_3d(dst + kHalfB, &tmk, &S.full[slot], 64, k_tile * kQT, k_unit);
        }
        v_tile = k_tile;
        v_unit = k_unit;
        ++pair;
        return true;
      };
      bool ok = true;
      Item w;
      for (uint32_t k = 0; ok; ++k) {
        const Got got = take_item(
            p, S.ring, k, &w, [&](uint64_t* bar, uint32_t phase) { return mbar_wait(bar, phase & 1, &S.abort); },
            [](uint64_t* bar) { mbar_arrive(bar); });
        if (got != kItem) {
          ok = got == kEnd;
          break;
        }
        const List& list = w.list;
        const int zq = w.b * p.Hq + w.hq, unit = w.b * p.Hkv + w.hq / p.g;
        if (!(ok = put(list.tile(0), unit))) break;   // with the last item's last V: before the waits for Q
        for (int g = 0; ok && g < 2; ++g) {
          if (list.t[g] < 0) continue;
          if (used[g] > 0 && !(ok = mbar_wait(&S.qempty[g], (used[g] - 1) & 1, &S.abort))) break;
          mbar_arrive_expect_tx(&S.qfull[g], kLoadB);
          tma_load_3d(sm + kOffQ + g * kTileB, &tmq, &S.qfull[g], 0, list.t[g] * kQT, zq);
          if (DS > 4) tma_load_3d(sm + kOffQ + g * kTileB + kHalfB, &tmq, &S.qfull[g], 64, list.t[g] * kQT, zq);
          ++used[g];
        }
        for (int j = 1; ok && j < list.n; ++j) ok = put(list.tile(j), unit);
      }
      if (ok && v_tile >= 0) ok = put(-1, 0);
      if (!ok) {
        S.abort = 1;
        atomicOr(p.status, DROPKV_FLAG_TIMEOUT);
      }
      // every copy has landed before the CTA can leave
      for (uint32_t j = pair > 2 ? pair - 2 : 0; j < pair; ++j) drain_wait(&S.full[j & 1], (j >> 1) & 1);
      for (int g = 0; g < 2; ++g)
        if (used[g] > 0) drain_wait(&S.qfull[g], (used[g] - 1) & 1);
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    // The whole warp walks the list, one elected lane issues: descriptors and
    // tensor-memory addresses then stay in uniform registers, where the MMA
    // instruction takes them from.  (All 512 columns are the CTA's: they
    // start at 0.)
    const bool leader = elect_one();
    const uint64_t qd = desc_kmajor_sw128(smem_addr(sm + kOffQ), kQT, 0);
    const uint64_t kd = desc_kmajor_sw128(smem_addr(sm + kOffK), kQT, 0);
    const uint64_t vd = desc_mnmajor_sw128(smem_addr(sm + kOffV), kQT, 0);
    constexpr uint32_t idO = umma_idesc_bf16(128, DS <= 4 ? 64 : 128, 0, 1);
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, &S.abort)) != 0;
    };
    // S of group g from the K tile in slot `slot`
    auto issue_S = [&](int g, int slot, uint32_t id) {
      const uint64_t qg = qd + ((g * kTileB) >> 4), kg = kd + ((slot * kTileB) >> 4);
      if (leader) {
#pragma unroll
        for (int s = 0; s < DS; ++s) {
          const uint64_t at = ((s >> 2) * kHalfB + (s & 3) * 32) >> 4;   // as desc_kmajor_sw128 steps
          umma_bf16(128 * g, qg + at, kg + at, id, s > 0);
        }
        umma_commit(&S.sfull[g]);
      }
      __syncwarp();
    };
    // P V of group g, steps s0 .. s1 - 1 of 16 keys
    auto issue_PV = [&](int g, int slot, auto s0, auto s1, bool first) {
      const uint64_t vg = vd + ((slot * kTileB) >> 4);
      if (leader) {
#pragma unroll
        for (int s = decltype(s0)::value; s < decltype(s1)::value; ++s)
          umma_bf16_tmem_a(256 + 128 * g, 128 * g + 8 * s, vg + ((s * 16 * 128) >> 4), idO, !first || s > 0);
      }
      __syncwarp();
    };
    using Zero = std::integral_constant<int, 0>;
    using Four = std::integral_constant<int, 4>;
    using Eight = std::integral_constant<int, 8>;
    using Narrow = std::integral_constant<int, kNarrow / 16>;
    uint32_t pair0 = 0, seen0 = 0, seen1 = 0, used0 = 0, used1 = 0;   // entries, tiles and items of the groups so far
    Item w, w2;                                   // the item, the one after
    uint32_t taken = 0;
    auto take = [&](Item* to) {
      return take_item(p, S.ring, taken++, to, wait, [&](uint64_t* bar) {
        __syncwarp();
        if (leader) mbar_arrive(bar);
        __syncwarp();
      });
    };
    Got got = take(&w);
    bool have = got == kItem, ok = got != kGaveUp;
    // the first S of group g in an item that begins with pair pr
    auto first_S = [&](int g, const Item& x, uint32_t pr) {
      if (!wait(&S.qfull[g], g ? used1++ : used0++)) return false;
      tc_fence_after();
      if (x.list.narrow == 0) issue_S(g, pr & 1, umma_idesc_bf16(128, kNarrow, 0, 0));
      else issue_S(g, pr & 1, umma_idesc_bf16(128, 128, 0, 0));
      return true;
    };
    if (have) {
      ok = wait(&S.full[0], 0);
      if (ok && w.list.takes(0, 0)) ok = first_S(0, w, 0);
      if (ok && w.list.takes(1, 0)) ok = first_S(1, w, 0);
    }
    while (ok && have) {
      got = take(&w2);
      if (!(ok = got != kGaveUp)) break;
      const bool more = got == kItem;
      const List& list = w.list;
      bool first0 = true, first1 = true;
      // Entry i: P V of it and S of the entry after it, group 0, then group 1.
      // plain: neither is narrow, skipped or the item's last.
      auto entry = [&](int i, auto plain) {
        constexpr bool kPlain = decltype(plain)::value;
        const uint32_t pr = pair0 + i + 1;        // V(i), K of the entry after it
        if (!wait(&S.full[pr & 1], pr >> 1)) return false;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t& seen = g ? seen1 : seen0;
          bool& first = g ? first1 : first0;
          if (kPlain || list.takes(g, i)) {
            if (SPLIT) {
              if (!wait(&S.pfull[g][0], seen)) return false;
              tc_fence_after();
              if (!kPlain && i == list.narrow) issue_PV(g, pr & 1, Zero{}, Narrow{}, first);
              else issue_PV(g, pr & 1, Zero{}, Four{}, !kPlain && first);
              if (!wait(&S.pfull[g][1], seen)) return false;
              tc_fence_after();
              if (kPlain || i != list.narrow) issue_PV(g, pr & 1, Four{}, Eight{}, false);
            } else {
              if (!wait(&S.pfull[g][1], seen)) return false;
              tc_fence_after();
              if (!kPlain && i == list.narrow) issue_PV(g, pr & 1, Zero{}, Narrow{}, first);
              else issue_PV(g, pr & 1, Zero{}, Eight{}, !kPlain && first);
            }
            first = false;
            ++seen;
            if (!kPlain && list.tile(i) == list.t[g] && leader) umma_commit(&S.odone[g]);
          }
          // the group's next S, over P, which P V issued before it has read
          if (kPlain) {
            issue_S(g, pr & 1, umma_idesc_bf16(128, 128, 0, 0));
          } else if (i + 1 < list.n) {
            if (list.takes(g, i + 1)) {
              // (a group that passes over entry 0 meets its Q here)
              if (g == 1 && list.skip == 0 && i == 0 && !wait(&S.qfull[1], used1++)) return false;
              if (i + 1 == list.narrow) issue_S(g, pr & 1, umma_idesc_bf16(128, kNarrow, 0, 0));
              else issue_S(g, pr & 1, umma_idesc_bf16(128, 128, 0, 0));
            }
          } else if (more && w2.list.takes(g, 0)) {
            if (!first_S(g, w2, pr)) return false;
          }
        }
        return true;
      };
      int i = 0;
      for (; ok && i < min(list.ns + 2, list.n); ++i) ok = entry(i, std::false_type{});
      for (; ok && i < list.n - 2; ++i) ok = entry(i, std::true_type{});
      for (; ok && i < list.n; ++i) ok = entry(i, std::false_type{});
      pair0 += list.n;
      w = w2;
      have = more;
    }
    if (!ok && leader) {
      S.abort = 1;
      atomicOr(p.status, DROPKV_FLAG_TIMEOUT);
    }
    // no MMA may still be writing TMEM when it is released
    if (leader) {
      umma_commit(&S.drain);
      drain_wait(&S.drain, 0);
    }
    __syncwarp();
  } else if (warp == kWalker) {
    // A slot comes free when the item in it is done, and an item of many
    // million keys takes longer than a wait's limit: the other roles' waits
    // tell whether the CTA moves, and their abort ends this one.
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      for (int t = 0; t < kWalkerWaits; ++t) {
        if (__all_sync(0xffffffffu, mbar_wait(bar, phase & 1, &S.abort))) return true;
        if (__any_sync(0xffffffffu, *static_cast<volatile int*>(&S.abort) != 0)) return false;
      }
      return false;
    };
    if (!walk_items(p, S.ring, lane, wait) && lane == 0) {
      S.abort = 1;
      atomicOr(p.status, DROPKV_FLAG_TIMEOUT);
    }
    __syncwarp();
  } else if (warp < 8) {
    softmax_group<SPLIT, DS>(p, S, sm, tmem, warp, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

}  // namespace

namespace {
template <bool SPLIT, int DS>
cudaError_t launch(const WindowCall& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, int sms,
                   cudaStream_t st) {
  const cudaError_t e = allow_smem<window_prefill_kernel<SPLIT, DS>>(kWinSmem);
  if (e != cudaSuccess) return e;
  const long long most = (long long)((p.n_max + 2 * kQT - 1) / (2 * kQT)) * p.Hq * p.B;
  const dim3 grid((unsigned)std::min<long long>(most, sms));
  return launch_pdl(window_prefill_kernel<SPLIT, DS>, grid, dim3(kWinThreads), kWinSmem, st, tq, tk, tv, p);
}
}  // namespace

cudaError_t launch_window(const WindowCall& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          int sms, cudaStream_t st) {
  const bool split = p.window == 0 || p.window >= kSplitWindow;
  auto pick = [&](auto wide) {
    constexpr int DS = decltype(wide)::value;
    return split ? launch<true, DS>(p, tq, tk, tv, sms, st) : launch<false, DS>(p, tq, tk, tv, sms, st);
  };
  if (p.d <= 64) return pick(std::integral_constant<int, 4>{});
  if (p.d <= 96) return pick(std::integral_constant<int, 6>{});
  return pick(std::integral_constant<int, 8>{});
}

}  // namespace kvcache

#ifdef DROPKV_TEST_HOOKS
#include "../../include/kvcache_test_hooks.h"
extern "C" dropkv_status kvcache_test_skip_window_pair(int32_t cta, int32_t pair) {
  const int v[2] = {cta, pair};
  return cudaMemcpyToSymbol(kvcache::g_test_skip_pair, v, sizeof v) == cudaSuccess ? DROPKV_OK : DROPKV_ERR_CUDA;
}
#endif
