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
constexpr int kProducer = 8, kIssuer = 9, kWinThreads = 32 * 12;   // warps 10, 11 idle (register shares)
constexpr int kOffQ = 0, kOffK = 2 * kTileB, kOffV = 4 * kTileB, kOffSmall = 6 * kTileB;
constexpr uint32_t kCols = 512;                   // group g: S / P at [128 g, +128), O at [256 + 128 g, +128)
constexpr float kMove = 24.0f;                    // base-2 logarithm by which a maximum may pass its reference
constexpr uint64_t kDrain = 20000000ull;          // 20 ms to drain copies after an abort

constexpr int kNarrow = 32;
constexpr int kSplitWindow = 1536;                // windows from which on P goes in halves (even at 1024)

struct Small {
  uint64_t qfull[2], qempty[2];   // group g's Q: landed; its last S of the item complete
  uint64_t full[2], empty[2];     // K and V pairs: landed; released by the groups (one arrival each)
  uint64_t sfull[2];   // group g: its next S, and every MMA issued before it, complete
  uint64_t pfull[2][2];   // group g: the first and the second half of its P written by the group's four warps
  uint64_t odone[2];   // group g: its last P V of the item complete
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
constexpr int kWinSmem = kOffSmall + (int)sizeof(Small) + 1024;
static_assert(kWinSmem <= 232448, "shared memory exceeds the per-CTA limit");

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

// The items of the call in order: sequence by sequence, pairs of query tiles
// from the sequence's end (the last tile is group 1's), heads innermost.  A
// CTA takes every gridDim.x-th; each role walks the same cursor.
struct Cursor {
  int b = -1, pairs = 0;                          // sequence, its pairs of query tiles
  int nb = 0;
  long long first = 0;                            // items before it
};
__device__ __forceinline__ int length_of(const WindowCall& p, int b) {
  const int nb = p.lengths ? p.lengths[b] : p.n_max;
  return nb < 0 || nb > p.n_max ? 0 : nb;
}
struct Item {
  int b, hq, nb;
  List list;
};
// Item `it`, if there is one.
__device__ __forceinline__ bool item_at(const WindowCall& p, Cursor& c, long long it, Item* w) {
  while (c.b < 0 || it >= c.first + (long long)c.pairs * p.Hq) {
    c.first += (long long)c.pairs * p.Hq;
    if (++c.b >= p.B) return false;
    c.nb = length_of(p, c.b);
    c.pairs = (c.nb + 2 * kQT - 1) / (2 * kQT);
  }
  const int y = (int)(it - c.first), x = y / p.Hq;
  w->b = c.b;
  w->nb = c.nb;
  w->hq = y - x * p.Hq;
  const int t1 = (c.nb + kQT - 1) / kQT - 1 - 2 * x;
  w->list = make_list(p, t1 - 1, t1);
  return true;
}

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
// place.  Columns [from, to) and [0, first) are seen.  follow(factor) lets O
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
  Cursor at;
  Item w;
  for (long long it = blockIdx.x; item_at(p, at, it, &w); it += gridDim.x) {
    const List& list = w.list;
    const int n = list.n, tg = list.t[g], pos = tg * kQT + row;
    if (tg < 0) {
      for (int j = 0; j < n; ++j)
        if (!pass(j)) { give_up(); return; }
      pair0 += n;
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
        if (j0 + kQT <= w.nb) return true;
        const uint32_t pr = pair0 + i + 1;
        if (!wait(&S.full[pr & 1], pr >> 1)) return false;
        if (j0 + row >= w.nb) {
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
    __nv_bfloat16* orow = p.out + (((size_t)w.b * p.Hq + w.hq) * p.n_max + pos) * p.d;
#pragma unroll 1
    for (int c0 = 0; c0 < p.d; c0 += 32) {
      float o[32];
      __syncwarp();                               // rows past the end stored nothing
      tmem_ld16(tO + c0, o);
      tmem_ld16(tO + c0 + 16, o + 16);
      tmem_wait_ld();
      if (pos < w.nb) {
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

// SPLIT: P V of a tile begins on the first half of P while the softmax is at
// the second.  With many tiles per item it shortens the chain softmax -> P V ->
// S that bounds the kernel (32768 tokens, window 4096: 1.45 -> 1.36 ms); with
// few, most of them masked, the extra barrier costs more (2051 tokens, window
// 333: 60 -> 65 us).
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
        mbar_arrive_expect_tx(&S.full[slot], (k_tile >= 0 ? kLoadB : 0) + (v_tile >= 0 ? kLoadB : 0));
        if (v_tile >= 0) {                        // needed first
          uint8_t* dst = sm + kOffV + slot * kTileB;
          tma_load_3d(dst, &tmv, &S.full[slot], 0, v_tile * kQT, v_unit);
          if (DS > 4) tma_load_3d(dst + kHalfB, &tmv, &S.full[slot], 64, v_tile * kQT, v_unit);
        }
        if (k_tile >= 0) {
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
      Cursor at;
      Item w;
      for (long long it = blockIdx.x; ok && item_at(p, at, it, &w); it += gridDim.x) {
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
    Cursor at;
    Item w, w2;                                   // the item, the one after
    long long it = blockIdx.x;
    bool have = item_at(p, at, it, &w), ok = true;
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
      it += gridDim.x;
      const bool more = item_at(p, at, it, &w2);
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
