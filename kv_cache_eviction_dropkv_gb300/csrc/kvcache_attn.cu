// Attention of a few query rows per sequence over the paged 8-bit cache.
//
//   x_rj = q_r . (ck_j s_k(page of j)) / sqrt(d),  o_r = sum_j p_rj cv_j s_v / sum_j p_rj,
//   p_rj = exp(x_rj - m_r) over the tokens row r sees.
//
// The call reads each visible code once and computes 4 R operations per code
// pair for the R = g T query rows of a KV head: it is bound by memory, and
// the kernel's work is to keep copies in flight and to turn bytes into fp16
// operands cheaply.
//
// Work is cut into tiles of 32 tokens of one KV head (a tile lies inside a
// page, so it has one K and one V scale).  The tiles of the whole call,
// counted on the device from the lengths and the window, are dealt out to the
// warps of one resident wave in equal contiguous runs, so ragged batches
// leave no tail.  A warp holds 8 or 16 of a KV head's rows; more are dealt as
// row groups: the warps of one run, one per group, stand side by side and read
// the same tiles at about the same time, so the cache is read from memory
// once.  A warp is on its own: it copies its tiles with cp.async into its own
// ring of kStages tiles and keeps its rows' softmax state and outputs in
// registers; no barrier of the block stands in its loop.  A run that holds a
// whole unit (sequence, head, row group) writes the output; the pieces of one
// that is cut by run borders go to the workspace and a second kernel joins
// them in run order (no atomics: results do not depend on timing).  Where the
// table or the window bounds the units tightly, the host skips the deal
// (make_attn_plan has the rules and times): few units go to a CTA or a cluster
// each, whose warps take the tiles in turn and join through shared memory
// behind one barrier (up to two waves of CTAs), and many short ones to a warp
// each, with nothing to join (up to four waves).
//
// Per tile, on mma.m16n8k16 with the tokens on the M side, so that 8 query
// rows fill the N side (a decode step has g = 1 to 8 rows per KV head; the
// 128-row tcgen05 tile would be 94 % padding and wants its operands as 16-bit
// tiles in shared memory, which is four times the traffic of these bytes):
//   S^T[32 tokens x 8 rows] = K . Q^T,  then O^T[d x 8 rows] += V^T . P.
// The index of a contraction may be permuted freely if both operands agree:
// a lane takes 16 contiguous bytes of a K row as its k elements of four MMAs
// (one 128-bit shared load), and 16 contiguous channels of a V row as its row
// indices of eight MMAs.  P goes from S^T's accumulator layout to the B
// operand with one movmatrix per 8 x 8 block.  Rows of 128 bytes are staged
// with their 16-byte chunks XOR-ed by the token's low bits: both kinds of
// read then touch all banks.
#include <algorithm>
#include <cmath>

#include "kvcache_internal.cuh"
#include "sm103_ptx.cuh"

namespace kvcache {
namespace {

using dropkv::ex2_approx;
using dropkv::f2_add;
using dropkv::f2_fma;
using dropkv::f2_hi;
using dropkv::f2_lo;
using dropkv::f2_mul;
using dropkv::f2_pack;
using dropkv::grid_dep_launch;
using dropkv::grid_dep_wait;
using dropkv::launch_pdl;

constexpr int kTok = 32;                    // tokens of a tile
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStages = 2;
constexpr int kPitch = 128;                 // bytes of a staged row
constexpr int kStageBytes = 2 * kTok * kPitch;   // K rows, then V rows
constexpr int kMeta = 64;                   // tile descriptions a warp holds (two batches of 32)
struct alignas(16) Tile {
  long long at;                             // byte offset of its first row in the layer's K or V
  int tok;                                  // first token
  int len;                                  // tokens of its sequence
  int unit;                                 // entry * Hkv + head
  float ks, lv;                             // K scale, log2 of the V scale
  int how;                                  // kPartial, kMasked, kUnreadable
};
constexpr int kPartial = 1;                 // some of its slots are seen by no row
constexpr int kMasked = 2;                  // some row does not see some of its tokens
constexpr int kUnreadable = 4;              // its table entry is no page
// CTAs per SM: registers allow three where a row has at most 64 channels (with
// three instead of two, e4m3 and int8: 1 x 131072 tokens, 8 heads, 37.0 -> 34.9
// and 40.8 -> 35.3 us; 24 x up to 4000, 32 heads, one row 47.1 -> 39.8 and 52.9
// -> 40.6; 48 x 3-8191, window 2000, 47.7 -> 42.5; 46 x 1347-3921 with 35 rows
// 264 -> 239), two above (three: 51.9 -> 55.2 us).
__host__ __device__ constexpr int kCtas(int d) { return d <= 64 ? 3 : 2; }
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr int kSmem = kRingBytes + kWarps * kMeta * (int)sizeof(Tile);
constexpr int kJoinThreads = 128, kJoinWide = 512;   // 4 rows; 1 row
constexpr int kTeamTiles = 8;               // most tiles a warp takes of a unit that has a team
constexpr int kSoloTiles = 12;              // most tiles of a unit that one warp takes alone
constexpr int kUnitCost = 3;                // tiles that taking up a unit is worth
// A row's reference moves only when a tile's maximum is this far above it
// (base-2 logarithm), so probabilities stay below 2^8 (fp16 holds 2^16).
constexpr float kMoveLog2 = 8.0f;
// Probabilities enter P V as fp16 times 2^7: up to 2^15 of fp16's 2^16 above,
// so that those far below the reference are not dropped from the output while
// the sum counts them (2^-25 of the reference is fp16's last bit: a million
// such tokens behind one dominant key are 1/32 of the output).  What is lost
// is at most 2^-32 of the reference for each; outputs are multiplied by 2^-7
// as they are written, apart from the factor of the sum, which may be tiny.
constexpr float kLiftLog2 = 7.0f, kUnlift = 0x1p-7f;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same from a zero accumulator.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Rank in the cluster; barrier of all its threads (shared memory written
// before is visible after); 16 bytes at this CTA's address `addr` in CTA `rank`.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, uint32_t rank) {
  float4 v;
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 16 bytes into shared memory, zeros when !take.
__device__ __forceinline__ void cp16(uint32_t dst, const uint8_t* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_cg(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const uint8_t* src, bool take) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(take ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// What a sequence's length, T and the window leave to read: tiles [0, ns) and
// [s2, s2 + rest).
struct Span {
  int ns, s2, tiles;
  int lo;                                   // first token some row's window reaches
};
__device__ __forceinline__ Span span_of(int len, int T, int window, int sinks) {
  Span s;
  const int end = (len + kTok - 1) / kTok;
  s.lo = window > 0 ? max(0, max(0, len - T) - window + 1) : 0;
  s.ns = window > 0 ? (min(sinks, s.lo) + kTok - 1) / kTok : 0;
  s.s2 = max(s.lo / kTok, s.ns);
  s.tiles = s.ns + end - s.s2;
  if (len <= 0) s.ns = s.s2 = s.tiles = 0;
  return s;
}

// Length of entry i's sequence; 0 (and a flag, once) when it cannot be served.
__device__ __forceinline__ int entry_len(const AttnCall& p, int i, bool report) {
  const int s = p.seqs ? p.seqs[i] : i;
  if (s < 0 || s >= p.c.S) {
    if (report) flag(p.c.status, KVCACHE_FLAG_BAD_SEQ);
    return 0;
  }
  const int len = p.c.length[s], held = p.c.count[s];
  if (len < 0 || held < 0 || held > p.c.M || (long long)len > ((long long)held << p.c.page_log2)) {
    if (report) flag(p.c.status, DROPKV_FLAG_BAD_LENGTH);
    return 0;
  }
  return len;
}

// The tiles of the call lie in a row: sequence by sequence, unit by unit.  For
// the deal each unit is kUnitCost tiles longer than it is (its query rows are
// loaded and its output written), and the runs are equal parts of that.
struct Deal {
  uint32_t share, more;                     // the first `more` runs have share + 1, the others share
};
__device__ __forceinline__ uint32_t cost_of(int tiles) { return tiles > 0 ? tiles + kUnitCost : 0; }
__device__ __forceinline__ int entry_tiles(const AttnCall& p, int b) {
  return span_of(entry_len(p, b, false), p.T, p.window, p.sinks).tiles;
}
// Cost per head of all entries, over the warp's lanes (mine: the tiles of
// entry `lane`, which every scan starts with).
__device__ __forceinline__ uint32_t sum_cost(const AttnCall& p, int lane, int mine) {
  uint32_t c = cost_of(mine);
  for (int b = lane + 32; b < p.n; b += 32) c += cost_of(entry_tiles(p, b));
  return __reduce_add_sync(0xffffffffu, c);
}
__device__ __forceinline__ Deal make_deal(uint32_t cost, uint32_t runs) {
  Deal d;
  d.share = cost / runs;
  d.more = cost - d.share * runs;
  return d;
}
__device__ __forceinline__ uint32_t run_start(const Deal& d, uint32_t w) { return w * d.share + min(w, d.more); }
// The run that holds cost position x.
__device__ __forceinline__ uint32_t run_of(const Deal& d, uint32_t x) {
  const uint32_t cut = d.more * (d.share + 1);
  return x < cut ? x / (d.share + 1) : d.more + (x - cut) / d.share;
}
// Cost position x as a place among the tiles: entry b, `first` tiles before
// it, and the tile of the call that x stands at.
struct Place {
  int b, tiles;                             // entry and its tiles per unit (0: past the end)
  uint32_t first, tile;
  uint32_t last;                            // cost position of the last tile of x's unit
};
__device__ __forceinline__ Place find_place(const AttnCall& p, int lane, int mine, uint32_t upb, uint32_t x) {
  Place r;
  uint32_t cost0 = 0, tiles0 = 0;           // before this batch of entries
  for (int base = 0; base < p.n; base += 32) {
    const int b = base + lane;
    const int t = base == 0 ? mine : b < p.n ? entry_tiles(p, b) : 0;
    uint32_t cost = cost_of(t) * upb, tiles = t * upb;
    const uint32_t own_cost = cost, own_tiles = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, cost, o), z = __shfl_up_sync(0xffffffffu, tiles, o);
      if (lane >= o) {
        cost += y;
        tiles += z;
      }
    }
    const unsigned past = __ballot_sync(0xffffffffu, cost0 + cost > x);
    if (past) {
      const int l = __ffs(past) - 1;
      r.b = base + l;
      r.tiles = __shfl_sync(0xffffffffu, t, l);
      r.first = tiles0 + __shfl_sync(0xffffffffu, tiles - own_tiles, l);
      const uint32_t in = x - (cost0 + __shfl_sync(0xffffffffu, cost - own_cost, l));
      const uint32_t per = cost_of(r.tiles), u = in / per;
      const int k = (int)(in - u * per) - kUnitCost;
      r.tile = r.first + u * r.tiles + max(k, 0);
      r.last = x - (k + kUnitCost) + per - 1;
      return r;
    }
    cost0 += __shfl_sync(0xffffffffu, cost, 31);
    tiles0 += __shfl_sync(0xffffffffu, tiles, 31);
  }
  r.b = p.n;
  r.tiles = 0;
  r.first = r.tile = tiles0;
  r.last = x;
  return r;
}

// Pieces of a row: softmax references m (sums) and M (outputs), the sum l
// and four output channels.
struct Joined {
  float m, M, l;
  float4 o;
};
__device__ __forceinline__ void join_in(Joined& a, float m, float l, float M, const float4& o) {
  const float mn = fmaxf(a.m, m), Mn = fmaxf(a.M, M);
  const float fa = a.m == mn ? 1.f : ex2_approx(a.m - mn), fb = m == mn ? 1.f : ex2_approx(m - mn);
  const float Fa = a.M == Mn ? 1.f : ex2_approx(a.M - Mn), Fb = M == Mn ? 1.f : ex2_approx(M - Mn);
  a.l = a.l * fa + l * fb;
  a.o.x = a.o.x * Fa + o.x * Fb;
  a.o.y = a.o.y * Fa + o.y * Fb;
  a.o.z = a.o.z * Fa + o.z * Fb;
  a.o.w = a.o.w * Fa + o.w * Fb;
  a.m = mn;
  a.M = Mn;
}
__device__ __forceinline__ Joined nothing_joined() {
  Joined a;
  a.m = a.M = -INFINITY;
  a.l = 0.f;
  a.o = make_float4(0.f, 0.f, 0.f, 0.f);
  return a;
}
// Row r of head h of entry b: channels 4 lane .. 4 lane + 3; 0 where nothing was seen.
__device__ __forceinline__ void write_row(const AttnCall& p, int b, int h, int r, int lane, const Joined& a) {
  if (lane * 4 >= p.c.d) return;
  const float f = a.l == 0.f ? 0.f : ex2_approx(a.M - a.m) / a.l;
  const __nv_bfloat162 h0 = __floats2bfloat162_rn(a.o.x * kUnlift * f, a.o.y * kUnlift * f),
                       h1 = __floats2bfloat162_rn(a.o.z * kUnlift * f, a.o.w * kUnlift * f);
  uint2 w = make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
  if (a.l == 0.f) w = make_uint2(0u, 0u);
  *reinterpret_cast<uint2*>(p.out + (((size_t)b * p.Hq + (size_t)h * p.g) * p.T + r) * p.c.d + lane * 4) = w;
}

// EXACT: d == DP, so that a tile's row offsets are constants.
template <int CODE, int DP, int NR, bool EXACT>
__global__ void __launch_bounds__(kThreads, kCtas(DP)) attention_kernel(const AttnCall p) {
  constexpr int KS = DP / 16;               // MMAs along d for S, and row blocks of O
  constexpr int KB = DP / 4, VB = DP / 8;   // bytes a lane takes of a K row, of a V row
  constexpr int RB = 8 * NR;
  extern __shared__ uint8_t smem[];
  grid_dep_wait();
  grid_dep_launch();
  const Cache& c = p.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g8 = lane >> 2, c4 = lane & 3;
  const int worker = blockIdx.x * kWarps + warp;
  const int upb = c.Hkv;                    // units (heads) per sequence
  // team: the unit of this CTA's cluster (of p.team CTAs), with its row group
  const int mate = p.team > 1 ? (int)cluster_rank() : 0, unit_rg = p.team ? (int)blockIdx.x / p.team : 0;
  const int rg = (p.team ? unit_rg : worker) % p.RG;   // the warp's row group
  uint8_t* ring = smem + warp * kStages * kStageBytes;
  const uint32_t ring_s = dropkv::smem_addr(ring);
  // this warp's run: tiles x0, x0 + stride, ... below x1 of the call; entry b0
  // holds x0 and begins at tile cum0
  uint32_t x0, x1, cum0 = 0;
  int b0, stride = 1;
  bool cut = false;                         // the run begins inside a unit
  int run_last = 0;                         // last run of the unit the next run begins inside
  if (p.team) {
    // the unit, dealt to the warps tile by tile; tiles are counted from its entry on
    const int un = unit_rg / p.RG;
    b0 = un / upb;
    const int tiles = span_of(entry_len(p, b0, true), p.T, p.window, p.sinks).tiles;
    x1 = (uint32_t)(un - b0 * upb + 1) * tiles;
    x0 = x1 - tiles + mate * kWarps + warp;
    stride = kWarps * p.team;
  } else if (p.solo) {
    // one unit and row group, all its tiles
    if (worker >= p.workers) return;
    const int un = worker / p.RG;
    b0 = un / upb;
    const int h = un - b0 * upb;
    const int tiles = span_of(entry_len(p, b0, true), p.T, p.window, p.sinks).tiles;
    if (tiles == 0) {                       // its rows see nothing
      const int r0 = rg * RB, units8 = c.d / 8;
      uint4* o = reinterpret_cast<uint4*>(p.out + (((size_t)b0 * p.Hq + (size_t)h * p.g) * p.T + r0) * c.d);
      for (int u = lane; u < min(RB, p.R - r0) * units8; u += 32) o[u] = make_uint4(0, 0, 0, 0);
      return;
    }
    x1 = (uint32_t)(h + 1) * tiles;         // counted from its entry on
    x0 = x1 - tiles;
  } else {
    if (worker >= p.workers) return;
    // rows of sequences with nothing to read
    for (int b = worker; b < p.n; b += p.workers) {
      if (span_of(entry_len(p, b, true), p.T, p.window, p.sinks).tiles > 0) continue;
      if (p.by_unit)
        for (int u = lane; u < upb * p.RG; u += 32) p.cuts[b * upb * p.RG + u] = make_int2(-1, 0);
      uint4* o = reinterpret_cast<uint4*>(p.out + (size_t)b * p.Hq * p.T * c.d);
      for (int u = lane; u < p.Hq * p.T * (c.d / 8); u += 32) o[u] = make_uint4(0, 0, 0, 0);
    }
    const int mine = lane < p.n ? entry_tiles(p, lane) : 0;
    const int run = worker / p.RG;
    const Deal deal = make_deal(sum_cost(p, lane, mine) * upb, p.workers / p.RG);
    const Place from = find_place(p, lane, mine, upb, run_start(deal, run));
    const Place to = find_place(p, lane, mine, upb, run_start(deal, run + 1));
    x0 = from.tile;
    x1 = to.tile;
    if (to.tiles > 0) run_last = run_of(deal, to.last);
    b0 = from.b;
    cum0 = from.first;
    cut = from.tiles > 0 && (x0 - cum0) % (uint32_t)from.tiles != 0;
    if (!p.by_unit && lane == 0) p.cuts[worker] = make_int2(-1, 0);
    if (x0 >= x1) return;
  }

  // columns past d stay zero in every stage (copies never touch them)
  if (c.d < kPitch)
    for (int u = lane; u < kStages * kStageBytes / 16; u += 32)
      reinterpret_cast<uint4*>(ring)[u] = make_uint4(0, 0, 0, 0);
  __syncwarp();

  // -------------------------------------------------- tile descriptions
  // Lane l describes tile 32 k + l of the run (table entry and scales:
  // two dependent loads, 32 tiles ahead of their use).
  Tile* meta = reinterpret_cast<Tile*>(smem + kRingBytes) + warp * kMeta;
  int wb = b0;                              // entry the lane's cursor stands at
  uint32_t wcum = cum0;
  auto describe = [&](uint32_t x, Tile* to) {
    if (x >= x1) return;
    int len = entry_len(p, wb, false);
    Span s = span_of(len, p.T, p.window, p.sinks);
    while (x >= wcum + s.tiles * upb) {
      wcum += s.tiles * upb;
      ++wb;
      len = entry_len(p, wb, false);
      s = span_of(len, p.T, p.window, p.sinks);
    }
    const uint32_t y = x - wcum, u = y / (uint32_t)s.tiles;
    const int k = (int)(y - u * s.tiles);
    const int tok = (k < s.ns ? k : s.s2 + (k - s.ns)) * kTok;
    const int sq = p.seqs ? p.seqs[wb] : wb;
    const int pg = c.table[(size_t)sq * c.M + (tok >> c.page_log2)];
    Tile t;
    t.tok = tok;
    t.len = len;
    t.unit = wb * upb + u;
    // slots [lo, len) and the first tokens are seen by some row, every row
    // sees up to len - T and (with a window) from len - window on
    const bool first = tok + kTok <= p.sinks;
    t.how = (tok + kTok > len || (tok < s.lo && !first) ? kPartial : 0) |
            (tok + kTok > len - p.T + 1 || (p.window > 0 && tok < len - p.window && !first) ? kMasked : 0);
    if (pg < 0 || pg >= c.P) {
      flag(c.status, KVCACHE_FLAG_BAD_PAGE);
      t.at = 0;
      t.ks = 0.f;
      t.lv = 0.f;
      t.how = kPartial | kMasked | kUnreadable;
    } else {
      const size_t ur = (size_t)pg * c.Hkv + u;
      t.at = (long long)(ur * c.page + (tok & (c.page - 1))) * c.d;
      t.ks = c.ks[ur];
      t.lv = __log2f(fmaxf(c.vs[ur], 0x1p-126f));
    }
    *to = t;
  };

  // -------------------------------------------------- copies
  const int units16 = (c.d + 15) >> 4;      // 16-byte pieces of a row (the last may be 8 bytes)
  const bool odd8 = (c.d & 15) != 0;
  auto copy_tile = [&](int stage, const Tile* from) {
    const long long at0 = from->at;
    const int tok = from->tok, len = from->len, how = from->how;
    const uint8_t* kp = c.k + at0;
    const uint8_t* vp = c.v + at0;
    const uint32_t base = ring_s + stage * kStageBytes;
    int v0 = 0, v1 = kTok, v2 = 0;          // rows [v0, v1) and [0, v2) are seen by some row
    if (how & kPartial) {
      v1 = how & kUnreadable ? 0 : min(kTok, len - tok);
      if (p.window > 0 && !(how & kUnreadable)) {
        v0 = max(0, span_of(len, p.T, p.window, p.sinks).lo - tok);
        v2 = min(v1, p.sinks - tok);
      }
    }
    if (!odd8 && !(how & kPartial)) {
      // the whole tile: 8 lanes take a row's 16-byte pieces, 4 rows at a time
      // (rows r and r + 8 share a swizzle)
      const int piece = lane & 7, r0 = lane >> 3;
      if (piece < units16) {
        const uint32_t even = base + r0 * kPitch + ((piece ^ r0) << 4);
        const uint32_t odd = base + (r0 + 4) * kPitch + ((piece ^ (r0 + 4)) << 4);
        kp += r0 * c.d + piece * 16;
        vp += r0 * c.d + piece * 16;
        const int step = EXACT ? 4 * DP : 4 * c.d;
#pragma unroll
        for (int u = 0; u < kTok / 4; ++u) {
          const uint32_t at = (u & 1 ? odd : even) + (u >> 1) * 8 * kPitch;
          cp_async_cg(at, kp + u * step);
          cp_async_cg(at + kTok * kPitch, vp + u * step);
        }
      }
    } else if (!odd8) {
      // 8 lanes take a row's 16-byte pieces, 4 rows at a time
      const int piece = lane & 7, r0 = lane >> 3;
      if (piece < units16) {
#pragma unroll
        for (int u = 0; u < kTok / 4; ++u) {
          const int r = r0 + 4 * u;
          const bool take = (r >= v0 && r < v1) || r < v2;
          const uint32_t at = base + r * kPitch + ((piece ^ (r & 7)) << 4);
          const size_t off = take ? (size_t)r * c.d + piece * 16 : 0;
          cp16(at, kp + off, take);
          cp16(at + kTok * kPitch, vp + off, take);
        }
      }
    } else {
      const int piece = lane & 15, r0 = lane >> 4;   // 8-byte pieces, 2 rows at a time
      if (piece * 8 < c.d) {
#pragma unroll 4
        for (int u = 0; u < kTok / 2; ++u) {
          const int r = r0 + 2 * u;
          const bool take = (r >= v0 && r < v1) || r < v2;
          const uint32_t at = base + r * kPitch + (((piece >> 1) ^ (r & 7)) << 4) + (piece & 1) * 8;
          const size_t off = take ? (size_t)r * c.d + piece * 8 : 0;
          cp8(at, kp + off, take);
          cp8(at + kTok * kPitch, vp + off, take);
        }
      }
    }
  };

  // -------------------------------------------------- state of the current unit
  uint32_t qf[NR][KS][2];                   // query rows as the B operand
  float fq[NR][2];                          // rows 2 c4, 2 c4 + 1: logit factor (base-2)
  int pos[NR][2];                           // their positions (-1: no such row)
  float o[NR][KS][4];
  float m[NR][2], M[NR][2], l[NR][2];
  int unit = -1, len = 0;
  int unit_first = 0;                       // tile of the run the unit's part starts at

  auto load_unit = [&](int un, int ln) {
    unit = un;
    len = ln;
    const int b = un / upb, h = un - b * upb;
    const __nv_bfloat16* q = p.q + ((size_t)b * p.Hq + (size_t)h * p.g) * p.T * c.d;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const int r = rg * RB + nr * 8 + g8;
      float x[KB];
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < KB; e += 8) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < p.R && c4 * KB + e < c.d) w = *reinterpret_cast<const uint4*>(q + (size_t)r * c.d + c4 * KB + e);
        const uint32_t w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[e + 2 * i] = __uint_as_float(w4[i] << 16);
          x[e + 2 * i + 1] = __uint_as_float(w4[i] & 0xFFFF0000u);
          amax = fmaxf(amax, fmaxf(fabsf(x[e + 2 * i]), fabsf(x[e + 2 * i + 1])));
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // a power of two that brings the row's largest element to [2^14, 2^15)
      const int e = min(126, max(-113, 14 - ((int)(__float_as_uint(amax) >> 23) - 127)));
      const float up = __uint_as_float((uint32_t)(e + 127) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        qf[nr][s][0] = pack_half2(x[4 * s] * up, x[4 * s + 1] * up);
        qf[nr][s][1] = pack_half2(x[4 * s + 2] * up, x[4 * s + 3] * up);
      }
      // lane (g8, c4) needs the factors of rows 2 c4 and 2 c4 + 1 (held by lanes with that g8)
      const float f = down * p.scale_log2;
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        fq[nr][e2] = __shfl_sync(0xffffffffu, f, (2 * c4 + e2) * 4);
        const int rr = rg * RB + nr * 8 + 2 * c4 + e2;
        pos[nr][e2] = rr < p.R ? ln - p.T + rr % p.T : -1;
        m[nr][e2] = M[nr][e2] = -INFINITY;
        l[nr][e2] = 0.f;
      }
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nr][s][i] = 0.f;
    }
  };

  // The unit's part ends: the output, or this run's piece of it.
  auto store_unit = [&](bool whole, int slot) {
    if (lane == 0) {
      // who joins it: the run it begins in says so
      if (p.by_unit) {
        if (whole) p.cuts[unit * p.RG + rg] = make_int2(-1, 0);
        else if (slot == 1) p.cuts[unit * p.RG + rg] = make_int2(worker / p.RG, run_last);
      } else if (slot == 1 && !whole) {
        p.cuts[worker] = make_int2(unit, run_last);
      }
    }
    const int b = unit / upb, h = unit - b * upb;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], s);
        const int rl = nr * 8 + 2 * c4 + e, r = rg * RB + rl;
        if (r >= p.R) continue;
        if (whole) {
          // o stands for o 2^(M - m - 7); a row that saw nothing has l = 0
          const float f = l[nr][e] == 0.f ? 0.f : ex2_approx(M[nr][e] - m[nr][e]) / l[nr][e];
          __nv_bfloat16* dst = p.out + (((size_t)b * p.Hq + (size_t)h * p.g) * p.T + r) * c.d + g8 * VB;
#pragma unroll
          for (int s = 0; s < KS; s += 4) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 h2 =
                  __floats2bfloat162_rn(o[nr][s + i][e] * kUnlift * f, o[nr][s + i][2 + e] * kUnlift * f);
              w[i] = l[nr][e] == 0.f ? 0u : *reinterpret_cast<const uint32_t*>(&h2);
            }
            if (g8 * VB + 2 * s < c.d) *reinterpret_cast<uint4*>(dst + 2 * s) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          const size_t row = ((size_t)worker * 2 + slot) * RB + rl;
          float* dst = p.part_o + row * c.d + g8 * VB;
#pragma unroll
          for (int s = 0; s < KS; s += 2)
            if (g8 * VB + 2 * s < c.d)
              *reinterpret_cast<float4*>(dst + 2 * s) =
                  make_float4(o[nr][s][e], o[nr][s][2 + e], o[nr][s + 1][e], o[nr][s + 1][2 + e]);
          if (g8 == 0) p.part_s[row] = make_float4(m[nr][e], l[nr][e], M[nr][e], 0.f);
        }
      }
  };

  // -------------------------------------------------- the run
  const int T_run = x0 < x1 ? (int)(x1 - x0 + stride - 1) / stride : 0;
  describe(x0 + lane * stride, meta + lane);
  __syncwarp();
  auto issue = [&](int i) {                 // stage the copy of run tile i
    if (i < T_run) copy_tile(i % kStages, meta + (i & (kMeta - 1)));
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

#pragma unroll 1
  for (int i = 0; i < T_run; ++i) {
    // the batch after this one takes the place of the one before
    if ((i & 31) == 0) describe(x0 + (i + 32 + lane) * stride, meta + ((i + 32) & (kMeta - 1)) + lane);
    __syncwarp();                           // tile i - 1 has been read by every lane
    issue(i + kStages - 1);
    const Tile* now = meta + (i & (kMeta - 1));
    const int un = now->unit, tok = now->tok, ln = now->len, how = now->how;
    const float ks = now->ks, lv = now->lv;
    if (un != unit) {
      if (unit >= 0) {
        // the part before ends with its unit; it is whole when the unit began in this run
        const Span s = span_of(len, p.T, p.window, p.sinks);
        store_unit(i - unit_first >= s.tiles, 0);
      }
      load_unit(un, ln);
      unit_first = i;
    }
    cp_wait<kStages - 1>();
    __syncwarp();
    const uint8_t* sk = ring + (i % kStages) * kStageBytes;
    const uint8_t* sv = sk + kTok * kPitch;

    // S^T: tokens mt * 16 + g8 (+ 8) against rows 2 c4 (+ 1)
    float s[NR][2][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int ch = 0; ch < KB / 16; ++ch) {
        const int t0 = mt * 16 + g8;        // t0 & 7 == (t0 + 8) & 7
        const int at = (((c4 * (KB / 16) + ch) ^ (t0 & 7)) << 4);
        const uint4 wa = *reinterpret_cast<const uint4*>(sk + t0 * kPitch + at);
        const uint4 wb4 = *reinterpret_cast<const uint4*>(sk + (t0 + 8) * kPitch + at);
        const uint32_t a4[4] = {wa.x, wa.y, wa.z, wa.w}, b4[4] = {wb4.x, wb4.y, wb4.z, wb4.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t a[4];
          codes_to_half<CODE>(a4[q], a[0], a[2]);
          codes_to_half<CODE>(b4[q], a[1], a[3]);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            if (ch == 0 && q == 0) mma_f16_first(s[nr][mt], a, qf[nr][0][0], qf[nr][0][1]);
            else mma_f16(s[nr][mt], a, qf[nr][ch * 4 + q][0], qf[nr][ch * 4 + q][1]);
          }
        }
      }
    }

    // masks: only where some row does not see some token of the tile
    if (how & kMasked) {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = tok + mt * 16 + g8 + (e >> 1) * 8, i_pos = pos[nr][e & 1];
            const bool sees = !(how & kUnreadable) && j <= i_pos && (p.window == 0 || j > i_pos - p.window || j < p.sinks);
            if (!sees) s[nr][mt][e] = -INFINITY;
          }
    }

    // softmax of the tile: references m (sums) and M (outputs, which carry the V scale)
    uint32_t pb[NR][2][2];                  // P as the B operand
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      float f[2], mt2[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[e] = fmaxf(fq[nr][e] * ks, 0x1p-126f);   // never 0: a masked logit stays -inf
        float t = fmaxf(fmaxf(s[nr][0][e], s[nr][0][2 + e]), fmaxf(s[nr][1][e], s[nr][1][2 + e]));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
        mt2[e] = t == -INFINITY ? -INFINITY : t * f[e];
      }
      const bool move = mt2[0] > m[nr][0] + kMoveLog2 || mt2[1] > m[nr][1] + kMoveLog2 ||
                        mt2[0] + lv > M[nr][0] + kMoveLog2 || mt2[1] + lv > M[nr][1] + kMoveLog2;
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = mt2[e] > m[nr][e] + kMoveLog2 ? mt2[e] : m[nr][e];
          const float Mn = mt2[e] + lv > M[nr][e] + kMoveLog2 ? mt2[e] + lv : M[nr][e];
          const float fl = m[nr][e] == mn ? 1.f : ex2_approx(m[nr][e] - mn);   // 0 from an empty state
          const float fo = M[nr][e] == Mn ? 1.f : ex2_approx(M[nr][e] - Mn);
          m[nr][e] = mn;
          M[nr][e] = Mn;
          l[nr][e] *= fl;
#pragma unroll
          for (int q = 0; q < KS; ++q) {
            o[nr][q][e] *= fo;
            o[nr][q][2 + e] *= fo;
          }
        }
      }
      // rows 2 c4 and 2 c4 + 1 side by side in packed pairs
      const float r0 = m[nr][0] == -INFINITY ? 0.f : m[nr][0], r1 = m[nr][1] == -INFINITY ? 0.f : m[nr][1];
      const uint64_t f2 = f2_pack(f[0], f[1]), n2 = f2_pack(-r0, -r1);
      // P enters the product as p 2^(lv + m - M + 7) <= 2^15; the cap keeps 0 times it finite
      const uint64_t cv2 = f2_pack(ex2_approx(fminf(lv + r0 - M[nr][0], 100.f) + kLiftLog2),
                                   ex2_approx(fminf(lv + r1 - M[nr][1], 100.f) + kLiftLog2));
      uint64_t sum2 = 0ull;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          const uint64_t x2 = f2_fma(f2_pack(s[nr][mt][2 * e2], s[nr][mt][2 * e2 + 1]), f2, n2);
          const uint64_t p2 = f2_pack(ex2_approx(f2_lo(x2)), ex2_approx(f2_hi(x2)));
          sum2 = f2_add(sum2, p2);
          const uint64_t w2 = f2_mul(p2, cv2);
          pb[nr][mt][e2] = movmatrix(pack_half2(f2_lo(w2), f2_hi(w2)));
        }
      l[nr][0] += f2_lo(sum2);
      l[nr][1] += f2_hi(sum2);
    }

    // O^T += V^T P: k index (2 c4, 2 c4 + 1, +8, +9) = tokens, rows = the lane's channels
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t vw[4][VB / 4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int tk = mt * 16 + 2 * c4 + (t & 1) + (t >> 1) * 8;
        if constexpr (VB == 16) {
          const uint4 w = *reinterpret_cast<const uint4*>(sv + tk * kPitch + ((g8 ^ (tk & 7)) << 4));
          vw[t][0] = w.x; vw[t][1] = w.y; vw[t][2] = w.z; vw[t][3] = w.w;
        } else {
          const uint2 w =
              *reinterpret_cast<const uint2*>(sv + tk * kPitch + (((g8 >> 1) ^ (tk & 7)) << 4) + (g8 & 1) * 8);
          vw[t][0] = w.x; vw[t][1] = w.y;
        }
      }
#pragma unroll
      for (int j = 0; j < VB / 4; ++j) {
        uint32_t a0[4], a1[4];              // row blocks 2 j (channels 4 j, 4 j + 1) and 2 j + 1
        codes_to_half<CODE>(__byte_perm(vw[0][j], vw[1][j], 0x5140), a0[0], a0[1]);
        codes_to_half<CODE>(__byte_perm(vw[0][j], vw[1][j], 0x7362), a1[0], a1[1]);
        codes_to_half<CODE>(__byte_perm(vw[2][j], vw[3][j], 0x5140), a0[2], a0[3]);
        codes_to_half<CODE>(__byte_perm(vw[2][j], vw[3][j], 0x7362), a1[2], a1[3]);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          mma_f16(o[nr][2 * j], a0, pb[nr][mt][0], pb[nr][mt][1]);
          mma_f16(o[nr][2 * j + 1], a1, pb[nr][mt][0], pb[nr][mt][1]);
        }
      }
    }
  }
  if (p.team) {
    // the warps' pieces of the unit, through shared memory (each warp's ring)
    float* po = reinterpret_cast<float*>(ring);
    float4* ps = reinterpret_cast<float4*>(meta);
    __syncwarp();
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rl = nr * 8 + 2 * c4 + e;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], x);
#pragma unroll
        for (int s = 0; s < KS; s += 2)
          *reinterpret_cast<float4*>(po + rl * DP + g8 * VB + 2 * s) =
              T_run > 0 ? make_float4(o[nr][s][e], o[nr][s][2 + e], o[nr][s + 1][e], o[nr][s + 1][2 + e])
                        : make_float4(0.f, 0.f, 0.f, 0.f);
        if (g8 == 0)
          ps[rl] = T_run > 0 ? make_float4(m[nr][e], l[nr][e], M[nr][e], 0.f) : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
      }
    // the rows are shared out over the team's warps
    if (p.team > 1) cluster_sync();
    else __syncthreads();
    const uint32_t base = dropkv::smem_addr(smem);
    const int h = (unit_rg / p.RG) % upb;
    for (int rl = mate * kWarps + warp; rl < min(RB, p.R - rg * RB); rl += stride) {
      Joined a = nothing_joined();
      for (int mt = 0; mt < p.team; ++mt) {
        float4 st[kWarps], ov[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const uint32_t sa = base + kRingBytes + w * kMeta * (int)sizeof(Tile) + rl * 16;
          const uint32_t oa = base + w * kStages * kStageBytes + (rl * DP + lane * 4) * 4;
          st[w] = ld_cluster(sa, mt);
          ov[w] = lane * 4 < DP ? ld_cluster(oa, mt) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) join_in(a, st[w].x, st[w].y, st[w].z, ov[w]);
      }
      write_row(p, b0, h, rg * RB + rl, lane, a);
    }
    if (p.team > 1) cluster_sync();         // no CTA leaves while its shared memory is read
    return;
  }
  // the last part: whole when all tiles of its unit lie in this run; else its
  // piece goes to slot 0 if the unit began before the run, slot 1 if it began inside
  const int tiles = span_of(len, p.T, p.window, p.sinks).tiles;
  store_unit(T_run - unit_first >= tiles, unit_first == 0 && cut ? 0 : 1);
}

// Joins the pieces of the units that run borders cut, in run order.  Each
// unit's first run has left word of its last one (per unit, or per run where
// there are more units than runs), so nothing is searched for here.
// ROWWISE: a CTA joins one row of a unit, its warps sharing out the pieces
// with all loads in flight at once (few units, up to hundreds of pieces
// each); else each warp joins a row on its own (few pieces each).
template <bool ROWWISE>
__global__ void __launch_bounds__(ROWWISE ? kJoinWide : kJoinThreads) join_kernel(const AttnCall p) {
  constexpr int kW = (ROWWISE ? kJoinWide : kJoinThreads) / 32, kBatch = ROWWISE ? 10 : 8;
  grid_dep_wait();
  // Three attention CTAs fill an SM's registers.  Started while CTAs of the
  // join are there, they settle beside them, and the hole that these leave is
  // too small for the third, which then runs behind the others: there the next
  // kernel starts once the join is gone (attention after attention, one row
  // per head, e4m3: 24 x up to 4000 tokens of 32 heads 55.3 -> 39.2 us, 32 x
  // up to 2000 38.7 -> 31.0; with a store between, which clears the SMs,
  // 45.0 -> 45.2 and 36.1 -> 37.0, 1 x 131072 tokens 39.9 -> 37.9).
  if (kCtas(p.c.d) <= 2) grid_dep_launch();
  __shared__ float4 s_o[kW][32];
  __shared__ float s_l[kW], s_m[kW], s_M[kW];
  const Cache& c = p.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int2 cut = p.cuts[blockIdx.x];
  if (cut.x < 0) return;
  const int un = p.by_unit ? (int)blockIdx.x / p.RG : cut.x, rg = blockIdx.x % p.RG;
  const int w0 = p.by_unit ? cut.x : (int)blockIdx.x / p.RG, w1 = cut.y;   // runs
  const int b = un / c.Hkv, h = un - b * c.Hkv;
  const int rows = min(p.RB, p.R - rg * p.RB);
  const bool cols = lane * 4 < c.d;
  // pieces w0 + first, w0 + first + step, ... of row rl; the unit begins in
  // run w0 (its slot 1) and before every later one (slot 0)
  auto take = [&](int rl, int first, int step) {
    Joined a = nothing_joined();
    for (int base = w0 + first; base <= w1; base += step * kBatch) {
      float4 st[kBatch], ov[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int w = base + k * step;
        st[k] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
        ov[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (w <= w1) {
          const size_t row = (((size_t)w * p.RG + rg) * 2 + (w == w0 ? 1 : 0)) * p.RB + rl;
          st[k] = p.part_s[row];
          if (cols) ov[k] = *reinterpret_cast<const float4*>(p.part_o + row * c.d + lane * 4);
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) join_in(a, st[k].x, st[k].y, st[k].z, ov[k]);
    }
    return a;
  };
  if constexpr (ROWWISE) {
    const int rl = blockIdx.y;
    if (rl >= rows) return;
    Joined a = take(rl, warp, kW);
    s_o[warp][lane] = a.o;
    if (lane == 0) {
      s_l[warp] = a.l;
      s_m[warp] = a.m;
      s_M[warp] = a.M;
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int k = 1; k < kW; ++k) join_in(a, s_m[k], s_l[k], s_M[k], s_o[k][lane]);
    write_row(p, b, h, rg * p.RB + rl, lane, a);
  } else {
    const int rl = blockIdx.y * kW + warp;
    if (rl < rows) write_row(p, b, h, rg * p.RB + rl, lane, take(rl, 0, 1));
  }
}

cudaError_t launch_team(void (*kern)(AttnCall), unsigned units, const AttnCall& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units * p.team);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.team;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.team > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int CODE, int DP, int NR, bool EXACT>
cudaError_t launch_t(const AttnCall& p, cudaStream_t st) {
  auto kern = attention_kernel<CODE, DP, NR, EXACT>;
  cudaError_t e = allow_smem<attention_kernel<CODE, DP, NR, EXACT>>(kSmem);
  if (e != cudaSuccess) return e;
  const unsigned units = (unsigned)(p.n * p.c.Hkv * p.RG);
  if (p.team) return launch_team(kern, units, p, st);
  e = launch_pdl(kern, dim3((p.workers + kWarps - 1) / kWarps), dim3(kThreads), kSmem, st, p);
  if (e != cudaSuccess || p.solo) return e;
  if (p.rowwise) return launch_pdl(join_kernel<true>, dim3(units, std::min(p.RB, p.R)), dim3(kJoinWide), 0, st, p);
  return launch_pdl(join_kernel<false>, dim3(p.by_unit ? units : p.workers, (std::min(p.RB, p.R) + 3) / 4),
                    dim3(kJoinThreads), 0, st, p);
}

template <int CODE>
cudaError_t launch_code(const AttnCall& p, cudaStream_t st) {
  const int NR = p.RB / 8;
  if (p.c.d == 128) return NR == 1 ? launch_t<CODE, 128, 1, true>(p, st) : launch_t<CODE, 128, 2, true>(p, st);
  if (p.c.d == 64) return NR == 1 ? launch_t<CODE, 64, 1, true>(p, st) : launch_t<CODE, 64, 2, true>(p, st);
  if (p.c.d > 64) return NR == 1 ? launch_t<CODE, 128, 1, false>(p, st) : launch_t<CODE, 128, 2, false>(p, st);
  return NR == 1 ? launch_t<CODE, 64, 1, false>(p, st) : launch_t<CODE, 64, 2, false>(p, st);
}

// One wave.
long long wave_of(int sms, int d) { return (long long)sms * kCtas(d) * kWarps; }
// The workspace: outputs of the pieces, their softmax states, who joins what.
size_t pieces_o(long long workers, int RB, int d) { return ((size_t)workers * 2 * RB * d * 4 + 255) / 256 * 256; }
size_t pieces_s(long long workers, int RB) { return ((size_t)workers * 2 * RB * 16 + 255) / 256 * 256; }

}  // namespace

bool make_attn_plan(const kvcache_shape& s, int n, int Hq, int T, int window, int sinks, int sms, AttnPlan* a) {
  const long long R = (long long)Hq / s.Hkv * T;
  // most tiles a unit can have
  long long cap = ((long long)s.max_pages * s.page + kTok - 1) / kTok;
  if ((cap + kUnitCost) * s.Hkv * n >= (1LL << 31)) return false;
  if (window > 0)
    cap = std::min(cap, ((long long)window + T + kTok - 2) / kTok + 1 + ((long long)sinks + kTok - 1) / kTok);
  // Rows a warp holds: 8, or 16 where there are more and each warp has many
  // tiles (32 rows, 16 x 4000 tokens: 49.9 us against 63.7 with 8; 2 x 16000
  // tokens, 3 tiles a warp: 18.8 against 16.7).  Short units that go to one
  // warp each: 16 where 8 would take more than one wave (128 x 64 tokens, 16
  // rows: 13.7 -> 10.4; 16 x 64 tokens, 24 rows would lose, 6.7 -> 8.8).
  const long long pairs16 = (R + 15) / 16 * n * s.Hkv * cap;
  const long long units8 = (R + 7) / 8 * n * s.Hkv, units16 = (R + 15) / 16 * n * s.Hkv, wave = wave_of(sms, s.d);
  const bool shorts = cap <= kSoloTiles;
  a->RB = R > 8 && (pairs16 >= 16 * wave || (shorts && units8 > wave && units16 <= 4 * wave)) ? 16 : 8;
  a->RG = (int)((R + a->RB - 1) / a->RB);
  const long long units = (long long)n * s.Hkv * a->RG;   // with their row groups
  if (units * a->RB >= (1LL << 31)) return false;
  // Many short units (more than have a CTA each at once): a warp each, nothing
  // dealt and nothing to join (8 heads, 152 x 128 tokens: 14.3 -> 8.8 us, 76 x
  // 256: 12.8 -> 10.7, 512 x 32: 25.4 -> 19.7, 152 x 1-384: 21.0 -> 16.6; over
  // four waves both take the same, and from 16 tiles on equal lengths lose, 42 x
  // 512 of 32 heads 42.5 -> 46.7).
  a->solo = shorts && units > 2LL * sms && units <= 4 * wave ? 1 : 0;
  if (a->solo) {
    a->workers = (int)units;
    a->team = a->by_unit = a->rowwise = 0;
    a->part_s = a->cuts = a->total = 0;
    return true;
  }
  // Few units of moderate length: a cluster of 1 to 8 CTAs each, joined through
  // shared memory, no second kernel.  (The bounds count two CTAs an SM, also
  // for heads of up to 64 channels, of which three fit.)  More CTAs while a warp has over 2 tiles
  // and they fit one wave; two waves for units of at most 5 tiles a warp (64 x
  // 300 tokens: 15.8 -> 14.6 us; 48 x 1000 tokens would lose, 26.8 -> 28.9).
  int team = 1;
  while (team < 8 && units * 2 * team <= 2LL * sms && cap > 2LL * kWarps * team) team *= 2;
  a->team = (units <= 2LL * sms && cap <= (long long)kTeamTiles * kWarps * team) ||
                    (units <= 4LL * sms && cap <= 5 * kWarps)
                ? team
                : 0;
  a->workers = (int)(std::max(1LL, std::min(wave_of(sms, s.d) / a->RG, (long long)n * s.Hkv * cap)) * a->RG);
  // Joins: by row where the rows are fewer than the CTAs they can fill
  a->by_unit = units <= a->workers ? 1 : 0;
  a->rowwise = a->by_unit && units * std::min<long long>(R, a->RB) <= 4LL * sms ? 1 : 0;
  a->part_s = pieces_o(a->workers, a->RB, s.d);
  a->cuts = a->part_s + pieces_s(a->workers, a->RB);
  a->total = a->cuts + (size_t)a->workers * 8;
  return true;
}

size_t attn_workspace_bound(const kvcache_shape& s, int Hq, int T, int sms) {
  const long long R = (long long)Hq / s.Hkv * T;
  size_t most = 0;
  for (int RB = 8; RB <= 16; RB += 8) {
    const long long w = std::max(wave_of(sms, s.d), (R + RB - 1) / RB);
    most = std::max(most, pieces_o(w, RB, s.d) + pieces_s(w, RB) + (size_t)w * 8);
  }
  return most;
}

cudaError_t launch_attention(const AttnCall& p, cudaStream_t st) {
  return p.c.code == KVCACHE_INT8 ? launch_code<KVCACHE_INT8>(p, st) : launch_code<KVCACHE_E4M3>(p, st);
}

}  // namespace kvcache
