// Attention over the paged 8-bit cache: the plan of a call and its launch.
#include "kvcache_attn.cuh"

namespace kvcache {
namespace {

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
  return p.c.code == KVCACHE_INT8 ? launch_code<false, KVCACHE_INT8>(p, st) : launch_code<false, KVCACHE_E4M3>(p, st);
}

}  // namespace kvcache
