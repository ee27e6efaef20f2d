// Host side of include/kvcache_step.h: argument checks and launches.  Nothing
// here allocates device memory.
#include <cmath>

#include "kvcache_step_internal.cuh"

using namespace kvcache;
using dropkv::current_sms;
using dropkv::ranges_overlap;

namespace {

dropkv_status open_rotary(const kvcache_rotary* r, Turning* t) {
  if (!r) return DROPKV_ERR_INVALID_ARG;
  if (r->d < 1 || r->dims < 0 || r->dims > r->d || (r->layout != KVCACHE_HALF && r->layout != KVCACHE_INTERLEAVED) ||
      !(r->eps > 0.f) || !std::isfinite(r->eps) || !std::isfinite(r->amplitude) || (r->dims > 0 && !r->turns) ||
      !aligned(r->turns) || !aligned(r->q_norm) || !aligned(r->k_norm))
    return DROPKV_ERR_INVALID_ARG;
  if (r->d % 8 != 0 || r->d > dropkv::kDPad || r->dims % 8 != 0) return DROPKV_ERR_UNSUPPORTED;
  t->turns = reinterpret_cast<const unsigned long long*>(r->turns);
  t->d = r->d;
  t->dims = r->dims;
  t->half = r->layout == KVCACHE_HALF;
  t->eps = r->eps;
  t->amplitude = r->amplitude;
  t->inv_d = 1.0f / (float)r->d;
  return DROPKV_OK;
}

// Rows of n sequences with `heads` heads of `rows` rows each; *bytes: from the
// first to behind the last of them.  A stride over a single item is not used.
bool open_rows(const kvcache_rows& r, long long n, long long heads, long long rows, int d, Rows* to, size_t* bytes) {
  const long long count[3] = {n, heads, rows};
  long long stride[3] = {r.seq, r.head, r.row}, end = d;
  if (!r.data || !aligned(r.data)) return false;
  for (int i = 0; i < 3; ++i) {
    if (count[i] <= 1) stride[i] = 0;
    if (stride[i] < 0 || stride[i] % 8 != 0 || stride[i] > (1LL << 46) / std::max(1LL, count[i])) return false;
    end += stride[i] * std::max(0LL, count[i] - 1);
  }
  to->p = static_cast<const __nv_bfloat16*>(r.data);
  to->seq = stride[0];
  to->head = stride[1];
  to->row = stride[2];
  *bytes = (size_t)end * 2;
  return true;
}

bool dense(const Rows& r, long long n, long long heads, long long rows, int d) {
  return (rows <= 1 || r.row == d) && (heads <= 1 || r.head == rows * d) && (n <= 1 || r.seq == heads * rows * d);
}

// The tiles of all units' shared tokens, at their most, in 32 bits.
bool counts_fit(const kvcache_shape& s, int n, int Hq, int T, int G) {
  const double tiles = (double)s.max_pages * s.page / 128 + 1, units = (double)n * Hq * T / 128 + (double)G * s.Hkv;
  return tiles * units < 2147483648.0;
}

// Cycles that sharing saves, roughly, over all SMs, were the cache's table full of
// shared tokens.  For 128 of them and a KV head: the shared kernel's tile, once for
// a group's rows, against kvcache_attention's, for each member and up to 8 rows
// (three quarters of it for each 8 more; it finds the pages in L2 after the first).
// Where d is no multiple of 16 the codes come in smaller pieces on both sides.
double cycles_saved(const kvcache_shape& s, int n, int G, double R) {
  const double rows = (double)n / G * R;
  const bool odd = s.d % 16 != 0;
  const double apart = n * (odd ? 2000.0 : 700.0 + 5 * s.d) * std::max(1.0, 0.75 * std::ceil(R / 8));
  const double shared = G * (rows > 128 ? 4000 * std::ceil(rows / 256) : odd ? 4000 : 2570);
  return (double)s.max_pages * s.page / 128 * s.Hkv * (apart - shared);
}
// Three more short kernels cost some 35 us (67000 cycles at 1.9 GHz); as tables are
// longer than what is shared, a third more is asked for (with 67000, 10 x 2-5 behind
// 2300 to 3600, 16 heads of 128, 3 rows, would take 81 us instead of attention's 62).
// Attention and shared, us, with up to 200 tokens of their own:
//   8, 16 x 16000 tokens in one group, 8 heads of 128       41 and 69   49 and 54
//   8, 16 x 4000, 32 heads of 96, int8                      47 and 84   47 and 51
//   64 x 32768, 8 heads of 128                              428         87
//   10 x 2 behind 18000-28000, 4 heads of 96, 7 rows        68          98
//   11 x 3 behind 19000-63000, 8 heads of 16, 4 rows        189         247
//   2 x 4 behind 23000-48000, 16 heads of 80, 40 rows       513         184
//   10 x 4-7 behind 64000-96000, one head of 112, 6 rows    161         119
// Short prompts in a long table are where it is wrong: 8 behind 100, 1000, 4000
// tokens, 8 heads of 128, 512 to 10000 pages of 64: 12, 14, 19     33, 32, 37
constexpr double kSharingCycles = 90000;

// The workspace of a shared attention (byte offsets); the second half's parts
// and cuts have the sizes given.
struct SharedSpace {
  size_t plan, entries, info, groups, piece_o, piece_s, own_o, own_s, part_o, part_s, cuts, total;
};
SharedSpace make_shared_space(const kvcache_shape& s, int n, int Hq, int T, int G, int sms, size_t part_o, size_t part_s,
                              size_t cuts) {
  SharedSpace w;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += (bytes + 255) / 256 * 256;
    return x;
  };
  const size_t rows = (size_t)n * Hq * T, pieces = (size_t)sms * 256 + 2 * rows;
  w.plan = take(sizeof(SharedPlan));
  w.entries = take((size_t)n * 3 * 4);
  w.info = take((size_t)n * 16);
  w.groups = take(((size_t)G * 4 + 1) * 4);
  w.piece_o = take(pieces * s.d * 4);
  w.piece_s = take(pieces * 16);
  w.own_o = take(rows * s.d * 4);
  w.own_s = take(rows * 16);
  w.part_o = take(part_o);
  w.part_s = take(part_s);
  w.cuts = take(cuts);
  w.total = at;
  return w;
}

}  // namespace

extern "C" {

dropkv_status kvcache_rotate(const kvcache_rotate_call* call) {
  if (!call) return DROPKV_ERR_INVALID_ARG;
  RotateCall p{};
  const dropkv_status st = open_rotary(call->rotary, &p.how);
  if (st != DROPKV_OK) return st;
  const int d = p.how.d;
  if (call->B < 0 || call->n < 0 || call->Hq < 1 || call->Hkv < 1 || !call->status || !aligned(call->status, 4) ||
      !aligned(call->positions, 4) || !aligned(call->lengths, 4) ||
      (call->position_kind != KVCACHE_FIRST && call->position_kind != KVCACHE_EACH))
    return DROPKV_ERR_INVALID_ARG;
  if ((long long)call->Hq + call->Hkv > 65535 || (long long)call->B * call->n >= (1LL << 31)) return DROPKV_ERR_UNSUPPORTED;
  if (call->B == 0 || call->n == 0 || (!call->q.data && !call->k.data)) return DROPKV_OK;
  const kvcache_rows* in[2] = {&call->q, &call->k};
  void* out[2] = {call->q_out, call->k_out};
  size_t in_bytes[2] = {0, 0}, out_bytes[2] = {0, 0};
  p.heads[0] = call->Hq;
  p.heads[1] = call->Hkv;
  for (int w = 0; w < 2; ++w) {
    if (!in[w]->data) continue;
    if (!open_rows(*in[w], call->B, p.heads[w], call->n, d, &p.in[w], &in_bytes[w]) || !out[w] || !aligned(out[w]))
      return DROPKV_ERR_INVALID_ARG;
    p.out[w] = static_cast<__nv_bfloat16*>(out[w]);
    out_bytes[w] = (size_t)call->B * p.heads[w] * call->n * d * 2;
  }
  for (int w = 0; w < 2; ++w)
    for (int x = 0; x < 2; ++x) {
      if (!in[w]->data || !in[x]->data) continue;
      const bool in_place = w == x && in[x]->data == out[w] && dense(p.in[x], call->B, p.heads[x], call->n, d);
      if (!in_place && ranges_overlap(out[w], out_bytes[w], in[x]->data, in_bytes[x])) return DROPKV_ERR_INVALID_ARG;
      if (w != x && ranges_overlap(out[w], out_bytes[w], out[x], out_bytes[x])) return DROPKV_ERR_INVALID_ARG;
    }
  p.weight[0] = call->rotary->q_norm;
  p.weight[1] = call->rotary->k_norm;
  p.positions = call->positions;
  p.each = call->position_kind == KVCACHE_EACH;
  p.lengths = call->lengths;
  p.B = call->B;
  p.n = call->n;
  p.status = call->status;
  const int sms = current_sms(nullptr);
  if (sms <= 0) return DROPKV_ERR_CUDA;
  return launched(launch_rotate(p, sms, call->stream));
}

dropkv_status kvcache_rotate_store(const kvcache_rotate_store_call* call) {
  if (!call) return DROPKV_ERR_INVALID_ARG;
  RotateStoreCall p{};
  dropkv_status st = open_cache(call->shape, call->cache, call->layer, call->n, call->status, &p.c);
  if (st != DROPKV_OK) return st;
  st = open_rotary(call->rotary, &p.how);
  if (st != DROPKV_OK) return st;
  const int n = call->n, rows = call->rows, d = p.c.d, Hkv = p.c.Hkv;
  if (p.how.d != d || rows < 0 || (call->q.data && call->Hq < 1) || !aligned(call->seqs, 4) ||
      !aligned(call->counts, 4) || !aligned(call->positions, 4) ||
      (call->position_kind != KVCACHE_FIRST && call->position_kind != KVCACHE_EACH))
    return DROPKV_ERR_INVALID_ARG;
  if (n == 0 || rows == 0) return DROPKV_OK;
  const long long Hq = call->q.data ? call->Hq : 0;
  if (Hq * rows >= (1LL << 30) || (rows / (long long)p.c.page + 2) * 2 * Hkv + Hq * rows / 16 >= (1LL << 31))
    return DROPKV_ERR_UNSUPPORTED;
  size_t bytes[3] = {0, 0, 0};
  if (!open_rows(call->k, n, Hkv, rows, d, &p.kv[0], &bytes[0]) ||
      !open_rows(call->v, n, Hkv, rows, d, &p.kv[1], &bytes[1]))
    return DROPKV_ERR_INVALID_ARG;
  if (call->q.data) {
    const size_t out = (size_t)n * Hq * rows * d * 2;
    if (!open_rows(call->q, n, Hq, rows, d, &p.q, &bytes[2]) || !call->q_out || !aligned(call->q_out) ||
        ranges_overlap(call->q_out, out, call->q.data, bytes[2]) ||
        ranges_overlap(call->q_out, out, call->k.data, bytes[0]) ||
        ranges_overlap(call->q_out, out, call->v.data, bytes[1]))
      return DROPKV_ERR_INVALID_ARG;
  }
  p.q_out = static_cast<__nv_bfloat16*>(call->q_out);
  p.q_weight = call->rotary->q_norm;
  p.k_weight = call->rotary->k_norm;
  p.seqs = call->seqs;
  p.counts = call->counts;
  p.positions = call->positions;
  p.each = call->position_kind == KVCACHE_EACH;
  p.n = n;
  p.Hq = (int)Hq;
  p.rows = rows;
  return launched(launch_rotate_store(p, call->stream));
}

dropkv_status kvcache_read(const kvcache_read_call* call) {
  if (!call) return DROPKV_ERR_INVALID_ARG;
  ReadCall p{};
  const dropkv_status st = open_cache(call->shape, call->cache, call->layer, call->n, call->status, &p.c);
  if (st != DROPKV_OK) return st;
  if (call->rows < 0 || !aligned(call->seqs, 4) || !aligned(call->starts, 4) || !aligned(call->counts, 4))
    return DROPKV_ERR_INVALID_ARG;
  if (call->n == 0 || call->rows == 0) return DROPKV_OK;
  const size_t bytes = (size_t)call->n * p.c.Hkv * call->rows * p.c.d * 2;
  if (!call->k_out || !call->v_out || !aligned(call->k_out) || !aligned(call->v_out) ||
      ranges_overlap(call->k_out, bytes, call->v_out, bytes))
    return DROPKV_ERR_INVALID_ARG;
  p.seqs = call->seqs;
  p.starts = call->starts;
  p.counts = call->counts;
  p.k = static_cast<__nv_bfloat16*>(call->k_out);
  p.v = static_cast<__nv_bfloat16*>(call->v_out);
  p.n = call->n;
  p.rows = call->rows;
  return launched(launch_read(p, call->stream));
}

size_t kvcache_shared_workspace_size(const kvcache_shape* shape, int32_t n, int32_t Hq, int32_t T, int32_t G) {
  const int sms = current_sms(nullptr);
  if (sms <= 0 || check_shape(shape) != DROPKV_OK || Hq < 1 || T < 1 || Hq % shape->Hkv != 0 || G < 1 || G > n ||
      n > shape->seqs || n > 65535 || (long long)Hq * T > kMaxSharedRows / n || !counts_fit(*shape, n, Hq, T, G))
    return 0;
  // the second half's pieces at their most, for any number of entries up to n
  const SharedSpace w = make_shared_space(*shape, n, Hq, T, G, sms, 0, 0, 0);
  return w.total + attn_workspace_bound(*shape, Hq, T, sms) + (size_t)n * shape->Hkv * ((Hq / shape->Hkv * T + 7) / 8) * 8 + 256;
}

dropkv_status kvcache_shared_attention(const kvcache_shared_attention_call* call) {
  if (!call) return DROPKV_ERR_INVALID_ARG;
  SharedCall p{};
  AttnCall& a = p.own;
  const dropkv_status st = open_cache(call->shape, call->cache, call->layer, call->n, call->status, &a.c);
  if (st != DROPKV_OK) return st;
  const kvcache_shape& shape = *call->shape;
  const int n = call->n, Hq = call->Hq, T = call->T;
  if (!call->q || !call->out || !aligned(call->q) || !aligned(call->out) || Hq < 1 || T < 1 || Hq % shape.Hkv != 0 ||
      !aligned(call->seqs, 4))
    return DROPKV_ERR_INVALID_ARG;
  if (n == 0) return DROPKV_OK;
  if (call->G < 1 || call->G > n || !call->groups || !aligned(call->groups, 4)) return DROPKV_ERR_INVALID_ARG;
  if ((long long)Hq * T > kMaxSharedRows / n) return DROPKV_ERR_UNSUPPORTED;
  const size_t bytes = (size_t)n * Hq * T * shape.d * 2;
  if (ranges_overlap(call->q, bytes, call->out, bytes)) return DROPKV_ERR_INVALID_ARG;
  const int sms = current_sms(nullptr);
  if (sms <= 0) return DROPKV_ERR_CUDA;
  if (call->least < 0 ? cycles_saved(shape, n, call->G, (double)(Hq / shape.Hkv) * T) < kSharingCycles * sms
                      : 2.0 * n * shape.max_pages * shape.page * shape.Hkv * shape.d < (double)call->least)
    return kvcache_attention(call->shape, call->cache, call->layer, call->seqs, n, call->q, Hq, T, 0, 0, call->out,
                             call->workspace, call->workspace_bytes, call->status, call->stream);
  AttnPlan plan{};
  if (!make_attn_plan(shape, n, Hq, T, 0, 0, sms, &plan) || !counts_fit(shape, n, Hq, T, call->G)) return DROPKV_ERR_UNSUPPORTED;
  const bool by_runs = !plan.team && !plan.solo;
  const SharedSpace w = make_shared_space(shape, n, Hq, T, call->G, sms, by_runs ? plan.part_s : 0,
                                          by_runs ? plan.cuts - plan.part_s : 0,
                                          by_runs ? (size_t)n * shape.Hkv * plan.RG * 8 : 0);
  if (!call->workspace || call->workspace_bytes < w.total || !aligned(call->workspace)) return DROPKV_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(call->workspace);
  a.seqs = call->seqs;
  a.n = n; a.Hq = Hq; a.T = T;
  a.g = Hq / shape.Hkv;
  a.R = a.g * T;
  a.RB = plan.RB; a.RG = plan.RG; a.workers = plan.workers; a.solo = plan.solo; a.team = plan.team;
  a.by_unit = 1;
  a.q = static_cast<const __nv_bfloat16*>(call->q);
  a.out = static_cast<__nv_bfloat16*>(call->out);
  a.part_o = reinterpret_cast<float*>(ws + w.part_o);
  a.part_s = reinterpret_cast<float4*>(ws + w.part_s);
  a.cuts = reinterpret_cast<int2*>(ws + w.cuts);
  a.own_o = reinterpret_cast<float*>(ws + w.own_o);
  a.own_s = reinterpret_cast<float4*>(ws + w.own_s);
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)shape.d));
  p.by_runs = by_runs;
  p.groups = call->groups;
  p.G = call->G;
  p.sms = sms;
  p.plan = reinterpret_cast<SharedPlan*>(ws + w.plan);
  p.from = reinterpret_cast<int32_t*>(ws + w.entries);
  p.group = p.from + n;
  p.bound = p.group + n;
  p.info = reinterpret_cast<int4*>(ws + w.info);
  p.lead = reinterpret_cast<int32_t*>(ws + w.groups);
  p.active = p.lead + call->G;
  p.prefix = p.active + call->G;
  p.first = reinterpret_cast<uint32_t*>(p.prefix + call->G);
  p.piece_o = reinterpret_cast<float*>(ws + w.piece_o);
  p.piece_s = reinterpret_cast<float4*>(ws + w.piece_s);
  a.from = p.from;
  return launched(launch_shared(p, call->stream));
}

}  // extern "C"
