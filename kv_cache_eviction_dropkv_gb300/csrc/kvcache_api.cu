// Host side of include/kvcache.h: argument checks, the workspace plan and
// launches.  Nothing here allocates device memory.
#include <cmath>

#include "kvcache_internal.cuh"

using namespace kvcache;
using dropkv::current_sms;
using dropkv::ranges_overlap;

namespace {

bool aligned(const void* p, uintptr_t a = 16) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

dropkv_status check_shape(const kvcache_shape* s) {
  if (!s) return DROPKV_ERR_INVALID_ARG;
  if (s->layers < 1 || s->Hkv < 1 || s->d < 1 || s->page < 1 || s->pages < 1 || s->seqs < 1 || s->max_pages < 1 ||
      (s->code != KVCACHE_E4M3 && s->code != KVCACHE_INT8))
    return DROPKV_ERR_INVALID_ARG;
  if (s->d % 8 != 0 || s->d > dropkv::kDPad || (s->page != 32 && s->page != 64 && s->page != 128) ||
      s->pages > kMaxPages || s->Hkv > kMaxHeads || (long long)s->max_pages * s->page >= (1LL << 31))
    return DROPKV_ERR_UNSUPPORTED;
  return DROPKV_OK;
}

// The parts of a call that every entry point checks; fills the kernels' view.
dropkv_status open_cache(const kvcache_shape* s, const kvcache_buffers* b, int32_t layer, int32_t n, uint32_t* status,
                         Cache* c) {
  const dropkv_status st = check_shape(s);
  if (st != DROPKV_OK) return st;
  if (!b || !b->k || !b->v || !b->k_scale || !b->v_scale || !b->refs || !b->table || !b->count || !b->length ||
      !status || layer < 0 || layer >= s->layers || n < 0 || n > s->seqs)
    return DROPKV_ERR_INVALID_ARG;
  if (!aligned(b->k) || !aligned(b->v) || !aligned(b->k_scale) || !aligned(b->v_scale) || !aligned(b->refs) ||
      !aligned(b->table) || !aligned(b->count) || !aligned(b->length) || !aligned(status, 4))
    return DROPKV_ERR_INVALID_ARG;
  if (n > 65535) return DROPKV_ERR_UNSUPPORTED;
  const size_t units = (size_t)s->pages * s->Hkv;
  const size_t bytes = units * s->page * s->d;
  c->k = static_cast<uint8_t*>(b->k) + (size_t)layer * bytes;
  c->v = static_cast<uint8_t*>(b->v) + (size_t)layer * bytes;
  c->ks = b->k_scale + (size_t)layer * units;
  c->vs = b->v_scale + (size_t)layer * units;
  c->refs = b->refs; c->table = b->table; c->count = b->count; c->length = b->length;
  c->layers = s->layers; c->Hkv = s->Hkv; c->d = s->d; c->page = s->page;
  c->P = s->pages; c->S = s->seqs; c->M = s->max_pages;
  c->page_log2 = s->page == 32 ? 5 : s->page == 64 ? 6 : 7;
  c->code = s->code;
  c->status = status;
  return DROPKV_OK;
}

dropkv_status open_pages(const kvcache_shape* s, const kvcache_buffers* b, int32_t n, void* workspace,
                         size_t workspace_bytes, uint32_t* status, PageCall* p) {
  const dropkv_status st = open_cache(s, b, 0, n, status, &p->c);
  if (st != DROPKV_OK) return st;
  const PagePlan w = make_page_plan(s->seqs, s->pages);
  if (!workspace || workspace_bytes < w.total || !aligned(workspace)) return DROPKV_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p->n = n;
  p->claim = reinterpret_cast<int32_t*>(ws + w.claim);
  p->mark = reinterpret_cast<int32_t*>(ws + w.mark);
  p->from = reinterpret_cast<int32_t*>(ws + w.from);
  p->offs = reinterpret_cast<int32_t*>(ws + w.offs);
  p->entry = reinterpret_cast<int4*>(ws + w.entry);
  p->list = reinterpret_cast<int32_t*>(ws + w.list);
  p->rows = reinterpret_cast<int32_t*>(ws + w.rows);
  return DROPKV_OK;
}

dropkv_status launched(cudaError_t e) { return e == cudaSuccess ? DROPKV_OK : DROPKV_ERR_CUDA; }

dropkv_status reserve(const kvcache_shape* shape, const kvcache_buffers* cache, const int32_t* seqs, int32_t n,
                      const int32_t* extra, int32_t* granted, void* workspace, size_t workspace_bytes,
                      uint32_t* status, cudaStream_t stream) {
  PageCall p{};
  const dropkv_status st = open_pages(shape, cache, n, workspace, workspace_bytes, status, &p);
  if (st != DROPKV_OK) return st;
  if (!extra || !aligned(granted, 4)) return DROPKV_ERR_INVALID_ARG;
  if (n == 0) return DROPKV_OK;
  p.seqs = seqs;
  p.extra = extra;
  p.granted = granted;
  return launched(launch_reserve(p, stream));
}

}  // namespace

extern "C" {

size_t kvcache_workspace_size(const kvcache_shape* shape, int32_t Hq, int32_t T) {
  const int sms = current_sms(nullptr);
  if (sms <= 0 || check_shape(shape) != DROPKV_OK || Hq < 1 || T < 1 || Hq % shape->Hkv != 0) return 0;
  // the attention's pieces: at most one run per warp of a wave, at the widest row group
  const size_t pages = make_page_plan(shape->seqs, shape->pages).total;
  return std::max(pages, attn_workspace_bound(*shape, Hq, T, sms));
}

dropkv_status kvcache_reserve(const kvcache_shape* shape, const kvcache_buffers* cache, const int32_t* seqs, int32_t n,
                              const int32_t* extra, void* workspace, size_t workspace_bytes, uint32_t* status,
                              cudaStream_t stream) {
  return reserve(shape, cache, seqs, n, extra, nullptr, workspace, workspace_bytes, status, stream);
}

dropkv_status kvcache_store(const kvcache_shape* shape, const kvcache_buffers* cache, int32_t layer,
                            const int32_t* seqs, int32_t n, const void* k, const void* v, int32_t rows,
                            const int32_t* counts, uint32_t* status, cudaStream_t stream) {
  StoreCall p{};
  const dropkv_status st = open_cache(shape, cache, layer, n, status, &p.c);
  if (st != DROPKV_OK) return st;
  if (!k || !v || !aligned(k) || !aligned(v) || rows < 0) return DROPKV_ERR_INVALID_ARG;
  if (n == 0 || rows == 0) return DROPKV_OK;
  p.seqs = seqs;
  p.n = n;
  p.rows = rows;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.counts = counts;
  return launched(launch_store(p, stream));
}

dropkv_status kvcache_attention(const kvcache_shape* shape, const kvcache_buffers* cache, int32_t layer,
                                const int32_t* seqs, int32_t n, const void* q, int32_t Hq, int32_t T, int32_t window,
                                int32_t sinks, void* out, void* workspace, size_t workspace_bytes, uint32_t* status,
                                cudaStream_t stream) {
  AttnCall p{};
  const dropkv_status st = open_cache(shape, cache, layer, n, status, &p.c);
  if (st != DROPKV_OK) return st;
  if (!q || !out || !aligned(q) || !aligned(out) || Hq < 1 || T < 1 || Hq % shape->Hkv != 0 || window < 0 || sinks < 0)
    return DROPKV_ERR_INVALID_ARG;
  if ((long long)Hq * T >= (1LL << 31) / dropkv::kDPad) return DROPKV_ERR_UNSUPPORTED;
  if (n == 0) return DROPKV_OK;
  const size_t bytes = (size_t)n * Hq * T * shape->d * 2;
  if (ranges_overlap(q, bytes, out, bytes)) return DROPKV_ERR_INVALID_ARG;
  const int sms = current_sms(nullptr);
  if (sms <= 0) return DROPKV_ERR_CUDA;
  AttnPlan a;
  if (!make_attn_plan(*shape, n, Hq, T, window, sinks, sms, &a)) return DROPKV_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < a.total || !aligned(workspace)) return DROPKV_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.seqs = seqs;
  p.n = n; p.Hq = Hq; p.T = T;
  p.g = Hq / shape->Hkv;
  p.R = p.g * T;
  p.RB = a.RB; p.RG = a.RG; p.workers = a.workers; p.solo = a.solo; p.team = a.team; p.by_unit = a.by_unit; p.rowwise = a.rowwise;
  p.window = window;
  p.sinks = sinks;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_s = reinterpret_cast<float4*>(ws + a.part_s);
  p.cuts = reinterpret_cast<int2*>(ws + a.cuts);
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)shape->d));
  return launched(launch_attention(p, stream));
}

dropkv_status kvcache_fork(const kvcache_shape* shape, const kvcache_buffers* cache, const int32_t* src,
                           const int32_t* dst, int32_t n, int32_t share, void* workspace, size_t workspace_bytes,
                           uint32_t* status, cudaStream_t stream) {
  PageCall p{};
  const dropkv_status st = open_pages(shape, cache, n, workspace, workspace_bytes, status, &p);
  if (st != DROPKV_OK) return st;
  if (!src || !dst || (share != 0 && share != 1)) return DROPKV_ERR_INVALID_ARG;
  if (n == 0) return DROPKV_OK;
  p.seqs = src;
  p.other = dst;
  p.share = share;
  return launched(launch_fork(p, current_sms(nullptr), stream));
}

dropkv_status kvcache_compact(const kvcache_shape* shape, const kvcache_buffers* cache, const int32_t* seqs, int32_t n,
                              const int32_t* kept_idx, int32_t kept_stride, const int32_t* kept_len, void* workspace,
                              size_t workspace_bytes, uint32_t* status, cudaStream_t stream) {
  PageCall p{};
  const dropkv_status st = open_pages(shape, cache, n, workspace, workspace_bytes, status, &p);
  if (st != DROPKV_OK) return st;
  if ((!kept_idx && kept_stride > 0) || !kept_len || kept_stride < 0) return DROPKV_ERR_INVALID_ARG;
  if (n == 0) return DROPKV_OK;
  p.seqs = seqs;
  p.kept_idx = kept_idx;
  p.kept_stride = kept_stride;
  p.kept_len = kept_len;
  p.early = (long long)n * shape->max_pages <= kEarlyRows ? 1 : 0;
  return launched(launch_compact_pages(p, current_sms(nullptr), stream));
}

dropkv_status kvcache_free(const kvcache_shape* shape, const kvcache_buffers* cache, const int32_t* seqs, int32_t n,
                           uint32_t* status, cudaStream_t stream) {
  PageCall p{};
  const dropkv_status st = open_cache(shape, cache, 0, n, status, &p.c);
  if (st != DROPKV_OK) return st;
  if (n == 0) return DROPKV_OK;
  p.seqs = seqs;
  p.n = n;
  return launched(launch_free(p, stream));
}

dropkv_status kvcache_window_attention(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int32_t n_max, const void* q,
                                       const void* k, const void* v, const int32_t* lengths, int32_t window,
                                       int32_t sinks, void* attn_out, uint32_t* status, cudaStream_t stream) {
  if (B < 1 || Hq < 1 || Hkv < 1 || d < 1 || n_max < 1 || Hq % Hkv != 0 || window < 0 || sinks < 0)
    return DROPKV_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > dropkv::kDPad || B > 65535 || Hq > 65535 || n_max > (1 << 30) ||
      (long long)B * Hq >= (1LL << 31) || ((long long)n_max + 255) / 256 * Hq >= (1LL << 31))
    return DROPKV_ERR_UNSUPPORTED;
  if (!q || !k || !v || !attn_out || !status || !aligned(q) || !aligned(k) || !aligned(v) || !aligned(attn_out) ||
      !aligned(status, 4))
    return DROPKV_ERR_INVALID_ARG;
  const size_t row = (size_t)n_max * d * 2, q_bytes = (size_t)B * Hq * row, kv_bytes = (size_t)B * Hkv * row;
  if (ranges_overlap(attn_out, q_bytes, q, q_bytes) || ranges_overlap(attn_out, q_bytes, k, kv_bytes) ||
      ranges_overlap(attn_out, q_bytes, v, kv_bytes))
    return DROPKV_ERR_INVALID_ARG;
  const int sms = current_sms(nullptr);
  if (sms <= 0) return DROPKV_ERR_CUDA;
  CUtensorMap tq, tk, tv;
  if (!dropkv::encode_rows(&tq, q, d, n_max, B * Hq) || !dropkv::encode_rows(&tk, k, d, n_max, B * Hkv) ||
      !dropkv::encode_rows(&tv, v, d, n_max, B * Hkv))
    return DROPKV_ERR_CUDA;
  WindowCall p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(attn_out);
  p.lengths = lengths;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.g = Hq / Hkv; p.d = d; p.n_max = n_max;
  p.window = std::min(window, n_max);      // the same rows, and positions stay in 32 bits
  p.sinks = std::min(sinks, n_max);
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)d));
  p.status = status;
  return launched(launch_window(p, tq, tk, tv, sms, stream));
}

dropkv_status kvcache_run(const kvcache_call* c) {
  if (!c) return DROPKV_ERR_INVALID_ARG;
  const int32_t* in0 = static_cast<const int32_t*>(c->in[0]);
  switch (c->op) {
    case KVCACHE_RESERVE:
      return kvcache_reserve(c->shape, c->cache, c->seqs, c->n, in0, c->workspace, c->workspace_bytes, c->status,
                             c->stream);
    case KVCACHE_RESERVE_GRANTED:
      if (!c->out) return DROPKV_ERR_INVALID_ARG;
      return reserve(c->shape, c->cache, c->seqs, c->n, in0, static_cast<int32_t*>(c->out), c->workspace,
                     c->workspace_bytes, c->status, c->stream);
    case KVCACHE_STORE:
      return kvcache_store(c->shape, c->cache, c->layer, c->seqs, c->n, c->in[0], c->in[1], c->arg[0],
                           static_cast<const int32_t*>(c->in[2]), c->status, c->stream);
    case KVCACHE_ATTENTION:
      return kvcache_attention(c->shape, c->cache, c->layer, c->seqs, c->n, c->in[0], c->arg[0], c->arg[1], c->arg[2],
                               c->arg[3], c->out, c->workspace, c->workspace_bytes, c->status, c->stream);
    case KVCACHE_FORK:
      return kvcache_fork(c->shape, c->cache, c->seqs, in0, c->n, c->arg[0], c->workspace, c->workspace_bytes,
                          c->status, c->stream);
    case KVCACHE_COMPACT:
      return kvcache_compact(c->shape, c->cache, c->seqs, c->n, in0, c->arg[0],
                             static_cast<const int32_t*>(c->in[1]), c->workspace, c->workspace_bytes, c->status,
                             c->stream);
    case KVCACHE_FREE:
      return kvcache_free(c->shape, c->cache, c->seqs, c->n, c->status, c->stream);
    default: return DROPKV_ERR_INVALID_ARG;
  }
}

dropkv_status kvcache_read_status(const uint32_t* status, cudaStream_t stream, uint32_t* flags_out) {
  uint32_t f = 0;
  const dropkv_status st = dropkv_read_status(status, stream, &f);
  if (flags_out) *flags_out = f;
  if (st != DROPKV_OK) return st;
  if (f & (KVCACHE_FLAG_NO_PAGES | KVCACHE_FLAG_BAD_SEQ | KVCACHE_FLAG_BAD_PAGE)) return DROPKV_ERR_DEVICE_ARG;
  return DROPKV_OK;
}

}  // extern "C"
