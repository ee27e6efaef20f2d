/*
 * kvcache.h -- C ABI of the paged 8-bit KV cache and of the windowed prompt
 * attention (GB300, sm_103a), served by the same library as dropkv.h.
 *
 * What follows an eviction: the kept keys and values are stored in 8 bits, in
 * pages, and every new token attends over them; sequences are forked, copied,
 * evicted again and freed.  And the positional baseline next to the scored
 * ones: a prompt's causal attention over a sliding window with the first
 * tokens kept visible.
 *
 * The cache.  A page holds `page` consecutive tokens of one sequence, for all
 * layers and KV heads.  Codes are K [layers][pages][Hkv][page][d] and V the
 * same, one byte each; the scale of a (layer, page, head) is one float for K
 * and one for V, [layers][pages][Hkv]; a code stands for code * scale:
 *   KVCACHE_E4M3  code = 8-bit float (4 exponent, 3 mantissa bits, largest
 *                 448); the scale is the smallest power of two 2^e with
 *                 max|x| / 2^e <= 448, so that a change of scale moves no
 *                 mantissa bit of a normal code
 *   KVCACHE_INT8  code = integer in [-127, 127]; the scale is max|x| times the
 *                 32-bit reciprocal of 127
 * and never below 2^-120.  Sequence s holds count[s] pages, table[s][0 ..
 * count[s]), length[s] tokens, and count[s] = ceil(length[s] / page).
 * refs[p] counts the sequences that hold page p; 0 means free.  A partly
 * filled page is held by one sequence only (a fork copies it), so a store
 * never changes another sequence.  The calls that take pages take the lowest
 * free ones in order, so their results depend on the state alone.
 *
 * Conventions are those of dropkv.h (caller-owned, 16-byte aligned, densely
 * packed device buffers; asynchronous on `stream`; nothing allocated; status
 * codes and the 32-bit device status word).  The state arrays belong to one
 * stream of calls: calls on one cache that overlap on the GPU are the caller's
 * to order, as are calls that share a workspace.  Every call can be captured
 * into a CUDA graph.
 */
#ifndef KVCACHE_H
#define KVCACHE_H

#include "dropkv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KVCACHE_E4M3 0
#define KVCACHE_INT8 1

/* Bits of the device status word besides those of dropkv.h. */
#define KVCACHE_FLAG_NO_PAGES 0x1000u  /* fewer free pages than wanted: the call changed nothing */
#define KVCACHE_FLAG_BAD_SEQ  0x2000u  /* a sequence number out of range or named twice, a fork's
                                          destination that holds tokens or is a source */
#define KVCACHE_FLAG_BAD_PAGE 0x4000u  /* a table entry that is no page, a page shared where it is
                                          written, a reference count below 1 */
/* Also used: DROPKV_FLAG_BAD_LENGTH (a length, count or number of new tokens
 * that does not fit the sequence), DROPKV_FLAG_BAD_K (a kept count or kept
 * position outside the sequence), DROPKV_FLAG_OVERFLOW (more pages than
 * max_pages), DROPKV_FLAG_NONFINITE (an infinity or not-a-number was stored),
 * DROPKV_FLAG_TIMEOUT. */

/* Shape of a cache.  Supported: layers, Hkv, pages, seqs, max_pages >= 1; d a
 * multiple of 8 in [8, 128]; page 32, 64 or 128; pages <= 2^24;
 * max_pages * page < 2^31; Hkv <= 4096. */
typedef struct {
  int32_t layers;
  int32_t Hkv;
  int32_t d;
  int32_t page;
  int32_t pages;
  int32_t seqs;
  int32_t max_pages;
  int32_t code;      /* KVCACHE_E4M3 or KVCACHE_INT8 */
} kvcache_shape;

/* The cache's device buffers.  All state is the caller's: an empty cache has
 * refs, count and length zero and the table -1. */
typedef struct {
  void* k;           /* uint8 [layers][pages][Hkv][page][d] */
  void* v;
  float* k_scale;    /* [layers][pages][Hkv] */
  float* v_scale;
  int32_t* refs;     /* [pages] */
  int32_t* table;    /* [seqs][max_pages] */
  int32_t* count;    /* [seqs] */
  int32_t* length;   /* [seqs] */
} kvcache_buffers;

/* Bytes of device workspace the calls below need on this cache, for attention
 * calls of at most T query rows of Hq query heads over at most `seqs`
 * sequences (0: invalid or unsupported, or no device).  The workspace needs no
 * initial contents and keeps nothing from call to call. */
DROPKV_API size_t kvcache_workspace_size(const kvcache_shape* shape, int32_t Hq, int32_t T);

/* In all calls `seqs` is a device int32 [n] of sequence numbers, or NULL for
 * 0 .. n - 1 (n <= shape->seqs and <= 65535).  A number out of range is flagged
 * and left out (attention writes zeros for it).  A sequence named twice is
 * flagged and served for its first entry alone by reserve, store, fork (as a
 * destination) and compact; attention serves every entry, and free releases
 * the sequence once. */

/* Make room for extra[i] >= 0 (device int32 [n]) more tokens of sequence
 * seqs[i]: length grows by extra[i], and pages are taken as needed.  All or
 * nothing: with too few free pages nothing changes (FLAG_NO_PAGES).  A
 * sequence whose pages would pass max_pages is flagged and left out.
 *
 * A refusal is known on the device alone until the status word is read, and a
 * kvcache_store of `extra` tokens behind it would replace the last tokens that
 * the sequence has.  So either the status is read first, or the reservation is
 * made by a record (kvcache_run, KVCACHE_RESERVE_GRANTED), whose `out` is a
 * device int32 [n]: it takes what each entry was granted, extra[i] or 0, and
 * goes to kvcache_store as `counts`, which then stores nothing where nothing
 * was granted. */
DROPKV_API dropkv_status kvcache_reserve(const kvcache_shape* shape, const kvcache_buffers* cache,
                                         const int32_t* seqs, int32_t n, const int32_t* extra, void* workspace,
                                         size_t workspace_bytes, uint32_t* status, cudaStream_t stream);

/* Store rows of one layer: the last counts[i] tokens of sequence seqs[i] (its
 * length already holds them) take the codes of rows 0 .. counts[i] - 1.
 *   k, v    device bf16 [n][Hkv][rows][d] (dropkv_compact's k_out and v_out
 *           with out_rows = rows and counts = kept_len, for example)
 *   counts  device int32 [n], 0 <= counts[i] <= rows, or NULL for rows; what
 *           kvcache_reserve granted, where it may have refused (see there)
 * Per (page, head): the scale is that of the new values' largest magnitude;
 * in a page that holds earlier tokens it is the larger of that and the old
 * scale, and when it grows the earlier codes are rounded again at the new
 * scale.  Slots behind the last token are left as they were.  Infinities
 * saturate, not-a-number is stored as such (e4m3) or as 0 (int8); both are
 * flagged and take no part in the scale.  Storing the same tokens again gives
 * the same cache. */
DROPKV_API dropkv_status kvcache_store(const kvcache_shape* shape, const kvcache_buffers* cache, int32_t layer,
                                       const int32_t* seqs, int32_t n, const void* k, const void* v, int32_t rows,
                                       const int32_t* counts, uint32_t* status, cudaStream_t stream);

/* Attention of the last T tokens of each sequence over one layer of the cache
 * (their keys and values are in it): query row t of sequence i stands at
 * position p = length - T + t and sees the tokens j <= p with, when window >
 * 0, j > p - window or j < sinks; out = softmax(q k / sqrt(d)) v, 0 for a row
 * that sees nothing.  Query head h reads KV head h / (Hq / Hkv).
 *   q, out  device bf16 [n][Hq][T][d], must not overlap
 *   window  0 (all tokens; sinks ignored) or >= 1;  sinks >= 0
 * Supported: Hq * T < 2^24; n * Hkv * (max_pages * page / 32 + 3) < 2^31;
 * n * Hq * T < 2^31 with each KV head's rows (Hq / Hkv * T) rounded up to a
 * multiple of 16.
 * Numerics: codes and query rows enter the tensor cores as fp16 (each query
 * row scaled by a power of two first; both exact but for query elements 2^-29
 * below their row's largest), probabilities as fp16 (off by 2^-11 of
 * themselves, or 2^-32 of the row's largest where that is more; weighted by
 * the scales of their values), sums and softmax statistics are fp32.  Queries must be finite and logits within fp32's
 * range; anything else gives its own rows undefined values.  Slots that no row
 * sees are never read.  An e4m3
 * not-a-number code that one row sees makes every row of its KV head
 * not-a-number. */
DROPKV_API dropkv_status kvcache_attention(const kvcache_shape* shape, const kvcache_buffers* cache, int32_t layer,
                                           const int32_t* seqs, int32_t n, const void* q, int32_t Hq, int32_t T,
                                           int32_t window, int32_t sinks, void* out, void* workspace,
                                           size_t workspace_bytes, uint32_t* status, cudaStream_t stream);

/* Sequence dst[i] (empty) becomes a branch of src[i] (device int32 [n] each;
 * a source may be named several times).  share = 1: the full pages are held
 * by both and the partly filled last one is copied; share = 0: every page is
 * copied.  All layers, codes and scales.  All or nothing as kvcache_reserve. */
DROPKV_API dropkv_status kvcache_fork(const kvcache_shape* shape, const kvcache_buffers* cache, const int32_t* src,
                                      const int32_t* dst, int32_t n, int32_t share, void* workspace,
                                      size_t workspace_bytes, uint32_t* status, cudaStream_t stream);

/* Keep kept_len[i] tokens of sequence seqs[i]: token kept_idx[l][i][h][m]
 * becomes token m of layer l and head h.
 *   kept_idx  device int32 [layers][n][Hkv][kept_stride] (dropkv_select's
 *             kept_idx per layer), any positions < length, in any order
 *             (may be NULL when kept_stride is 0)
 *   kept_len  device int32 [n], 0 <= kept_len[i] <= length and kept_stride
 * The kept tokens move to new pages and the old ones are released, so a
 * branch that shares pages is evicted alone; while the call runs both are
 * held (FLAG_NO_PAGES when they do not fit: nothing changes).  A new page's
 * scale is the largest of its tokens' old scales; codes of that scale are
 * copied, the others rounded again at it.  Slots behind the last kept token
 * are left as they were. */
DROPKV_API dropkv_status kvcache_compact(const kvcache_shape* shape, const kvcache_buffers* cache,
                                         const int32_t* seqs, int32_t n, const int32_t* kept_idx,
                                         int32_t kept_stride, const int32_t* kept_len, void* workspace,
                                         size_t workspace_bytes, uint32_t* status, cudaStream_t stream);

/* Release every page of the sequences, which become empty. */
DROPKV_API dropkv_status kvcache_free(const kvcache_shape* shape, const kvcache_buffers* cache, const int32_t* seqs,
                                      int32_t n, uint32_t* status, cudaStream_t stream);

/* A prompt's causal attention over a sliding window with the first tokens
 * kept visible: row i < n_b sees the keys j <= i with j > i - window or j <
 * sinks (window 0: every j <= i).
 *   q, attn_out  device bf16 [B][Hq][n_max][d];  k, v  device bf16
 *                [B][Hkv][n_max][d];  rows >= n_b are neither read into a
 *                result nor written
 *   lengths      device int32 [B], 0 <= n_b <= n_max, or NULL for n_max
 * Values and keys of live rows must be finite (a key tile of 128 tokens
 * enters the tensor cores whole, and 0 times an infinity is not 0).
 * Numerics: probabilities enter the product with V as bf16 (off by 2^-8 of
 * themselves) and are summed unrounded; sums and softmax statistics are fp32.
 * Supported: Hq % Hkv == 0; d a multiple of 8 in [8, 128]; B, Hq <= 65535;
 * n_max <= 2^30; Hq * ceil(n_max / 256) < 2^31. */
DROPKV_API dropkv_status kvcache_window_attention(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int32_t n_max,
                                                  const void* q, const void* k, const void* v,
                                                  const int32_t* lengths, int32_t window, int32_t sinks,
                                                  void* attn_out, uint32_t* status, cudaStream_t stream);

/* One of the cache's calls above as a record, for bindings that pay for every
 * argument they pass: kvcache_run makes the call that `op` names with the
 * fields that stand beside it and ignores the others.
 *   op                 in[0]     in[1]     in[2]   out  arg
 *   KVCACHE_RESERVE    extra
 *   KVCACHE_STORE      k         v         counts       rows
 *   KVCACHE_ATTENTION  q                           out  Hq, T, window, sinks
 *   KVCACHE_FORK       dst                              share    (seqs: src)
 *   KVCACHE_COMPACT    kept_idx  kept_len               kept_stride
 *   KVCACHE_FREE
 *   KVCACHE_RESERVE_GRANTED   extra, and out: granted (kvcache_reserve says
 *                      what for) */
#define KVCACHE_RESERVE   0
#define KVCACHE_STORE     1
#define KVCACHE_ATTENTION 2
#define KVCACHE_FORK      3
#define KVCACHE_COMPACT   4
#define KVCACHE_FREE      5
#define KVCACHE_RESERVE_GRANTED 16
typedef struct {
  const kvcache_shape* shape;
  const kvcache_buffers* cache;
  void* workspace;
  size_t workspace_bytes;
  uint32_t* status;
  cudaStream_t stream;
  const int32_t* seqs;
  const void* in[3];
  void* out;
  int32_t op, layer, n;
  int32_t arg[4];
} kvcache_call;
DROPKV_API dropkv_status kvcache_run(const kvcache_call* call);

/* dropkv_read_status with this header's flags as well (they map to
 * DROPKV_ERR_DEVICE_ARG). */
DROPKV_API dropkv_status kvcache_read_status(const uint32_t* status, cudaStream_t stream, uint32_t* flags_out);

#ifdef __cplusplus
}
#endif
#endif /* KVCACHE_H */
