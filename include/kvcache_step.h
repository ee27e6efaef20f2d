/*
 * kvcache_step.h -- C ABI of what surrounds the paged 8-bit cache of kvcache.h
 * in a serving step (GB300, sm_103a), served by the same library:
 *   - queries and keys get their per-head norm and their positions, out of the
 *     layer's projection into the layout that attention and scoring read, or,
 *     for tokens that go into the cache, with their keys and values stored in
 *     the same call;
 *   - tokens of the cache are read back as bf16 rows, to be scored again;
 *   - forked sequences attend over the pages they share once for all.
 *
 * Conventions are those of kvcache.h (caller-owned device buffers, 16-byte
 * aligned; asynchronous on `stream`; nothing allocated; status codes and the
 * device status word).  Every call takes one record; fields it has no use for
 * are ignored.  Calls on one cache or one workspace that overlap on the GPU
 * are the caller's to order.
 */
#ifndef KVCACHE_STEP_H
#define KVCACHE_STEP_H

#include "kvcache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Which channels of a head turn together: pair i is (i, i + dims / 2) or
 * (2 i, 2 i + 1). */
#define KVCACHE_HALF        0
#define KVCACHE_INTERLEAVED 1

/* Norm and rotation of a head's d channels x:
 *   y = x / sqrt(mean(x^2) + eps) * weight     where there is a weight, else x
 *   (y_a, y_b) = amplitude (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
 * for the pairs i of the first `dims` channels, with t = 2 pi position
 * turns[i] / 2^64.  The other channels keep y.  A position is any 32-bit
 * number: position * turns[i] modulo 2^64 is the angle without error, so far
 * positions lose nothing.  Sums and products are fp32 (the sine and cosine are
 * off by 2^-23 at most), results are rounded once, to bf16.
 * Supported: d a multiple of 8 in [8, 128]; dims a multiple of 8 in [0, d];
 * eps > 0; both finite. */
typedef struct {
  const uint64_t* turns;   /* device [dims / 2]: turns per position, in units of 2^-64 turn */
  const float* q_norm;     /* device [d], or NULL: queries are not normed */
  const float* k_norm;
  int32_t d, dims, layout;
  float eps, amplitude;
} kvcache_rotary;

/* bf16 rows of d adjacent channels, anywhere: row t of head h of sequence b
 * begins b * seq + h * head + t * row elements after `data`.  data is 16-byte
 * aligned, strides are multiples of 8, from 0 on. */
typedef struct {
  const void* data;
  int64_t seq, head, row;
} kvcache_rows;

/* positions of a call with n sequences of `rows` rows each */
#define KVCACHE_FIRST 0    /* device int32 [n]: row t of sequence i stands at positions[i] + t */
#define KVCACHE_EACH  1    /* device int32 [n][rows] */

/* Norm and rotation of a batch's queries and keys.
 *   q, k          [B][Hq][n][d], [B][Hkv][n][d] as kvcache_rows (data NULL: left out)
 *   q_out, k_out  device bf16 of that shape, densely packed; q_out may be q
 *                 itself where that is densely packed too (k_out k), and
 *                 overlaps nothing else
 *   positions     as position_kind says, or NULL: row t stands at t
 *   lengths       device int32 [B], 0 <= lengths[b] <= n, or NULL for n; rows
 *                 from lengths[b] on are neither read nor written.  A length
 *                 out of range is flagged, and the sequence left out
 * Supported: Hq + Hkv <= 65535; B * n < 2^31. */
typedef struct {
  const kvcache_rotary* rotary;
  kvcache_rows q, k;
  void *q_out, *k_out;
  const int32_t *positions, *lengths;
  uint32_t* status;
  cudaStream_t stream;
  int32_t B, Hq, Hkv, n, position_kind;
} kvcache_rotate_call;
DROPKV_API dropkv_status kvcache_rotate(const kvcache_rotate_call* call);

/* kvcache_store of keys that are normed and turned on the way (the values are
 * stored as they are), and the same tokens' queries: one call for what
 * kvcache_rotate and kvcache_store do in two, with the same results.
 *   q, k, v    [n][Hq][rows][d], [n][Hkv][rows][d] twice, as kvcache_rows
 *              (q.data NULL: no queries)
 *   q_out      device bf16 [n][Hq][rows][d], densely packed, overlapping
 *              neither q, k nor v; rows from counts[i] on are left as they were
 *   positions  as position_kind says, or NULL: a token stands at its place in
 *              its sequence (length - counts[i] + t).  After an eviction
 *              places are no positions: pass them
 *   counts, seqs as in kvcache_store; an entry that is left out there (a
 *              sequence that does not exist or is named twice, a count that
 *              does not fit) gets no queries either
 * The rotary's d is the cache's.  Supported: Hq * rows < 2^30; (rows / page + 2) * 2
 * Hkv + Hq * rows / 16 < 2^31. */
typedef struct {
  const kvcache_shape* shape;
  const kvcache_buffers* cache;
  const kvcache_rotary* rotary;
  kvcache_rows q, k, v;
  void* q_out;
  const int32_t *seqs, *counts, *positions;
  uint32_t* status;
  cudaStream_t stream;
  int32_t layer, n, Hq, rows, position_kind;
} kvcache_rotate_store_call;
DROPKV_API dropkv_status kvcache_rotate_store(const kvcache_rotate_store_call* call);

/* Tokens of one layer as bf16 rows: rows 0 .. counts[i] - 1 of entry i become
 * code * scale of the tokens starts[i] .. starts[i] + counts[i] - 1 of
 * sequence seqs[i], rounded to bf16 (e4m3: exact).
 *   k_out, v_out  device bf16 [n][Hkv][rows][d]; rows from counts[i] on are
 *                 left as they were
 *   starts        device int32 [n], or NULL for 0
 *   counts        device int32 [n], 0 <= counts[i] <= rows, or NULL for all
 *                 tokens from starts[i] on
 * An entry whose sequence does not exist, or whose tokens are not all there or
 * do not fit the rows, is flagged and left out, and so are a bad page's
 * tokens.  A sequence may be named several times. */
typedef struct {
  const kvcache_shape* shape;
  const kvcache_buffers* cache;
  const int32_t *seqs, *starts, *counts;
  void *k_out, *v_out;
  uint32_t* status;
  cudaStream_t stream;
  int32_t layer, n, rows;
} kvcache_read_call;
DROPKV_API dropkv_status kvcache_read(const kvcache_read_call* call);

/* kvcache_attention without a window for entries that come in groups: group j
 * is entries groups[j] .. groups[j + 1] - 1, forks of one sequence or
 * otherwise sequences that begin with the same pages.  The full pages with
 * which the tables of all its sequences begin, up to the token that the first
 * query row of each sees, are read once for the whole group; which these are
 * is found on the device, so the results are kvcache_attention's whatever the
 * groups (up to roundings: sums in another order, probabilities relative to
 * another reference).  Sequences that
 * hold less than a full page before their last T tokens take no part in the
 * sharing.
 *   least   where n * max_pages * page * Hkv * d * 2, the most bytes of keys and
 *           values that kvcache_attention could have to read, is below this,
 *           the call is kvcache_attention and the groups are not looked at
 *           (sharing adds three short kernels); negative: where sharing would
 *           not be faster, by the shape, n, G, Hq and T, if the table were full
 *           of shared tokens (lengths are the device's: short prefixes in a
 *           table for far longer sequences are shared although they need not be)
 *   groups  device int32 [G + 1], groups[0] = 0, not decreasing, groups[G] =
 *           n; anything else is flagged (DROPKV_FLAG_BAD_LENGTH) and nothing
 *           is shared
 * Numerics: kvcache_attention's, for the shared tokens too (their probabilities
 * are off by 2^-11 of themselves, or 2^-32 of the row's largest where that is
 * more; weighted by the scales of their values).  Supported:
 * what kvcache_attention supports with n * Hq * T <= 2^22, 1 <= G <= n and
 * (max_pages * page / 128 + 1) * (n * Hq * T / 128 + G * Hkv) < 2^31. */
typedef struct {
  const kvcache_shape* shape;
  const kvcache_buffers* cache;
  const int32_t *seqs, *groups;
  const void* q;
  void* out;
  void* workspace;
  size_t workspace_bytes;
  uint32_t* status;
  cudaStream_t stream;
  int64_t least;
  int32_t layer, n, Hq, T, G;
} kvcache_shared_attention_call;
DROPKV_API dropkv_status kvcache_shared_attention(const kvcache_shared_attention_call* call);

/* Bytes of device workspace for shared attention calls of at most n entries in
 * at most G groups, with Hq query heads and at most T rows (0: unsupported or
 * invalid, or no device).  No initial contents; keeps nothing. */
DROPKV_API size_t kvcache_shared_workspace_size(const kvcache_shape* shape, int32_t n, int32_t Hq, int32_t T,
                                                int32_t G);

#ifdef __cplusplus
}
#endif
#endif /* KVCACHE_STEP_H */
