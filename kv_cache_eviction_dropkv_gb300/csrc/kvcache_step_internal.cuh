// Internal declarations of what surrounds the cache in a step
// (include/kvcache_step.h): parameter blocks and launchers.
#pragma once
#include "../../include/kvcache_step.h"
#include "kvcache_internal.cuh"

namespace kvcache {

constexpr long long kMaxSharedRows = 1 << 22;   // query rows of a shared attention call

struct Rows {
  const __nv_bfloat16* p;        // null: left out
  long long seq, head, row;      // strides in elements
};
struct Turning {
  const unsigned long long* turns;   // [dims / 2], 2^-64 turns per position
  int d, dims, half;             // half: pair i is (i, i + dims / 2), else (2 i, 2 i + 1)
  float eps, amplitude, inv_d;
};

struct RotateCall {
  Turning how;
  Rows in[2];                    // queries, keys
  __nv_bfloat16* out[2];
  const float* weight[2];
  int heads[2];
  const int32_t *positions, *lengths;
  int each;                      // 1: a position per row
  int B, n;
  int chunk, chunks;             // heads a CTA takes; CTAs that take the queries' heads
  uint32_t* status;
};
cudaError_t launch_rotate(RotateCall p, int sms, cudaStream_t st);

struct RotateStoreCall {
  Cache c;                       // k, v, ks, vs at the layer
  Turning how;
  Rows q, kv[2];
  __nv_bfloat16* q_out;
  const float *q_weight, *k_weight;
  const int32_t *seqs, *counts, *positions;
  int each;
  int n, Hq, rows;
  int touched;                   // pages that `rows` tokens touch at most
  int q_chunk, kv_heads;         // query heads of one token that its lanes take, KV heads of a page that a CTA takes
};
cudaError_t launch_rotate_store(RotateStoreCall p, cudaStream_t st);

struct ReadCall {
  Cache c;                       // k, v, ks, vs at the layer
  const int32_t *seqs, *starts, *counts;
  __nv_bfloat16 *k, *v;
  int n, rows;
};
cudaError_t launch_read(const ReadCall& p, cudaStream_t st);

// A shared attention: what its plan kernel finds out, for the kernels behind it.
struct SharedPlan {
  uint32_t total, runs;          // tiles of all shared parts; runs that they are dealt to
  int unit_rows;                 // rows of a unit: 128 where no group has more per KV head, else 256
};
struct SharedCall {
  AttnCall own;                  // the second half (from, own_o, own_s, parts, cuts)
  int by_runs;                   // 1: it is dealt to runs, and cuts say which units they cut
  const int32_t* groups;
  int G, sms;
  SharedPlan* plan;
  int32_t *from, *group, *bound; // per entry: first token of its own, group, full pages before its last T tokens
  int32_t *lead, *active, *prefix;   // per group: first entry that takes part, how many do, shared pages
  int4* info;                    // per entry: shared tokens, first entry and rows per KV head of its group, its first tile
  uint32_t* first;               // [G + 1] per group: tiles before it
  float* piece_o;                // [sms * 256 + 2 n Hq T][d]
  float4* piece_s;
};
cudaError_t launch_shared(const SharedCall& p, cudaStream_t st);

}  // namespace kvcache
