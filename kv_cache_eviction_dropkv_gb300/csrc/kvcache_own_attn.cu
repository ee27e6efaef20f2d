// The second half of a shared attention: each entry's own tokens.
#include "kvcache_attn.cuh"

namespace kvcache {

cudaError_t launch_own_attention(const AttnCall& p, cudaStream_t st) {
  return p.c.code == KVCACHE_INT8 ? launch_code<true, KVCACHE_INT8>(p, st) : launch_code<true, KVCACHE_E4M3>(p, st);
}

}  // namespace kvcache
