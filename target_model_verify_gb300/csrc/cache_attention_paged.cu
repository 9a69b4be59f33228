// Instances of the cache attention (cache_attention.cuh) over paged bf16 caches.
#include "cache_attention.cuh"

namespace specdec {

cudaError_t launch_cache_attention_paged(const CacheAttnLaunch& A, int D, const CUtensorMap& tmap_k,
                                         const CUtensorMap& tmap_v, const CUtensorMap& tmap_q,
                                         cudaStream_t stream) {
  switch (D) {
    case 64: return cache_attn::launch_rows<false, 64, true>(A, tmap_k, tmap_v, tmap_q, stream);
    case 128: return cache_attn::launch_rows<false, 128, true>(A, tmap_k, tmap_v, tmap_q, stream);
    case 256: return cache_attn::launch_rows<false, 256, true>(A, tmap_k, tmap_v, tmap_q, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace specdec
