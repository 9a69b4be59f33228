// Instances of the cache attention (cache_attention.cuh) over bf16 caches.
#include "cache_attention.cuh"

namespace specdec {

cudaError_t launch_cache_attention_bf16(const CacheAttnLaunch& A, int D, const CUtensorMap& tmap_k,
                                        const CUtensorMap& tmap_v, const CUtensorMap& tmap_q,
                                        cudaStream_t stream) {
  switch (D) {
    case 64: return cache_attn::launch_rows<false, 64>(A, tmap_k, tmap_v, tmap_q, stream);
    case 128: return cache_attn::launch_rows<false, 128>(A, tmap_k, tmap_v, tmap_q, stream);
    case 256: return cache_attn::launch_rows<false, 256>(A, tmap_k, tmap_v, tmap_q, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace specdec
