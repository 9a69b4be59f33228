// Instances of the cache attention (cache_attention.cuh) over e4m3 caches.
#include "cache_attention_keys.cuh"

namespace specdec {

cudaError_t launch_cache_attention_kv8(const CacheAttnLaunch& A, int D, const CUtensorMap& tmap_k,
                                       const CUtensorMap& tmap_v, const CUtensorMap& tmap_q,
                                       cudaStream_t stream) {
  if (cache_attn_by_keys(A, D))
    return A.cap > 0.f || A.slopes ? cache_attn::launch_keys<true>(A, tmap_k, tmap_v, stream)
                                   : cache_attn::launch_keys<false>(A, tmap_k, tmap_v, stream);
  switch (D) {
    case 64: return cache_attn::launch_rows<true, 64>(A, tmap_k, tmap_v, tmap_q, stream);
    case 128: return cache_attn::launch_rows<true, 128>(A, tmap_k, tmap_v, tmap_q, stream);
    case 256: return cache_attn::launch_rows<true, 256>(A, tmap_k, tmap_v, tmap_q, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace specdec
