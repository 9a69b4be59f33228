// C ABI of the 8-bit cache and of the attention with caps, biases, windows
// and trees: argument checks, workspace plan, tensor maps and launches.
#include <cmath>

#include "kernels.h"

using namespace specdec;

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool head_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

int check_shape(int B, int n_new, int Hq, int Hkv, int D, int Lmax) {
  if (B < 0 || n_new < 1 || n_new > SPECDEC_MAX_TREE_NODES || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 ||
      !head_dim_ok(D) || Lmax < n_new || Lmax > (1 << 30))
    return SPECDEC_ERR_UNSUPPORTED;
  if (Hq / Hkv > 128 || Hq > (1 << 20)) return SPECDEC_ERR_UNSUPPORTED;
  if ((__int128)B * Lmax * Hkv * D >= ((__int128)1 << 40)) return SPECDEC_ERR_UNSUPPORTED;
  // (sequence, KV head, row group) tiles and their blocks of 64 keys or more
  // are counted in 32 bits
  if ((long long)B * Hq * n_new >= (1ll << 31)) return SPECDEC_ERR_UNSUPPORTED;
  if ((__int128)B * Hkv * n_new * (Lmax / 64 + 8) >= ((__int128)1 << 31)) return SPECDEC_ERR_UNSUPPORTED;
  return SPECDEC_OK;
}

struct AttnPlan {
  int n_groups, group_pos;
  size_t off_notes, off_ml, off_o, total;
};

// The new positions in equal groups of at most 128 query rows per KV head;
// the partials of the tiles that the CTAs share, two per CTA, whatever the
// batch and the lengths.
AttnPlan make_plan(bool e4m3, int n_new, int G, int D) {
  AttnPlan p;
  const int most = 128 / G;
  p.n_groups = (n_new + most - 1) / most;
  p.group_pos = (n_new + p.n_groups - 1) / p.n_groups;
  p.n_groups = (n_new + p.group_pos - 1) / p.group_pos;
  size_t off = align_up(sizeof(WsHeader));
  const int ctas = cache_attn_can_key(e4m3, D, p.group_pos * G) ? kCacheAttnMaxCtas : kCacheAttnCtas;
  const size_t rows = (size_t)2 * ctas * cache_attn_rows(p.group_pos * G);
  p.off_notes = off;
  off = align_up(off + ctas * sizeof(int4));
  p.off_ml = off;
  off = align_up(off + rows * 2 * sizeof(float));
  p.off_o = off;
  off = align_up(off + rows * D * sizeof(float));
  p.total = off;
  return p;
}

// The cache as a 4-D tensor {D, Hkv, Lmax, B}; box: up to 128 bytes of a row
// x one head x one block of rows, swizzled.
bool encode_cache(CUtensorMap* map, const void* base, bool e4m3, int B, int Lmax, int Hkv, int D, int block) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t es = e4m3 ? 1 : 2, row = (cuuint64_t)D * es;
  const cuuint32_t panel = row < 128 ? (cuuint32_t)row : 128u;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)Lmax, (cuuint64_t)B};
  const cuuint64_t strides[3] = {row, row * Hkv, row * Hkv * Lmax};
  const cuuint32_t box[4] = {panel / (cuuint32_t)es, 1, (cuuint32_t)block, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            panel == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            panel == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as a 4-D tensor {D, Hq, n_new, B}; box: 64 dims of a group's
// rows of one KV head, positions past n_new read as zeros.
bool encode_queries(CUtensorMap* map, const void* q, long long q_stride, int B, int n_new, int Hq, int G, int D,
                    int group_pos) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)n_new, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)q_stride * 2, (cuuint64_t)q_stride * 2 * n_new};
  const cuuint32_t box[4] = {64, (cuuint32_t)G, (cuuint32_t)group_pos, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int attention(bool e4m3, const void* q, long long q_stride, const void* k_cache, const void* v_cache,
              const float* k_scale, const float* v_scale, const int32_t* seq_lens, const int32_t* parent,
              const float* slopes, int B, int n_new, int Hq, int Hkv, int D, int Lmax, float scale,
              float softcap, int window, void* out, void* workspace, size_t workspace_bytes,
              void* stream_ptr) {
  int rc = check_shape(B, n_new, Hq, Hkv, D, Lmax);
  if (rc != SPECDEC_OK) return rc;
  if (B == 0) return SPECDEC_OK;
  if (!q || !k_cache || !v_cache || !seq_lens || !out) return SPECDEC_ERR_INVALID_ARG;
  if (e4m3 && (!k_scale || !v_scale)) return SPECDEC_ERR_INVALID_ARG;
  if ((((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out) & 15u) != 0)
    return SPECDEC_ERR_INVALID_ARG;
  if (((((uintptr_t)k_scale | (uintptr_t)v_scale | (uintptr_t)slopes | (uintptr_t)seq_lens)) & 3u) != 0)
    return SPECDEC_ERR_INVALID_ARG;
  if (q_stride < (long long)Hq * D || q_stride % 8 != 0 || q_stride >= (1ll << 31)) return SPECDEC_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0)
    return SPECDEC_ERR_INVALID_ARG;
  // its reciprocal is used, and the tanh rounds to 2^-22 of it
  if (softcap > 0.f && (softcap < 1e-30f || softcap > 1000.f)) return SPECDEC_ERR_INVALID_ARG;
  // factors of the scores stay normal numbers, and a score of 0 stays 0
  if (scale > 0.f && (scale < 1e-30f || scale > 1e30f)) return SPECDEC_ERR_INVALID_ARG;
  CacheAttnLaunch A;
  A.tree = parent != nullptr;
  A.max_depth = n_new - 1;
  if (parent) {
    if (parent[0] != -1) return SPECDEC_ERR_INVALID_ARG;
    for (int w = 0; w < 4; ++w) A.anc[0][w] = w == 0 ? 1u : 0u;
    A.depth[0] = 0;
    A.max_depth = 0;
    for (int i = 1; i < n_new; ++i) {
      const int p = parent[i];
      if (p < 0 || p >= i) return SPECDEC_ERR_INVALID_ARG;
      for (int w = 0; w < 4; ++w) A.anc[i][w] = A.anc[p][w];
      A.anc[i][i >> 5] |= 1u << (i & 31);
      A.depth[i] = (uint8_t)(A.depth[p] + 1);
      if (A.depth[i] > A.max_depth) A.max_depth = A.depth[i];
    }
  }
  const int G = Hq / Hkv;
  const AttnPlan pl = make_plan(e4m3, n_new, G, D);
  if (!workspace || ((uintptr_t)workspace % kAlign) != 0 || workspace_bytes < pl.total)
    return SPECDEC_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  A.B = B;
  A.n_new = n_new;
  A.Hq = Hq;
  A.Hkv = Hkv;
  A.G = G;
  A.Lmax = Lmax;
  A.n_groups = pl.n_groups;
  A.group_pos = pl.group_pos;
  A.window = window < Lmax ? window : 0;      // no distance reaches Lmax, and the kernels' differences stay in 32 bits
  // at least two parts per head: with more heads than that, a CTA takes them all in turn
  A.head_lanes = 2 * Hkv <= kCacheAttnCtas ? Hkv : 1;
  A.note_tiles = 0;                          // the launch decides
  A.n_scale = (Lmax + SPECDEC_KV8_BLOCK - 1) / SPECDEC_KV8_BLOCK;
  A.scale = scale > 0.f ? scale : 1.f / std::sqrt((float)D);
  A.cap = softcap;
  A.cap_exp = softcap > 0.f ? 2.f * kLog2e / softcap : 0.f;
  A.q_stride = q_stride;
  A.q = static_cast<const __nv_bfloat16*>(q);
  A.v = v_cache;
  A.k_scale = k_scale;
  A.v_scale = v_scale;
  A.slopes = slopes;
  A.seq_lens = seq_lens;
  A.out = static_cast<__nv_bfloat16*>(out);
  A.part_ml = reinterpret_cast<float*>(ws + pl.off_ml);
  A.part_o = reinterpret_cast<float*>(ws + pl.off_o);
  A.notes = reinterpret_cast<int4*>(ws + pl.off_notes);
  A.status = reinterpret_cast<int*>(ws);
  CUtensorMap tk, tv, tq;
  const int block = cache_attn_block(D, cache_attn_rows(pl.group_pos * G));
  if (!encode_cache(&tk, k_cache, e4m3, B, Lmax, Hkv, D, block) ||
      !encode_cache(&tv, v_cache, e4m3, B, Lmax, Hkv, D, block))
    return SPECDEC_ERR_CUDA;
  if (e4m3)
    tq = tk;                                   // not read: the kernel converts the queries itself
  else if (!encode_queries(&tq, q, q_stride, B, n_new, Hq, G, D, pl.group_pos))
    return SPECDEC_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const cudaError_t e = e4m3 ? launch_cache_attention_kv8(A, D, tk, tv, tq, stream)
                             : launch_cache_attention_bf16(A, D, tk, tv, tq, stream);
  return e == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t specdec_kv8_append_workspace_size(void) { return align_up(sizeof(WsHeader)); }

int specdec_kv8_append(const void* k_new, long long k_stride, const void* v_new, long long v_stride,
                       const int32_t* start, const int32_t* counts, const int32_t* rows, int B, int n,
                       int Hkv, int D, int Lmax, void* k_cache, void* v_cache, float* k_scale,
                       float* v_scale, void* workspace, size_t workspace_bytes, void* stream_ptr) {
  if (B < 0 || n < 1 || Hkv < 1 || !head_dim_ok(D) || Lmax < 1 || Lmax > (1 << 30))
    return SPECDEC_ERR_UNSUPPORTED;
  if ((__int128)B * Lmax * Hkv * D >= ((__int128)1 << 40)) return SPECDEC_ERR_UNSUPPORTED;
  const long long max_blocks = ((long long)n + SPECDEC_KV8_BLOCK - 2) / SPECDEC_KV8_BLOCK + 1;
  if ((__int128)B * Hkv * (n / SPECDEC_KV8_BLOCK + 2) >= ((__int128)1 << 31)) return SPECDEC_ERR_UNSUPPORTED;
  if (B == 0) return SPECDEC_OK;
  if (!k_new || !v_new || !start || !k_cache || !v_cache || !k_scale || !v_scale)
    return SPECDEC_ERR_INVALID_ARG;
  if ((((uintptr_t)k_new | (uintptr_t)v_new | (uintptr_t)k_cache | (uintptr_t)v_cache) & 15u) != 0)
    return SPECDEC_ERR_INVALID_ARG;
  if ((((uintptr_t)k_scale | (uintptr_t)v_scale | (uintptr_t)start | (uintptr_t)counts |
        (uintptr_t)rows) & 3u) != 0)
    return SPECDEC_ERR_INVALID_ARG;
  const long long row = (long long)Hkv * D;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return SPECDEC_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace % kAlign) != 0 ||
      workspace_bytes < specdec_kv8_append_workspace_size())
    return SPECDEC_ERR_WORKSPACE;
  Kv8AppendLaunch A;
  A.B = B;
  A.n = n;
  A.Hkv = Hkv;
  A.D = D;
  A.Lmax = Lmax;
  A.n_scale = (Lmax + SPECDEC_KV8_BLOCK - 1) / SPECDEC_KV8_BLOCK;
  A.max_blocks = (int)max_blocks;
  A.src[0] = static_cast<const __nv_bfloat16*>(k_new);
  A.src[1] = static_cast<const __nv_bfloat16*>(v_new);
  A.stride[0] = k_stride;
  A.stride[1] = v_stride;
  A.cache[0] = static_cast<uint8_t*>(k_cache);
  A.cache[1] = static_cast<uint8_t*>(v_cache);
  A.scale[0] = k_scale;
  A.scale[1] = v_scale;
  A.start = start;
  A.counts = counts;
  A.rows = rows;
  A.status = reinterpret_cast<int*>(workspace);
  return launch_kv8_append(A, static_cast<cudaStream_t>(stream_ptr)) == cudaSuccess ? SPECDEC_OK
                                                                                    : SPECDEC_ERR_CUDA;
}

size_t specdec_verify_attention_kv8_workspace_size(int B, int n_new, int Hq, int Hkv, int D, int Lmax) {
  if (check_shape(B, n_new, Hq, Hkv, D, Lmax) != SPECDEC_OK) return 0;
  return make_plan(true, n_new, Hq / Hkv, D).total;
}

int specdec_verify_attention_kv8(const void* q, long long q_stride, const void* k_cache, const void* v_cache,
                                 const float* k_scale, const float* v_scale, const int32_t* seq_lens,
                                 const int32_t* parent, const float* slopes, int B, int n_new, int Hq,
                                 int Hkv, int D, int Lmax, float scale, float softcap, int window, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  return attention(true, q, q_stride, k_cache, v_cache, k_scale, v_scale, seq_lens, parent, slopes, B, n_new,
                   Hq, Hkv, D, Lmax, scale, softcap, window, out, workspace, workspace_bytes, stream);
}

size_t specdec_verify_attention_masked_workspace_size(int B, int n_new, int Hq, int Hkv, int D, int Lmax) {
  if (check_shape(B, n_new, Hq, Hkv, D, Lmax) != SPECDEC_OK) return 0;
  return make_plan(false, n_new, Hq / Hkv, D).total;
}

int specdec_verify_attention_masked(const void* q, long long q_stride, const void* k_cache,
                                    const void* v_cache, const int32_t* seq_lens, const int32_t* parent,
                                    const float* slopes, int B, int n_new, int Hq, int Hkv, int D, int Lmax,
                                    float scale, float softcap, int window, void* out, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  return attention(false, q, q_stride, k_cache, v_cache, nullptr, nullptr, seq_lens, parent, slopes, B, n_new,
                   Hq, Hkv, D, Lmax, scale, softcap, window, out, workspace, workspace_bytes, stream);
}

}  // extern "C"
