// C ABI of the attention over packed prompts: argument checks, workspace plan,
// tensor maps and launch.
#include <cmath>

#include "kernels.h"

using namespace specdec;

namespace {

constexpr size_t kAlign = 256;

int check_shape(int B, int T, int Hq, int Hkv, int D) {
  if (B < 0 || T < 0 || T > (1 << 30) || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq / Hkv > 128 || Hq > (1 << 20) ||
      (D != 64 && D != 128 && D != 256))
    return SPECDEC_ERR_UNSUPPORTED;
  if ((__int128)T * Hq * D >= ((__int128)1 << 40)) return SPECDEC_ERR_UNSUPPORTED;
  // (item, KV head) pairs are counted in 32 bits
  const long long items = T / (prompt_tiles(D) * (128 / (Hq / Hkv))) + (long long)B;
  if (items * Hkv >= (1ll << 31) - 4096) return SPECDEC_ERR_UNSUPPORTED;
  return SPECDEC_OK;
}

struct PromptPlan {
  int tile_tokens;
  long long max_items;
  size_t off_items, total;
};

// A sequence's last item may be partly filled: one more for each.
PromptPlan make_plan(int B, int T, int G, int D) {
  PromptPlan p;
  p.tile_tokens = 128 / G;
  p.max_items = T / (prompt_tiles(D) * p.tile_tokens) + (long long)B;
  p.off_items = 2 * kAlign;
  p.total = (p.off_items + p.max_items * sizeof(int4) + kAlign - 1) / kAlign * kAlign;
  return p;
}

// Rows of H heads as a 3-D tensor {D, H, T}; box: 64 dims x `heads` x `rows`.
bool encode_rows(CUtensorMap* map, const void* base, long long stride, int T, int H, int D, int heads, int rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool stride_ok(long long stride, long long row) {
  return stride >= row && stride % 8 == 0 && stride < (1ll << 31);
}

}  // namespace

extern "C" {

size_t specdec_prompt_attention_workspace_size(int B, int T, int Hq, int Hkv, int D) {
  if (check_shape(B, T, Hq, Hkv, D) != SPECDEC_OK) return 0;
  return make_plan(B, T, Hq / Hkv, D).total;
}

int specdec_prompt_attention(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                             long long v_stride, const int32_t* cu_seqlens, const float* slopes, int B, int T, int Hq,
                             int Hkv, int D, float scale, float softcap, int window, void* out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const int rc = check_shape(B, T, Hq, Hkv, D);
  if (rc != SPECDEC_OK) return rc;
  if (B == 0 || T == 0) return SPECDEC_OK;
  if (!q || !k || !v || !cu_seqlens || !out) return SPECDEC_ERR_INVALID_ARG;
  if ((((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)out) & 15u) != 0) return SPECDEC_ERR_INVALID_ARG;
  if ((((uintptr_t)slopes | (uintptr_t)cu_seqlens) & 3u) != 0) return SPECDEC_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, (long long)Hq * D) || !stride_ok(k_stride, (long long)Hkv * D) ||
      !stride_ok(v_stride, (long long)Hkv * D))
    return SPECDEC_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0) return SPECDEC_ERR_INVALID_ARG;
  // its reciprocal is used, and the tanh rounds to 2^-22 of it
  if (softcap > 0.f && (softcap < 1e-30f || softcap > 1000.f)) return SPECDEC_ERR_INVALID_ARG;
  // factors of the scores stay normal numbers, and a score of 0 stays 0
  if (scale > 0.f && (scale < 1e-30f || scale > 1e30f)) return SPECDEC_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  const PromptPlan pl = make_plan(B, T, G, D);
  if (!workspace || (uintptr_t)workspace % kAlign != 0 || workspace_bytes < pl.total) return SPECDEC_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  PromptLaunch A;
  A.B = B;
  A.T = T;
  A.Hq = Hq;
  A.Hkv = Hkv;
  A.G = G;
  A.tile_tokens = pl.tile_tokens;
  A.window = window < T ? window : 0;        // no distance reaches T
  A.cost_shift = 0;
  while ((T / prompt_block(D) + 1) >> A.cost_shift >= 1024) ++A.cost_shift;
  A.max_items = pl.max_items;
  A.v_stride = v_stride;
  A.scale = scale > 0.f ? scale : 1.f / std::sqrt((float)D);
  A.cap = softcap;
  A.cap_exp = cap_factor(softcap, A.scale);
  A.slopes = slopes;
  A.cu_seqlens = cu_seqlens;
  A.v = static_cast<const uint16_t*>(v);
  A.out = static_cast<__nv_bfloat16*>(out);
  // No list where a CTA has two items at most and a warp finds them in a few
  // steps: 33 short prompts (36 items x 4 KV heads, 64 dims) 9.5 -> 8.6 us.
  const bool list = pl.max_items * Hkv > 2 * kCacheAttnCtas || B > 256;
  A.items = list ? reinterpret_cast<int4*>(ws + pl.off_items) : nullptr;
  A.n_items = reinterpret_cast<int*>(ws + kAlign);
  A.next = A.n_items + 1;
  A.status = reinterpret_cast<int*>(ws);
  CUtensorMap tq, tk, tv;
  const int block = prompt_block(D);
  if (!encode_rows(&tq, q, q_stride, T, Hq, D, G, pl.tile_tokens) ||
      !encode_rows(&tk, k, k_stride, T, Hkv, D, 1, block) || !encode_rows(&tv, v, v_stride, T, Hkv, D, 1, block))
    return SPECDEC_ERR_CUDA;
  return launch_prompt_attention(A, D, tq, tk, tv, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SPECDEC_OK
             : SPECDEC_ERR_CUDA;
}

}  // extern "C"
