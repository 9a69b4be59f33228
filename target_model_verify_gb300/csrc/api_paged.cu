// C ABI of the paged cache's tables and rows: argument checks and launches.
// (Its attention: api_cache.cu.)
#include "kernels.h"

using namespace specdec;

namespace {

constexpr size_t kAlign = 256;

bool workspace_ok(const void* workspace, size_t bytes) {
  return workspace && (uintptr_t)workspace % kAlign == 0 && bytes >= sizeof(WsHeader);
}

}  // namespace

extern "C" {

size_t specdec_plan_pages_workspace_size(void) { return sizeof(WsHeader); }

int specdec_plan_pages(int32_t* table, int32_t* held, int32_t* free_pages, int32_t* n_free, const int32_t* start,
                       const int32_t* counts, const int32_t* cu_rows, int B, int max_pages, int n_pages, int page,
                       int n, long long n_slots, int32_t* slots, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (B < 0 || max_pages < 1 || n_pages < 1 || page_log2(page) < 0 || (long long)max_pages * page > (1 << 30) ||
      (long long)n_pages * page > (1 << 30))
    return SPECDEC_ERR_UNSUPPORTED;
  if (slots) {
    if (n_slots < 0 || n_slots >= (1ll << 31) - 4) return SPECDEC_ERR_UNSUPPORTED;
    if (!cu_rows && (n < 0 || (long long)B * n != n_slots)) return SPECDEC_ERR_INVALID_ARG;
  } else if (cu_rows) {
    return SPECDEC_ERR_INVALID_ARG;      // they say where a map's rows are
  }
  if (B == 0 && (!slots || n_slots == 0)) return SPECDEC_OK;
  if (!free_pages || !n_free || (B > 0 && (!table || !held || !start || !counts))) return SPECDEC_ERR_INVALID_ARG;
  if ((((uintptr_t)table | (uintptr_t)held | (uintptr_t)free_pages | (uintptr_t)n_free | (uintptr_t)start |
        (uintptr_t)counts | (uintptr_t)cu_rows | (uintptr_t)slots) & 3u) != 0)
    return SPECDEC_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes)) return SPECDEC_ERR_WORKSPACE;
  PagePlanLaunch A;
  A.B = B;
  A.max_pages = max_pages;
  A.n_pages = n_pages;
  A.page_log2 = page_log2(page);
  A.n = n;
  A.n_slots = slots ? n_slots : 0;
  A.table = table;
  A.held = held;
  A.free_pages = free_pages;
  A.n_free = n_free;
  A.start = start;
  A.counts = counts;
  A.cu_rows = cu_rows;
  A.slots = slots;
  A.status = static_cast<int*>(workspace);
  return launch_page_plan(A, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

size_t specdec_paged_append_workspace_size(void) { return sizeof(WsHeader); }

int specdec_paged_append(const void* k_new, long long k_stride, const void* v_new, long long v_stride,
                         const int32_t* slots, const int32_t* rows, int B, int n, int Hkv, int D, int n_pages,
                         int page, void* k_pages, void* v_pages, void* workspace, size_t workspace_bytes,
                         void* stream) {
  if (B < 0 || n < 0 || Hkv < 1 || Hkv > (1 << 20) || (D != 64 && D != 128 && D != 256) || page_log2(page) < 0 ||
      n_pages < 1 || (long long)n_pages * page > (1 << 30))
    return SPECDEC_ERR_UNSUPPORTED;
  if ((__int128)n_pages * page * Hkv * D >= ((__int128)1 << 40)) return SPECDEC_ERR_UNSUPPORTED;
  if ((long long)B * n >= (1ll << 31)) return SPECDEC_ERR_UNSUPPORTED;
  if (B == 0 || n == 0) return SPECDEC_OK;
  if (!k_new || !v_new || !slots || !k_pages || !v_pages) return SPECDEC_ERR_INVALID_ARG;
  if ((((uintptr_t)k_new | (uintptr_t)v_new | (uintptr_t)k_pages | (uintptr_t)v_pages) & 15u) != 0)
    return SPECDEC_ERR_INVALID_ARG;
  if ((((uintptr_t)slots | (uintptr_t)rows) & 3u) != 0) return SPECDEC_ERR_INVALID_ARG;
  const long long row = (long long)Hkv * D;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0 || k_stride >= (1ll << 31) ||
      v_stride >= (1ll << 31))
    return SPECDEC_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes)) return SPECDEC_ERR_WORKSPACE;
  PagedAppendLaunch A;
  A.rows_total = (long long)B * n;
  A.n = n;
  A.row_chunks = (int)(row / 8);
  A.pool_rows = (long long)n_pages * page;
  A.src[0] = static_cast<const uint4*>(k_new);
  A.src[1] = static_cast<const uint4*>(v_new);
  A.stride[0] = k_stride / 8;
  A.stride[1] = v_stride / 8;
  A.pages[0] = static_cast<uint4*>(k_pages);
  A.pages[1] = static_cast<uint4*>(v_pages);
  A.slots = slots;
  A.rows = rows;
  A.status = static_cast<int*>(workspace);
  return launch_paged_append(A, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // extern "C"
