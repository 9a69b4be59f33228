// Block tables and slot maps from the requests' lengths, on the GPU.
//
// Sequence b is to hold the pages of rows 0 .. start_b + count_b - 1:
//   want_b = ceil((start_b + count_b) / page).
// Pages want_b .. held_b - 1 go onto the stack of free pages, over all
// sequences in order, and then pages held_b .. want_b - 1 come off its top, in
// the same order, so the outcome is one whatever the timing. Where every page
// goes is a prefix sum over the sequences; the map of a row is
//   slot = table[b][row / page] * page + row % page.
//
// Bound: latency (a few bytes per sequence and row): the sums, then a trip to
// memory and a barrier for the pages given back, for the pages taken, and for
// the map. One CTA for a step's few entries, a cluster for prompts, whose
// CTAs compute the same sums and share the entries out.
#include "kernels.h"

namespace specdec {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

struct SeqPlan {
  int have, want;
  bool bad, broken;      // this sequence cannot be; the packed rows' offsets cannot
};

__device__ __forceinline__ SeqPlan plan_of(const PagePlanLaunch& A, int b) {
  const int start = A.start[b], count = A.counts[b], cap = A.max_pages << A.page_log2;
  SeqPlan p;
  p.have = __ldcg(A.held + b);
  p.bad = start < 0 || count < 0 || start > cap - count || p.have < 0 || p.have > A.max_pages;
  p.broken = false;
  if (A.slots) {
    if (A.cu_rows) {
      const int lo = A.cu_rows[b], hi = A.cu_rows[b + 1];
      p.broken = lo < 0 || hi < lo || hi > A.n_slots;
      p.bad = p.bad || p.broken || count > hi - lo;
    } else {
      p.bad = p.bad || count > A.n;
    }
  }
  if (p.bad) p.have = 0;
  p.want = p.bad ? 0 : (start + count + (1 << A.page_log2) - 1) >> A.page_log2;
  return p;
}

__device__ __forceinline__ void sync_all() {
  if (gridDim.x > 1)
    cluster_sync_all();
  else
    __syncthreads();
}

// Moves the pages that change hands one way, over all sequences in order:
// move(sequence, its entry of the table, the page's rank).
template <bool kTake, typename Move>
__device__ __forceinline__ void move_pages(const PagePlanLaunch& A, int* upto, int* from, int* warp_sum, Move move) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int carry = 0;
  for (int b0 = 0; b0 < A.B; b0 += kThreads) {
    SeqPlan p = {0, 0, true, false};
    if (b0 + tid < A.B) p = plan_of(A, b0 + tid);
    int run = kTake ? max(0, p.want - p.have) : max(0, p.have - p.want);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    if (lane == 31) warp_sum[warp] = run;
    __syncthreads();
    if (warp == 0) {
      int s = warp_sum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += x;
      }
      warp_sum[lane] = s;
    }
    __syncthreads();
    upto[tid] = run + (warp ? warp_sum[warp - 1] : 0);
    from[tid] = kTake ? p.have : p.want;
    __syncthreads();
    const int moves = upto[kThreads - 1];
    for (int m = (int)blockIdx.x * kThreads + tid; m < moves; m += (int)gridDim.x * kThreads) {
      int lo = 0, hi = kThreads - 1;                      // the first sequence with upto > m
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] > m)
          hi = mid;
        else
          lo = mid + 1;
      }
      move(b0 + lo, from[lo] + m - (lo ? upto[lo - 1] : 0), carry + m);
    }
    carry += moves;
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kThreads, 1) page_plan_kernel(const __grid_constant__ PagePlanLaunch A) {
  __shared__ int upto[kThreads], from[kThreads], warp_sum[32];
  __shared__ long long give_sum[kWarps], take_sum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_launch_dependents();          // the next kernel may get ready, and wait for this one's end
  grid_dependency_wait();
  // ---- how many pages change hands (64 bits: lengths may ask for any number) ----
  long long give = 0, take = 0;
  bool bad = false, broken = false;
  for (int b = tid; b < A.B; b += kThreads) {
    const SeqPlan p = plan_of(A, b);
    give += max(0, p.have - p.want);
    take += max(0, p.want - p.have);
    bad |= p.bad;
    broken |= p.broken;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    give += __shfl_xor_sync(0xffffffffu, give, o);
    take += __shfl_xor_sync(0xffffffffu, take, o);
  }
  if (lane == 0) {
    give_sum[warp] = give;
    take_sum[warp] = take;
  }
  bad = __syncthreads_or(bad);
  broken = __syncthreads_or(broken);
  give = take = 0;
  for (int w = 0; w < kWarps; ++w) {
    give += give_sum[w];
    take += take_sum[w];
  }
  const int n_free = __ldcg(A.n_free);
  const bool state_ok = !broken && n_free >= 0 && n_free <= A.n_pages && give <= A.n_pages - n_free;
  const bool enough = state_ok && take <= n_free + give, moves = enough && (give > 0 || take > 0);
  if (blockIdx.x == 0 && tid == 0)
    *A.status = !state_ok ? SPECDEC_ERR_INVALID_ARG
                : !enough ? SPECDEC_ERR_NO_PAGES
                          : (bad ? SPECDEC_ERR_INVALID_ARG : SPECDEC_OK);
  sync_all();                        // the status before the map's, and everyone knows what there was
  if (moves) {
    const int top = n_free + (int)give;
    if (give > 0) {
      move_pages<false>(A, upto, from, warp_sum, [&](int b, int x, int rank) {
        int32_t* const at = A.table + (size_t)b * A.max_pages + x;
        A.free_pages[n_free + rank] = __ldcg(at);
        *at = -1;
      });
      sync_all();
    }
    if (take > 0) {
      move_pages<true>(A, upto, from, warp_sum, [&](int b, int x, int rank) {
        A.table[(size_t)b * A.max_pages + x] = __ldcg(A.free_pages + top - 1 - rank);
      });
      sync_all();
    }
    // Who still looks at these below asks only whether they are in range, as both are.
    if (blockIdx.x == 0) {
      for (int b = tid; b < A.B; b += kThreads) {
        const SeqPlan p = plan_of(A, b);
        if (!p.bad && p.want != p.have) A.held[b] = p.want;
      }
      if (tid == 0) *A.n_free = top - (int)take;
    }
  }
  // ---- the map, four entries a thread ----
  if (!A.slots) return;
  const int mask = (1 << A.page_log2) - 1, n_slots = (int)A.n_slots;
  bool odd = false;
  for (long long t0 = 4ll * (blockIdx.x * kThreads + tid); t0 < n_slots; t0 += 4ll * gridDim.x * kThreads) {
    int b = 0, at_b = -1, begin = 0, end = 0, start = 0;      // a sequence's entries of the map, and what they hold
    if (enough && A.cu_rows) {
      int lo = -1, hi = A.B;                                  // the last sequence that begins at t0 or before
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (A.cu_rows[mid] <= t0)
          lo = mid;
        else
          hi = mid;
      }
      b = max(lo, 0);
    }
    int v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = (int)t0 + k;
      v[k] = -1;
      if (!enough || t >= n_slots) continue;
      if (A.cu_rows)
        while (b + 1 < A.B && A.cu_rows[b + 1] <= t) ++b;
      else
        b = t / A.n;
      if (b != at_b) {
        at_b = b;
        begin = end = 0;
        if (b < A.B && !plan_of(A, b).bad) {
          begin = A.cu_rows ? A.cu_rows[b] : b * A.n;
          end = begin + A.counts[b];
          start = A.start[b];
        }
      }
      if (t < begin || t >= end) continue;
      const int row = start + t - begin;
      const int id = __ldcg(A.table + (size_t)b * A.max_pages + (row >> A.page_log2));
      if ((unsigned)id < (unsigned)A.n_pages)
        v[k] = (id << A.page_log2) + (row & mask);
      else
        odd = true;
    }
    if (t0 + 4 <= n_slots && ((uintptr_t)A.slots & 15u) == 0) {
      *reinterpret_cast<int4*>(A.slots + t0) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (t0 + k < n_slots) A.slots[t0 + k] = v[k];
    }
  }
  if (odd) set_status(A.status, SPECDEC_ERR_INVALID_ARG);
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanLaunch& A, cudaStream_t stream) {
  const int ctas = A.n_slots > 4 * kThreads || A.B > kThreads ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, page_plan_kernel, A);
}

}  // namespace specdec
