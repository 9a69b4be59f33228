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
// Bound: latency (a few bytes per sequence and row). A step's plan is one CTA
// and two trips to memory: the lengths, and then, side by side, the pages given
// back, those taken (off the stack, or out of the entries just given back) and
// the map's old entries. Larger plans run as a cluster whose CTAs compute the
// same sums and share the entries out: first the pages given back, then, behind
// a barrier, the pages taken and the map, which reads those off the stack too.
// Measured (graph replays): 3.5 us for a step's plan of 8 sequences x 5 rows
// (7.4 with a trip and a barrier per phase), 19 us for 128k rows of 256 prompts
// planned and given back (29 with one CTA for a call without a map and the map
// behind the table's barrier). A step's call without a map, 8 sequences: 1.7 us,
// and 3.7 as a cluster, which it becomes with more than 16,384 table entries.
#include "kernels.h"

namespace specdec {
namespace {

constexpr int kFew = 256, kMany = 1024;      // threads of a step's CTA, and of a cluster's
constexpr int kCluster = 8;

__device__ __forceinline__ void sync_all() {
  if (gridDim.x > 1)
    cluster_sync_all();
  else
    __syncthreads();
}

// What kThreads consecutive sequences ask for.
template <int kThreads>
struct Chunk {
  int start[kThreads], have[kThreads], want[kThreads];
  int begin[kThreads], end[kThreads];                  // their entries of the map (none: begin = end)
  int give_upto[kThreads], take_upto[kThreads];        // pages that change hands up to and with each
  long long give_sum[kThreads / 32], take_sum[kThreads / 32];
  int taken[kThreads];                                 // few moves: the pages taken, in order
};

// The sequence with the move m, by its running count.
template <int kThreads>
__device__ __forceinline__ int owner(const int (&upto)[kThreads], int m) {
  int lo = 0, hi = kThreads - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (upto[mid] > m)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

struct Totals {
  long long give, take;
  bool bad, broken;            // a sequence that cannot be; packed rows' offsets that cannot
};

// Fills the chunk from sequence b0 on; every thread of the CTA, to the barrier at its end.
template <int kThreads>
__device__ __forceinline__ Totals load_chunk(const PagePlanLaunch& A, Chunk<kThreads>& C, int b0) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = b0 + tid;
  int have = 0, want = 0, start = 0, begin = 0, end = 0;
  bool bad = false, broken = false;
  if (b < A.B) {
    start = A.start[b];
    const int count = A.counts[b], cap = A.max_pages << A.page_log2;
    have = __ldcg(A.held + b);
    bad = start < 0 || count < 0 || start > cap - count || have < 0 || have > A.max_pages;
    int room = 0;
    if (A.slots) {
      if (A.cu_rows) {
        begin = A.cu_rows[b];
        const int hi = A.cu_rows[b + 1];
        broken = begin < 0 || hi < begin || hi > A.n_slots;
        room = broken ? 0 : hi - begin;
      } else {
        begin = b * A.n;
        room = A.n;
      }
      bad = bad || broken || count > room;
    }
    if (bad) have = 0;
    want = bad ? 0 : (start + count + (1 << A.page_log2) - 1) >> A.page_log2;
    end = bad ? begin : begin + count;
  }
  C.start[tid] = start;
  C.have[tid] = have;
  C.want[tid] = want;
  C.begin[tid] = begin;
  C.end[tid] = end;
  long long give = max(0, have - want), take = max(0, want - have);    // lengths may ask for more than 2^31 in all
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long g = __shfl_up_sync(0xffffffffu, give, o), t = __shfl_up_sync(0xffffffffu, take, o);
    if (lane >= o) {
      give += g;
      take += t;
    }
  }
  if (lane == 31) {
    C.give_sum[warp] = give;
    C.take_sum[warp] = take;
  }
  Totals sum = {0, 0, false, false};
  sum.bad = __syncthreads_or(bad);
  sum.broken = __syncthreads_or(broken);
  long long g0 = 0, t0 = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) {
      g0 = sum.give;
      t0 = sum.take;
    }
    sum.give += C.give_sum[w];
    sum.take += C.take_sum[w];
  }
  C.give_upto[tid] = (int)(g0 + give);           // used only where all of them fit 32 bits
  C.take_upto[tid] = (int)(t0 + take);
  __syncthreads();
  return sum;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1) page_plan_kernel(const __grid_constant__ PagePlanLaunch A) {
  __shared__ Chunk<kThreads> C;
  const int tid = threadIdx.x, mask = (1 << A.page_log2) - 1, n_slots = (int)A.n_slots;
  const int all = (int)gridDim.x * kThreads, me = (int)blockIdx.x * kThreads + tid;
  const bool one_chunk = A.B <= kThreads;
  grid_launch_dependents();          // the next kernel may get ready, and wait for this one's end
  grid_dependency_wait();
  const int n_free = __ldcg(A.n_free);
  Totals sum = load_chunk(A, C, 0);
  for (int b0 = kThreads; b0 < A.B; b0 += kThreads) {
    __syncthreads();
    const Totals s = load_chunk(A, C, b0);
    sum.give += s.give;
    sum.take += s.take;
    sum.bad |= s.bad;
    sum.broken |= s.broken;
  }
  const bool state_ok = !sum.broken && n_free >= 0 && n_free <= A.n_pages && sum.give <= A.n_pages - n_free;
  const bool enough = state_ok && sum.take <= n_free + sum.give;
  const int give = enough ? (int)sum.give : 0, take = enough ? (int)sum.take : 0, top = n_free + give;
  if (me == 0)
    *A.status = !state_ok ? SPECDEC_ERR_INVALID_ARG
                : !enough ? SPECDEC_ERR_NO_PAGES
                          : (sum.bad ? SPECDEC_ERR_INVALID_ARG : SPECDEC_OK);
  // Entries of the sequence s of the chunk at b0.
  auto entry = [&](int b0, int s, int x) { return A.table + (size_t)(b0 + s) * A.max_pages + x; };
  auto given = [&](int b0, int m) {
    const int s = owner(C.give_upto, m);
    return entry(b0, s, C.want[s] + m - (s ? C.give_upto[s - 1] : 0));
  };
  auto taken = [&](int b0, int m) {
    const int s = owner(C.take_upto, m);
    return entry(b0, s, C.have[s] + m - (s ? C.take_upto[s - 1] : 0));
  };
  bool odd = false;
  auto moved = [&](int id) {               // a page that changes hands
    odd |= (unsigned)id >= (unsigned)A.n_pages;
    return id;
  };
  auto slot_of = [&](int id, int row) {
    if ((unsigned)id < (unsigned)A.n_pages) return (id << A.page_log2) + (row & mask);
    odd = true;
    return -1;
  };
  auto put = [&](int t0, const int (&v)[4]) {
    if (t0 + 4 <= n_slots && ((uintptr_t)A.slots & 15u) == 0) {
      *reinterpret_cast<int4*>(A.slots + t0) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (t0 + k < n_slots) A.slots[t0 + k] = v[k];
    }
  };
  // The sequence with entry t of the map (the last that begins there or before), in one chunk.
  auto of_entry = [&](int t) {
    if (!A.cu_rows) return t / A.n;
    int lo = 0, hi = A.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (C.begin[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  };

  if (gridDim.x == 1 && one_chunk && give <= kThreads && take <= kThreads && n_slots <= 4 * kThreads) {
    // ---- few of everything: all loads ahead of all stores ----
    int given_id = 0, taken_id = 0, row[4], at[4], v[4];
    int32_t* const from = tid < give ? given(0, tid) : nullptr;
    int32_t* const to = tid < take ? taken(0, tid) : nullptr;
    if (from) given_id = __ldcg(from);
    if (to) {
      const int pos = top - 1 - tid;
      taken_id = __ldcg(pos < n_free ? A.free_pages + pos : given(0, pos - n_free));
    }
    // an entry of the map: an old page (v), or the at'th that is taken
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = 4 * tid + k;
      v[k] = at[k] = -1;
      if (!enough || t >= n_slots || A.B == 0) continue;
      const int s = of_entry(t);
      if (t < C.begin[s] || t >= C.end[s]) continue;
      row[k] = C.start[s] + t - C.begin[s];
      const int x = row[k] >> A.page_log2;
      if (x < C.have[s])
        v[k] = __ldcg(entry(0, s, x));
      else
        at[k] = x - C.have[s] + (s ? C.take_upto[s - 1] : 0);
      if (at[k] < 0) at[k] = -2;               // v is what the table held
    }
    if (to) C.taken[tid] = taken_id;
    __syncthreads();
    if (from) {
      *from = -1;
      A.free_pages[n_free + tid] = moved(given_id);
    }
    if (to) *to = moved(taken_id);
    if (enough && tid < A.B && C.want[tid] != C.have[tid]) A.held[tid] = C.want[tid];
    if (tid == 0 && (give || take)) *A.n_free = top - take;
    if (4 * tid < n_slots) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (at[k] != -1) v[k] = slot_of(at[k] >= 0 ? C.taken[at[k]] : v[k], row[k]);
      put(4 * tid, v);
    }
    if (odd) set_status(A.status, SPECDEC_ERR_INVALID_ARG);
    return;
  }

  sync_all();                        // everyone has read what there was; the status is there
  // Chunk by chunk, in order: what(chunk's first sequence, its first move's rank).
  auto chunks = [&](auto&& what) {
    for (int b0 = 0, rank = 0, step; b0 < A.B; b0 += kThreads, rank += step) {
      if (!one_chunk) {
        __syncthreads();
        load_chunk(A, C, b0);
      }
      step = what(b0, rank);
    }
  };
  auto set_held = [&](int b0, int) {
    if (b0 + tid < A.B && C.want[tid] != C.have[tid]) A.held[b0 + tid] = C.want[tid];
    return 0;
  };
  const bool moves = give > 0 || take > 0;
  if (moves && me == 0) *A.n_free = top - take;
  if (moves && one_chunk && blockIdx.x == 0) chunks(set_held);
  if (give > 0) {
    chunks([&](int b0, int rank) {
      const int here = C.give_upto[kThreads - 1];
      for (int m = me; m < here; m += all) {
        int32_t* const from = given(b0, m);
        A.free_pages[n_free + rank + m] = moved(__ldcg(from));
        *from = -1;
      }
      return here;
    });
    sync_all();                      // the stack is whole
  }
  if (take > 0)
    chunks([&](int b0, int rank) {
      const int here = C.take_upto[kThreads - 1];
      for (int m = me; m < here; m += all) *taken(b0, m) = moved(__ldcg(A.free_pages + top - 1 - rank - m));
      return here;
    });
  // ---- the map: pages that were there from the table, others from the stack as well ----
  auto page_at = [&](int b0, int rank, int s, int x) {
    return __ldcg(x < C.have[s] ? entry(b0, s, x)
                                : A.free_pages + top - 1 - rank - (s ? C.take_upto[s - 1] : 0) - (x - C.have[s]));
  };
  if (A.slots && enough && one_chunk && A.B > 0) {
    // four entries a thread, four times over, loads ahead of stores
    for (long long r0 = 0; r0 < n_slots; r0 += 16ll * all) {
      int id[4][4], row[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const long long t0 = r0 + 4ll * (r * all + me);
        int s = t0 < n_slots ? of_entry((int)t0) : 0, of = -1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          id[r][k] = row[r][k] = -1;
          if (t0 + k >= n_slots) continue;
          const int t = (int)t0 + k;
          while (s + 1 < A.B && C.begin[s + 1] <= t) ++s;
          if (t < C.begin[s] || t >= C.end[s]) continue;
          row[r][k] = C.start[s] + t - C.begin[s];
          if (k > 0 && s == of && (row[r][k] & mask) != 0)
            id[r][k] = id[r][k - 1];                          // the page of the entry before
          else
            id[r][k] = page_at(0, 0, s, row[r][k] >> A.page_log2);
          of = s;
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const long long t0 = r0 + 4ll * (r * all + me);
        int v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = row[r][k] < 0 ? -1 : slot_of(id[r][k], row[r][k]);
        if (t0 < n_slots) put((int)t0, v);
      }
    }
  } else if (A.slots) {
    // Nothing to map, or more sequences than threads: the gaps first, then each chunk's rows.
    for (long long t0 = 4ll * me; t0 < n_slots; t0 += 4ll * all) put((int)t0, {-1, -1, -1, -1});
    if (enough && !one_chunk) {
      sync_all();
      chunks([&](int b0, int rank) {
        const int lane = tid & 31, warps = all / 32;
        for (int s = me / 32; s < min(kThreads, A.B - b0); s += warps)
          for (long long t = C.begin[s] + (long long)lane; t < C.end[s]; t += 32) {      // (past 2^31 at the last step)
            const int row = C.start[s] + (int)(t - C.begin[s]);
            A.slots[t] = slot_of(page_at(b0, rank, s, row >> A.page_log2), row);
          }
        return C.take_upto[kThreads - 1];
      });
    }
  }
  if (odd) set_status(A.status, SPECDEC_ERR_INVALID_ARG);
  if (moves && !one_chunk) {
    sync_all();                      // nobody looks at the lengths any more
    if (blockIdx.x == 0) chunks(set_held);
  }
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanLaunch& A, cudaStream_t stream) {
  // One CTA while each of its threads has four entries of the map at most. Pages
  // that change hands are few then, except where a call without a map gives
  // back a whole batch's: how many is known on the device only, so the tables'
  // size stands for it.
  const bool one = A.B <= kMany && A.n_slots <= 4 * kMany && (A.n_slots > 0 || (long long)A.B * A.max_pages <= 16384);
  const bool few = one && A.B <= kFew && A.n_slots <= 4 * kFew;
  const int ctas = one ? 1 : kCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(few ? kFew : kMany);
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
  return few ? cudaLaunchKernelEx(&cfg, page_plan_kernel<kFew>, A) : cudaLaunchKernelEx(&cfg, page_plan_kernel<kMany>, A);
}

}  // namespace specdec
