// New positions' keys and values into a paged bf16 cache: row i goes to slot
// slots[i] of the pool, both K and V.
//
// Bound: HBM (8 bytes moved for a key and a value element), latency for a
// step's few rows. A warp (or part of one, for short rows) copies one row of
// K or of V in 16-byte pieces, four in flight to a lane, with the slot's load
// beside the row's. Measured (8 KV heads of 128, graph replays): 3.1 us for 256 x
// 5 rows (10.5 MB), 8.2 us for 10.3k rows of 16 prompts (84 MB, which stay in L2;
// 11.1 with the check of the map in the last CTA, which then began last, an entry
// at a time), 60 us for 65k rows (537 MB, 8900 GB/s with a part in L2; 95); one
// head of 64: 65k rows in 6.2 us (24).
#include "kernels.h"

namespace specdec {
namespace {

constexpr int kThreads = 256;

// kLanes: lanes to a row.
template <int kLanes>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ PagedAppendLaunch A) {
  grid_launch_dependents();          // the next kernel may get ready, and wait for this one's end
  grid_dependency_wait();
  if (blockIdx.x == 0) {
    // The first CTA alone checks the map of the call and writes the status word:
    // eight loads of four entries in flight to a thread, so that it keeps up with
    // the copies of short rows.
    int bad = 0;
    const long long quads = !A.rows && ((uintptr_t)A.slots & 15u) == 0 ? A.rows_total / 4 : 0;
    for (long long i0 = threadIdx.x; i0 < quads; i0 += 8 * kThreads) {
      int4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        v[k] = i0 + k * kThreads < quads ? reinterpret_cast<const int4*>(A.slots)[i0 + k * kThreads]
                                         : make_int4(-1, -1, -1, -1);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        bad |= min(min(v[k].x, v[k].y), min(v[k].z, v[k].w)) < -1 ||
               max(max(v[k].x, v[k].y), max(v[k].z, v[k].w)) >= A.pool_rows;
    }
    for (long long i0 = 4 * quads + threadIdx.x; i0 < A.rows_total; i0 += 8 * kThreads) {
      int slot[8], row[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const long long i = i0 + k * kThreads;
        slot[k] = i < A.rows_total ? A.slots[i] : -1;
        row[k] = A.rows && i < A.rows_total ? A.rows[i] : 0;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        bad |= slot[k] < -1 || slot[k] >= A.pool_rows || (slot[k] >= 0 && (unsigned)row[k] >= (unsigned)A.n);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *A.status = bad ? SPECDEC_ERR_INVALID_ARG : SPECDEC_OK;
    return;
  }
  const long long item = (long long)(blockIdx.x - 1) * (kThreads / kLanes) + threadIdx.x / kLanes;
  const long long i = item >> 1;
  if (i >= A.rows_total) return;
  const int kv = (int)(item & 1), c0 = threadIdx.x % kLanes;
  const int slot = A.slots[i];
  if (slot < 0 || slot >= A.pool_rows) return;
  long long from = i;
  if (A.rows) {
    const int r = A.rows[i];
    if ((unsigned)r >= (unsigned)A.n) return;
    from = i / A.n * A.n + r;
  }
  const uint4* const src = A.src[kv] + from * A.stride[kv];
  uint4* const dst = A.pages[kv] + (long long)slot * A.row_chunks;
  for (int c = c0; c < A.row_chunks; c += 4 * kLanes) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k * kLanes < A.row_chunks) v[k] = __ldcg(src + c + k * kLanes);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k * kLanes < A.row_chunks) dst[c + k * kLanes] = v[k];
  }
}

template <int kLanes>
cudaError_t launch_lanes(const PagedAppendLaunch& A, cudaStream_t stream) {
  constexpr int kItems = kThreads / kLanes;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((2 * A.rows_total + kItems - 1) / kItems + 1));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_append_kernel<kLanes>, A);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendLaunch& A, cudaStream_t stream) {
  return A.row_chunks <= 8 ? launch_lanes<8>(A, stream)
         : A.row_chunks <= 16 ? launch_lanes<16>(A, stream) : launch_lanes<32>(A, stream);
}

}  // namespace specdec
