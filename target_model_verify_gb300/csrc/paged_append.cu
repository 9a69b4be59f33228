// New positions' keys and values into a paged bf16 cache: row i goes to slot
// slots[i] of the pool, both K and V.
//
// Bound: HBM (8 bytes moved for a key and a value element), latency for a
// step's few rows. A warp (or part of one, for short rows) copies one row of
// K or of V in 16-byte pieces, four in flight to a lane, with the slot's load
// beside the row's. Measured (8 KV heads of 128): 3.1 us for 256 x 5 rows (10.5
// MB), 11.1 us for 20.5k rows of 16 prompts (84 MB, 7580 GB/s with the writes in
// L2; 16.8 us, 5000 GB/s, from cold caches).
#include "kernels.h"

namespace specdec {
namespace {

constexpr int kThreads = 256;

// kLanes: lanes to a row.
template <int kLanes>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ PagedAppendLaunch A) {
  grid_launch_dependents();          // the next kernel may get ready, and wait for this one's end
  grid_dependency_wait();
  if (blockIdx.x == gridDim.x - 1) {
    // the last CTA alone checks the map of the call and writes the status word
    int bad = 0;
    for (long long i = threadIdx.x; i < A.rows_total; i += kThreads) {
      const int slot = A.slots[i];
      if (slot < -1 || slot >= A.pool_rows || (slot >= 0 && A.rows && (unsigned)A.rows[i] >= (unsigned)A.n)) bad = 1;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *A.status = bad ? SPECDEC_ERR_INVALID_ARG : SPECDEC_OK;
    return;
  }
  const long long item = (long long)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
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
