// Appending to an 8-bit key/value cache: the new positions' keys and values,
// bf16, become e4m3 codes with one scale per (32 cache rows, KV head).
//
// For the rows of one block, scale s = 2^e with the smallest e (clamped to
// [-40, 40]) such that max |x| <= 448 s over the finite new values, and
// code = e4m3(x / s). A power of two loses nothing against a finer scale but
// the subnormal end (e4m3 keeps 4 significant bits at any exponent), makes
// x / s exact, and lets a block whose scale has to grow be re-encoded by an
// exponent shift. A block that already holds rows before `start` keeps the
// larger of its scale and the new rows' one.
//
// Bound: HBM for prompts (6 bytes moved per key/value pair of elements: 2 x 2
// read, 2 x 1 written), latency for a step's few rows. One warp owns a
// (block, KV head, K or V): the block's new rows stay in registers between
// the maximum and the encoding, so they are read once, and no other warp
// writes that block. Calls of up to kFew new rows keep registers for that
// many only, and in longer ones two warps share a block (16 rows each), so
// that more warps are resident. Measured (8 KV heads of 128): 2.3 us for one
// sequence's 5 rows (a launch's latency), 5.1 us for 256 sequences' (7.9 MB),
// 8.3 us for four ragged prompts of 3206 rows in all (19.7 MB, 2370 GB/s; 8.4
// us with one warp per block). A warp is a chain of two dependent trips to
// memory (its sequence's start and count, then rows and scale side by side;
// with a table of rows three) and the write. The grid has room for n rows of
// every sequence, so most of the prompts' 4129 CTAs (five per SM, more than
// five waves) find nothing to do. The tables are checked by one CTA: tree
// commits of 26 nodes take 3.1 us for 16 sequences, 6.8 for 64, 23.2 for 256
// (10.5 without the table of rows).
#include <cuda_fp16.h>

#include "kernels.h"

namespace specdec {
namespace {

constexpr int kT = SPECDEC_KV8_BLOCK;
constexpr int kWarps = 4;
constexpr int kFew = 8;
constexpr int kMinExp = -40, kMaxExp = 40;

// e4m3 pair from two floats: nearest, ties to even, saturating; NaN stays.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}
__device__ __forceinline__ float2 from_e4m3x2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// 448 = 1.75 * 2^8: the smallest e with amax <= 448 * 2^e, from the bits.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return amax > 0.f ? min(max(e, kMinExp), kMaxExp) : kMinExp;
}

__device__ __forceinline__ bool sequence_ok(const Kv8AppendLaunch& A, int start, int count) {
  return count <= A.n && start >= 0 && start <= A.Lmax - count;
}

// kMost: rows a warp holds; kSharers: warps that share a block.
template <int kD, int kMost, int kSharers>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const __grid_constant__ Kv8AppendLaunch A,
                                                             long long items) {
  grid_launch_dependents();          // the next kernel may get ready, and wait for this one's end
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == gridDim.x - 1) {
    // the last CTA alone checks the tables of the call and writes the status word
    int bad = 0;
    for (long long e = threadIdx.x; e < A.B; e += 32 * kWarps) {
      const int count = A.counts ? A.counts[e] : A.n;
      if (count > 0 && !sequence_ok(A, A.start[e], count)) bad = 1;
    }
    if (A.rows)
      for (long long e = threadIdx.x; e < (long long)A.B * A.n; e += 32 * kWarps) {
        // (a sequence's entries past its count are not read)
        const int count = A.counts ? A.counts[e / A.n] : A.n, i = (int)(e % A.n);
        if (i < count && (unsigned)A.rows[e] >= (unsigned)A.n) bad = 1;
      }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *A.status = bad ? SPECDEC_ERR_INVALID_ARG : SPECDEC_OK;
    return;
  }
  const int warp = threadIdx.x >> 5, sharer = warp % kSharers;
  const long long item = (long long)blockIdx.x * (kWarps / kSharers) + warp / kSharers;
  if (item >= items) return;
  const int kv = (int)(item & 1);
  const int h = (int)((item >> 1) % A.Hkv);
  const long long bl = (item >> 1) / A.Hkv;
  const int b = (int)(bl / A.max_blocks);
  const int start = A.start[b];
  const int count = A.counts ? A.counts[b] : A.n;
  if (count <= 0 || !sequence_ok(A, start, count)) return;
  const int blk = start / kT + (int)(bl % A.max_blocks);
  const int first = blk * kT;                       // the block's first cache row
  if (first >= start + count) return;

  constexpr int kLanes = kD / 8;                    // lanes per row, 8 values each
  constexpr int kRowsAtOnce = 32 / kLanes;
  constexpr int kSteps = kMost / kRowsAtOnce;
  const int c = lane % kLanes, r0 = lane / kLanes;
  const int base = max(first, start) + sharer * kMost;                     // this warp's first new row
  const int end = min(min(first + kT, start + count), base + kMost);
  float* scale_at = A.scale[kv] + ((size_t)b * A.Hkv + h) * A.n_scale + blk;
  const float was = first < start ? *scale_at : 0.f;
  uint4 x[kSteps];
  float amax = 0.f;
  bool ok = true;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int i = base + k * kRowsAtOnce + r0 - start;        // new row
    x[k] = make_uint4(0u, 0u, 0u, 0u);
    if (i < end - start) {
      int src = i;
      if (A.rows) {
        src = A.rows[(size_t)b * A.n + i];
        if (src < 0 || src >= A.n) {
          ok = false;
          src = 0;
        }
      }
      x[k] = __ldcg(reinterpret_cast<const uint4*>(A.src[kv] + ((size_t)b * A.n + src) * A.stride[kv] +
                                                  (size_t)h * kD + c * 8));
    }
  }
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float lo = fabsf(__uint_as_float(w[q] << 16)), hi = fabsf(__uint_as_float(w[q] & 0xffff0000u));
      if (lo < INFINITY) amax = fmaxf(amax, lo);
      if (hi < INFINITY) amax = fmaxf(amax, hi);
    }
  }
  ok = __all_sync(0xffffffffu, ok);
  amax = warp_max(amax);
  if constexpr (kSharers > 1) {
    // the sharers' maxima (and whether every row index was good)
    __shared__ float shared_max[kWarps];
    const int pair = warp / kSharers;
    if (lane == 0) shared_max[warp] = ok ? amax : -1.f;
    named_bar_sync(1 + pair, 32 * kSharers);
#pragma unroll
    for (int x = 0; x < kSharers; ++x) {
      const float a = shared_max[pair * kSharers + x];
      ok = ok && a >= 0.f;
      amax = fmaxf(amax, a);
    }
  }
  if (!ok) return;
  const float s = fmaxf(pow2(scale_exponent(amax)), was);
  const float inv = 1.f / s;
  uint8_t* out = A.cache[kv] + ((size_t)b * A.Lmax * A.Hkv + h) * kD + c * 8;
  const size_t pitch = (size_t)A.Hkv * kD;
  if (sharer == 0 && first < start && s != was) {
    // the block's scale grows: its earlier rows are encoded again
    const float ratio = was * inv;
    for (int r = first + r0; r < start; r += kRowsAtOnce) {
      uint2* at = reinterpret_cast<uint2*>(out + (size_t)r * pitch);
      const uint2 o = *at;
      const uint32_t w[2] = {o.x, o.y};
      uint32_t n[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float2 f0 = from_e4m3x2((uint16_t)w[q]), f1 = from_e4m3x2((uint16_t)(w[q] >> 16));
        n[q] = e4m3x2(f0.x * ratio, f0.y * ratio) | (e4m3x2(f1.x * ratio, f1.y * ratio) << 16);
      }
      *at = make_uint2(n[0], n[1]);
    }
  }
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int r = base + k * kRowsAtOnce + r0;
    if (r >= end) continue;
    const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
    uint32_t n[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      n[q] = e4m3x2(__uint_as_float(w[q] << 16) * inv, __uint_as_float(w[q] & 0xffff0000u) * inv);
    *reinterpret_cast<uint2*>(out + (size_t)r * pitch) = make_uint2(n[0] | (n[1] << 16), n[2] | (n[3] << 16));
  }
  if (sharer == 0 && lane == 0 && s != was) *scale_at = s;
}

template <int kD>
cudaError_t launch_dim(const Kv8AppendLaunch& A, cudaStream_t stream) {
  const long long items = 2ll * A.B * A.max_blocks * A.Hkv;
  const int per_cta = A.n <= kFew ? kWarps : kWarps / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((items + per_cta - 1) / per_cta + 1));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return A.n <= kFew ? cudaLaunchKernelEx(&cfg, append_kernel<kD, kFew, 1>, A, items)
                     : cudaLaunchKernelEx(&cfg, append_kernel<kD, kT / 2, 2>, A, items);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendLaunch& A, cudaStream_t stream) {
  switch (A.D) {
    case 64: return launch_dim<64>(A, stream);
    case 128: return launch_dim<128>(A, stream);
    case 256: return launch_dim<256>(A, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace specdec
