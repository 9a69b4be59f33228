// The paged cache attention (see cache_attention.cuh) for little work: up to
// 16 query rows per KV head, few and short sequences, where latency counts and
// not the rate.
//
// A cluster of CTAs takes one (sequence, KV head); its warps deal out the
// 16-row chunks of the cache, each one page's, and keep an online softmax of
// their own. Nothing waits for anything else until the end: a warp loads its
// chunks with cp.async, two in flight, and multiplies them with mma.sync (16
// query rows x 8 keys or dims a step), which needs no barriers, no tensor
// memory and no set-up, where the tcgen05 form spends 6 us on its roles, its
// merge kernel and 128 rows of products. The warps' parts are joined in shared
// memory, the CTAs' through the cluster's, and the output is written without a
// second kernel.
//
// Bound: latency. The lengths and the page table are one trip to memory (side
// by side, without a window), keys, values and queries the second; a chunk
// then costs a warp 0.75 us (1.4 at 256 dims), and the joins 1 us. Measured (8
// KV heads of 128, 4 query heads each, one token, pages of 16; graph replays),
// this and the tcgen05 form: 1 x 517 rows 5.8 / 10.6 us, 1 x 2048 6.6 / 12.0, 1
// x 8192 13.4 / 15.0, 4 x 2048 8.5 / 14.4, 16 x 517 8.6 / 18.5; 64 dims, 4 x
// 2048 6.5 / 12.2; 256 dims (4 KV heads), 1 x 517 7.2 / 12.1, 16 x 517 10.7 /
// 19.3. With more chunks per warp, where one sequence alone may hold a batch
// up, with more CTAs than run at once (64 x 517: 54 / 40) or with a second tile
// of 16 rows (20 rows, 1 x 517: 10.0 / 10.8, ragged 16 x 2048 31 / 20) it is
// no faster, and the other form is taken (cache_attn_by_few).
//
// The statistics are fp32; the probabilities enter the product, and the sum,
// rounded to bf16, as in the other form.
#include "cache_attention.cuh"

namespace specdec {
namespace cache_attn {

constexpr int kFewMost = 8;                       // CTAs of a cluster at most
constexpr int kFewKeys = 16;                      // rows of a chunk: a page's or a part of one

template <int kD>
struct FewShape {
  static constexpr int kWarps = cache_attn_few_warps(kD), kThreads = 32 * kWarps;
  static constexpr int kStages = 2;                             // chunks in flight per warp
  static constexpr int kRowBytes = kD * 2, kPieces = kD / 8;    // 16-byte pieces of a row
  static constexpr int kChunk = kFewKeys * kRowBytes;           // of K, or of V
  static constexpr int kWarpBytes = kStages * 2 * kChunk;
  static constexpr int kSmem = kWarps * kWarpBytes;
  static_assert(kCacheAttnFewRows * kD * 4 <= kWarpBytes, "a warp's part of the output fits its ring");
};

// What the kernel needs of a call (CacheAttnLaunch's tree alone is 2 KB to hand over).
struct FewLaunch {
  int B, n_new, Hq, Hkv, G, Lmax, window, tree, max_depth, max_pages, page_log2, n_pages;
  float scale, cap, cap_exp;
  long long q_stride;
  const __nv_bfloat16 *q, *k, *v;
  const float* slopes;
  const int32_t *seq_lens, *table;
  __nv_bfloat16* out;
  int* status;
  uint16_t anc[kCacheAttnFewRows];   // bit a of entry i: new position i sees new position a
  uint8_t depth[kCacheAttnFewRows];
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ bool not_finite2(uint32_t x) {       // either of two bf16
  return (((x & 0x7fff7fffu) + 0x00800080u) & 0x80008000u) != 0;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

template <int kD, bool kExtra>
__global__ void __launch_bounds__(FewShape<kD>::kThreads)
    few_attn_kernel(const __grid_constant__ FewLaunch A, int ctas) {
  using S = FewShape<kD>;
  constexpr int kRows = kCacheAttnFewRows, kWarps = S::kWarps, kThreads = S::kThreads;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ float2 warp_ml[kWarps][kRows];       // (reference, sum)
  __shared__ float2 cta_ml[kRows];
  __shared__ int flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % ctas, tile = blockIdx.x / ctas, all_warps = ctas * kWarps;
  const uint32_t smem = smem_u32(smem_raw);
  const int page = 1 << A.page_log2;
  auto sync_ctas = [&]() {
    if (ctas > 1)
      cluster_sync_all();
    else
      __syncthreads();
  };
  grid_launch_dependents();          // the next kernel may get ready, and wait for this one's end
  grid_dependency_wait();

  if (tile == A.B * A.Hkv) {
    // ---- the last cluster alone looks through the call's tables and writes the status word ----
    // (sequence, page) pairs dealt out over the threads, four at a time, so that
    // many sequences take no longer than the attention
    int bad = 0;
    const int per = A.window > 0 ? min(A.max_pages, (A.window + A.n_new + page - 1) / page + 1) : A.max_pages;
    const int pairs = A.B * per, step = ctas * kThreads;
    for (int e0 = rank * kThreads + threadIdx.x; e0 < pairs; e0 += 4 * step) {
      int L[4], id[4], p[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int e = e0 + x * step, b = e / per;
        L[x] = 0;
        if (e >= pairs) continue;
        L[x] = A.seq_lens[b];
        p[x] = e - b * per + (A.window > 0 ? max(0, L[x] - A.n_new - A.window + 1) >> A.page_log2 : 0);
        id[x] = p[x] < A.max_pages ? A.table[(size_t)b * A.max_pages + p[x]] : 0;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (L[x] != 0)
          bad |= L[x] < A.n_new || L[x] > A.Lmax ||
                 (p[x] <= (L[x] - 1) >> A.page_log2 && (unsigned)id[x] >= (unsigned)A.n_pages);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) flag = bad;
    sync_ctas();
    if (rank == 0 && warp == 0) {
      bad = lane < ctas ? ld_cluster_s32(mapa_shared(smem_u32(&flag), lane)) : 0;
      bad = __any_sync(0xffffffffu, bad);
      if (lane == 0) *A.status = bad ? SPECDEC_ERR_INVALID_ARG : SPECDEC_OK;
    }
    sync_ctas();
    return;
  }

  const int b = tile / A.Hkv, h = tile % A.Hkv, R = A.n_new * A.G, g = rank * kWarps + warp;
  const int32_t* const table = A.table + (size_t)b * A.max_pages;
  // The page of the warp's chunk first + g + all_warps * lane: it has no more
  // than 32. Without a window before the length is known, where there may be one.
  auto look_up = [&](int first) {
    const long long p = ((long long)first + g + (long long)all_warps * lane) >> (A.page_log2 - 4);
    return p < A.max_pages ? __ldcg(table + p) : -1;
  };
  int ids = A.window > 0 ? -1 : look_up(0);
  const int L = A.seq_lens[b];
  const bool none = L < A.n_new || L > A.Lmax;       // an unused slot, or a bad length
  const int P0 = L - A.n_new, first = A.window > 0 && !none ? max(0, P0 - A.window + 1) / kFewKeys : 0;
  if (A.window > 0 && !none) ids = look_up(first);
  const int chunks = none ? 0 : (L + kFewKeys - 1) / kFewKeys - first;
  const int mine = min(chunks > g ? (chunks - g + all_warps - 1) / all_warps : 0, 32);

  // ---- this warp's chunks on their way ----
  const uint32_t ring = smem + warp * S::kWarpBytes;
  auto fill = [&](int k) {
    if (k < mine) {
      const int id = __shfl_sync(0xffffffffu, ids, k);
      const int j0 = (first + g + all_warps * k) * kFewKeys;
      const bool good = (unsigned)id < (unsigned)A.n_pages;     // (else its rows count as zeros)
      const size_t row0 = good ? ((size_t)id << A.page_log2) + (j0 & (page - 1)) : 0;
      const uint32_t to = ring + (k % S::kStages) * 2 * S::kChunk;
      constexpr int kStep = 32 / S::kPieces;                    // rows that the warp copies at a time
      const int r0 = lane / S::kPieces, c = lane % S::kPieces;
      const size_t at = ((row0 + r0) * A.Hkv + h) * kD + c * 8, step = (size_t)kStep * A.Hkv * kD;
      const __nv_bfloat16 *ks = A.k + at, *vs = A.v + at;
#pragma unroll
      for (int r = r0; r < kFewKeys + r0; r += kStep, ks += step, vs += step) {
        const bool take = good && j0 + r < L;                   // (else the address is not read)
        const uint32_t dst = to + r * S::kRowBytes + ((c ^ (r & 7)) << 4);
        cp_async16(dst, take ? ks : A.k, take);
        cp_async16(dst + S::kChunk, take ? vs : A.v, take);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < S::kStages - 1; ++k) fill(k);

  // ---- queries, as A operands: rows lane / 4 and 8 further, dims 2 (lane % 4) and 8 further ----
  uint32_t q[kD / 16][4];
  int idx[2];                          // new position of each row
  float slope[2], dep[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = x * 8 + lane / 4, rr = min(r, R - 1), i = rr / A.G, head = h * A.G + rr % A.G;
    idx[x] = i;
    slope[x] = kExtra && A.slopes ? A.slopes[head] * kLog2e : 0.f;
    dep[x] = (float)(A.tree ? A.depth[i] : i);
    const uint32_t* src =
        reinterpret_cast<const uint32_t*>(A.q + ((size_t)b * A.n_new + i) * A.q_stride + (size_t)head * kD) + lane % 4;
#pragma unroll
    for (int t = 0; t < kD / 16; ++t) {
      q[t][x] = r < R && !none ? __ldcg(src + 8 * t) : 0u;
      q[t][x + 2] = r < R && !none ? __ldcg(src + 8 * t + 4) : 0u;
    }
  }

  float o[kD / 8][4], m_ref[2], l[2];
#pragma unroll
  for (int t = 0; t < kD / 8; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    m_ref[x] = -INFINITY;
    l[x] = 0.f;
  }
  // Whether the position of the thread's row x sees cache row j.
  auto sees = [&](int x, int j) {
    const int i = idx[x], a = j - P0;
    if (j >= L) return false;
    const int d = A.tree && a >= 0 ? A.depth[a] : a;           // where it stands, from the first new one
    if (A.window > 0 && (int)dep[x] - d >= A.window) return false;
    if (a < 0) return true;
    return A.tree ? ((A.anc[i] >> a) & 1u) != 0 : a <= i;
  };
  const int clean_hi = P0 + 1;         // chunks that end here or before, and begin at clean_lo or behind,
  const int clean_lo = A.window > 0 ? P0 + A.max_depth - A.window + 1 : 0;      // are seen whole by every row
  for (int k = 0; k < mine; ++k) {
    cp_async_wait<S::kStages - 2>();
    __syncwarp();
    fill(k + S::kStages - 1);          // into the place that the last chunk left
    const uint32_t kb = ring + (k % S::kStages) * 2 * S::kChunk, vb = kb + S::kChunk;
    const int j0 = (first + g + all_warps * k) * kFewKeys;
    const bool clean = j0 + kFewKeys <= clean_hi && j0 >= clean_lo;
    // ---- scores: rows x 16 keys ----
    float s[2][4];
#pragma unroll
    for (int y = 0; y < 2; ++y) s[y][0] = s[y][1] = s[y][2] = s[y][3] = 0.f;
    const int kr = ((lane >> 4) << 3) + (lane & 7), kc = (lane >> 3) & 1;
#pragma unroll
    for (int t = 0; t < kD / 16; ++t) {
      uint32_t f[4];
      ldsm4(f, kb + kr * S::kRowBytes + (((2 * t + kc) ^ (kr & 7)) << 4));
      mma_16816(s[0], q[t], f[0], f[1]);
      mma_16816(s[1], q[t], f[2], f[3]);
    }
    // ---- exponents, masks, references, probabilities ----
    uint32_t p[4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {              // of row lane / 4, or 8 further: keys 2 (lane % 4) (+ 1, + 8, + 9)
      float y[4] = {s[0][2 * x], s[0][2 * x + 1], s[1][2 * x], s[1][2 * x + 1]};
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int j = j0 + 2 * (lane % 4) + (z & 1) + (z & 2) * 4;
        float bias = 0.f;
        if (kExtra && A.slopes) {
          int a = j - P0;
          if (A.tree && a >= 0) a = A.depth[min(a, A.n_new - 1)];
          bias = slope[x] * ((float)a - dep[x]);
        }
        if (kExtra && A.cap > 0.f)
          y[z] = capped(y[z] * (A.scale * A.cap_exp), A.cap * kLog2e, A.cap * kLog2e + bias);
        else
          y[z] = __fadd_rn(__fmul_rn(y[z], A.scale * kLog2e), bias);      // rounded, as its reference will be
        if (!clean && !sees(x, j)) y[z] = -INFINITY;
      }
      float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const bool up = top > m_ref[x] + kHeadroom;
      if (__builtin_expect(__any_sync(0xffffffffu, up), 0)) {
        const float alpha = up ? ex2(m_ref[x] - top) : 1.f;
        if (up) m_ref[x] = top;
        l[x] *= alpha;
#pragma unroll
        for (int t = 0; t < kD / 8; ++t) {
          o[t][2 * x] *= alpha;
          o[t][2 * x + 1] *= alpha;
        }
      }
      const float ref = m_ref[x] == -INFINITY ? 0.f : m_ref[x];
#pragma unroll
      for (int z = 0; z < 4; ++z) y[z] = ex2(y[z] - ref);
      const uint32_t lo = pack2<false>(y[0], y[1]), hi = pack2<false>(y[2], y[3]);
      l[x] += (__uint_as_float(lo << 16) + __uint_as_float(lo & 0xffff0000u)) +
              (__uint_as_float(hi << 16) + __uint_as_float(hi & 0xffff0000u));
      p[x] = lo;
      p[x + 2] = hi;
    }
    if (!clean) {
      // Values that are no numbers would pass a zero probability: they are
      // added where they are seen, and stay out of the product.
      bool odd = false;
      for (int e = lane; e < kFewKeys * S::kPieces; e += 32) {
        const uint4 v = lds128(vb + e * 16);
        odd |= not_finite2(v.x) || not_finite2(v.y) || not_finite2(v.z) || not_finite2(v.w);
      }
      if (__builtin_expect(__any_sync(0xffffffffu, odd), 0)) {
#pragma unroll
        for (int t = 0; t < kD / 8; ++t)
          for (int r = 0; r < kFewKeys; ++r) {
            const uint32_t two = lds32(vb + r * S::kRowBytes + ((t ^ (r & 7)) << 4) + (lane % 4) * 4);
            if (!not_finite2(two)) continue;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const float x = __uint_as_float(z ? two & 0xffff0000u : two << 16);
              if (fabsf(x) < INFINITY) continue;
#pragma unroll
              for (int y = 0; y < 2; ++y)
                if (sees(y, j0 + r)) o[t][2 * y + z] += x;
            }
          }
        __syncwarp();
        for (int e = lane; e < kFewKeys * S::kPieces; e += 32) {
          const uint4 v = lds128(vb + e * 16);
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if ((w[x] & 0x7f80u) == 0x7f80u) w[x] &= 0xffff0000u;
            if ((w[x] & 0x7f800000u) == 0x7f800000u) w[x] &= 0x0000ffffu;
          }
          sts128(vb + e * 16, w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
      }
    }
    // ---- output += probabilities x values ----
    const int vr = (((lane >> 3) & 1) << 3) + (lane & 7), vc = lane >> 4;
#pragma unroll
    for (int t = 0; t < kD / 16; ++t) {
      uint32_t f[4];
      ldsm4_t(f, vb + vr * S::kRowBytes + (((2 * t + vc) ^ (vr & 7)) << 4));
      mma_16816(o[2 * t], p, f[0], f[1]);
      mma_16816(o[2 * t + 1], p, f[2], f[3]);
    }
  }
  cp_async_wait<0>();
  __syncwarp();

  // ---- the warps' parts, [rows][kD] fp32 each where its ring was, then the CTAs' ----
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = x * 8 + lane / 4;
    float sum = l[x];
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (lane % 4 == 0) warp_ml[warp][r] = make_float2(m_ref[x], sum);
    if (r < R)
#pragma unroll
      for (int t = 0; t < kD / 8; ++t)
        sts64(ring + (r * kD + t * 8 + (lane % 4) * 2) * 4, __float_as_uint(o[t][2 * x]),
              __float_as_uint(o[t][2 * x + 1]));
  }
  __syncthreads();
  for (int e = threadIdx.x; e < R * (kD / 4); e += kThreads) {
    const int r = e / (kD / 4);
    float M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, warp_ml[w][r].x);
    const float ref = M == -INFINITY ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float wgt = ex2(warp_ml[w][r].x - ref);
      const float4 v = lds128f(smem + w * S::kWarpBytes + e * 16);
      sum = fmaf(warp_ml[w][r].y, wgt, sum);
      acc.x = fmaf(v.x, wgt, acc.x);
      acc.y = fmaf(v.y, wgt, acc.y);
      acc.z = fmaf(v.z, wgt, acc.z);
      acc.w = fmaf(v.w, wgt, acc.w);
    }
    st_shared_v4(smem + e * 16, acc.x, acc.y, acc.z, acc.w);      // (nobody else reads or writes these)
    if (e % (kD / 4) == 0) cta_ml[r] = make_float2(M, sum);
  }
  sync_ctas();
  // rows dealt out over the CTAs, four dims a thread
  constexpr int kLanes = kD / 4;
  for (int r = rank * (kThreads / kLanes) + threadIdx.x / kLanes; r < R; r += ctas * (kThreads / kLanes)) {
    const int d = threadIdx.x % kLanes * 4;
    float2 ml[kFewMost];
    float4 v[kFewMost];
#pragma unroll
    for (int c = 0; c < kFewMost; ++c) {
      ml[c] = make_float2(-INFINITY, 0.f);
      v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c >= ctas) continue;
      const uint32_t at = mapa_shared(smem_u32(&cta_ml[r]), c);
      ml[c] = make_float2(ld_cluster_f32(at), ld_cluster_f32(at + 4));
      v[c] = ld_cluster_v4(mapa_shared(smem + (r * kD + d) * 4, c));
    }
    float M = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kFewMost; ++c) M = fmaxf(M, ml[c].x);
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int c = 0; c < kFewMost; ++c) {
      const float wgt = ex2(ml[c].x - ref);
      sum = fmaf(ml[c].y, wgt, sum);
      acc.x = fmaf(v[c].x, wgt, acc.x);
      acc.y = fmaf(v[c].y, wgt, acc.y);
      acc.z = fmaf(v[c].z, wgt, acc.z);
      acc.w = fmaf(v[c].w, wgt, acc.w);
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);       // NaN stays
    uint2* const to = reinterpret_cast<uint2*>(
        A.out + (((size_t)b * A.n_new + r / A.G) * A.Hq + (size_t)h * A.G + r % A.G) * kD + d);
    *to = make_uint2(pack2<false>(acc.x * inv, acc.y * inv), pack2<false>(acc.z * inv, acc.w * inv));
  }
  sync_ctas();                                   // nobody's shared memory goes while it is read
}

template <int kD, bool kExtra>
cudaError_t launch_few(const FewLaunch& A, cudaStream_t stream) {
  using S = FewShape<kD>;
  static std::atomic<int> smem_set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !smem_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(few_attn_kernel<kD, kExtra>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) smem_set[dev].store(1, std::memory_order_release);
  }
  const int tiles = A.B * A.Hkv + 1, ctas = cache_attn_few_ctas(tiles, kD);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * ctas));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
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
  return cudaLaunchKernelEx(&cfg, few_attn_kernel<kD, kExtra>, A, ctas);
}

template <int kD>
cudaError_t launch_few_dim(const FewLaunch& A, cudaStream_t stream) {
  return A.cap > 0.f || A.slopes ? launch_few<kD, true>(A, stream) : launch_few<kD, false>(A, stream);
}

}  // namespace cache_attn

cudaError_t launch_cache_attention_few(const CacheAttnLaunch& A, int D, const void* k_pages, cudaStream_t stream) {
  cache_attn::FewLaunch F;
  F.B = A.B;
  F.n_new = A.n_new;
  F.Hq = A.Hq;
  F.Hkv = A.Hkv;
  F.G = A.G;
  F.Lmax = A.Lmax;
  F.window = A.window;
  F.tree = A.tree;
  F.max_depth = A.max_depth;
  F.max_pages = A.max_pages;
  F.page_log2 = A.page_log2;
  F.n_pages = A.n_pages;
  F.scale = A.scale;
  F.cap = A.cap;
  F.cap_exp = A.cap_exp;
  F.q_stride = A.q_stride;
  F.q = A.q;
  F.k = static_cast<const __nv_bfloat16*>(k_pages);
  F.v = static_cast<const __nv_bfloat16*>(A.v);
  F.slopes = A.slopes;
  F.seq_lens = A.seq_lens;
  F.table = A.table;
  F.out = A.out;
  F.status = A.status;
  for (int i = 0; i < kCacheAttnFewRows; ++i) {
    const bool node = A.tree && i < A.n_new;
    F.anc[i] = node ? (uint16_t)A.anc[i][0] : 0;
    F.depth[i] = node ? A.depth[i] : 0;
  }
  switch (D) {
    case 64: return cache_attn::launch_few_dim<64>(F, stream);
    case 128: return cache_attn::launch_few_dim<128>(F, stream);
    case 256: return cache_attn::launch_few_dim<256>(F, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace specdec
