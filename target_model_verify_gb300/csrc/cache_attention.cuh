// Verify-step attention with caps, distance biases, windows and token trees,
// over a bf16 cache or over an e4m3 cache with block scales.
//
// For new position i (row r = i * G + gq of KV head h) and cache row j:
//   s_rj = scale * q_r . k_j            (k_j = s_k code_j for an e4m3 cache)
//   s_rj = cap * tanh(s_rj / cap)       when a cap is set
//   x_rj = log2(e) * (s_rj - slope_h * (pos_i - pos_j))
//   o_r  = sum_j 2^x_rj v_j / sum_j 2^x_rj   over the rows j that i sees
// with one pass over the cache, the running maximum and sum of the softmax
// in fp32. The scale of an e4m3 value block enters the exponent: with
// y_rj = x_rj + log2(s_v), o = sum 2^(y - M) code_j / sum (2^(y - M) / s_v),
// M the running maximum of y, so weights of every block share one range.
//
// Bound: HBM (each K and V row is read once per group of up to 64 query
// rows; R = n_new * G query rows give 2 R flops per cache byte at 16 bits
// and 4 R at 8).
//
// Schedule. The (sequence, KV head, row group) tiles, each a run of cache
// blocks as long as its own sequence (or window), are laid end to end and
// the run of blocks is cut into equal parts, one per CTA, on the device from
// seq_lens, so ragged batches keep every SM busy to the end. A tile that
// lies inside one part is finished by its CTA; the others leave (maximum,
// sum, unnormalised output) partials that combine_kernel merges.
//
// CTA: one producer thread feeds a ring of slots, alternately a block of K
// and a block of V (TMA boxes of up to 128 bytes x kBlk rows, swizzled);
// four consumer warps each take a quarter of the block's keys for S = Q K^T,
// exchange row maxima and the probabilities through shared memory, and each
// take a quarter of the head's dims for O += P V. So every K and V byte is
// read from shared memory (and, for e4m3, widened to f16) once per CTA
// whatever the number of query rows, and the output needs no merge between
// warps. Contractions are mma.sync m16n8k16 with fp32 accumulation, e4m3
// codes widened to f16 (exact) in registers; queries enter as f16 scaled by
// a power of two per row (exact down to 2^-28 of the row's maximum), so the
// only rounding before the output is that of the probabilities: to f16 (11
// bits) over an e4m3 cache, and to bf16 over a bf16 one, whose values need
// its range.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "kernels.h"

namespace specdec {
namespace cache_attn {

constexpr int kConsumers = 4;                  // warps that compute
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr unsigned long long kDrainNs = 1000000000ull;

template <bool kE4m3, int kD, int kMt>
struct Shape {
  static constexpr int kElem = kE4m3 ? 1 : 2;
  // keys per block: 16 KB of K at head dim 128 either way
  static constexpr int kBlk = cache_attn_block(kE4m3, kD);
  static constexpr int kRowBytes = kD * kElem;
  static constexpr int kPanelBytes = kRowBytes < 128 ? kRowBytes : 128;   // one TMA box row
  static constexpr int kPanels = kRowBytes / kPanelBytes;
  static constexpr int kSlotBytes = kBlk * kRowBytes;
  static constexpr int kNt = kBlk / kConsumers / 8;       // key n-tiles per warp in Q K^T
  static constexpr int kKs = kD / 16;                     // k steps of Q K^T
  static constexpr int kDw = kD / kConsumers;             // dims per warp in P V
  static constexpr int kNd = kDw / 8;                     // dim n-tiles per warp in P V
  static constexpr int kKk = kBlk / 16;                   // k steps of P V
  static constexpr int kRows = 16 * kMt;
  static constexpr int kQBytes = kMt * kKs * 512;         // fragment order
  static constexpr int kPBytes = kMt * kKk * 512;
  // row tables: reduction [kRows][4], position, index, scale, slope; tree: 128 x (4 words + depth)
  static constexpr int kTabBytes = kRows * 16 + 4 * kRows * 4 + 128 * 16 + 128 * 4;
  static constexpr int kFixed = 1024 + kQBytes + kPBytes + kTabBytes + 256;
  // two CTAs per SM (228 KB, 1 KB reserved each)
  static constexpr int kSlots = (113 * 1024 - kFixed) / kSlotBytes < 8
                                    ? (113 * 1024 - kFixed) / kSlotBytes : 8;
  static constexpr int kSmem = kFixed + kSlots * kSlotBytes;
  static_assert(kSlots >= 2, "a K and a V block must fit");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void lds64(uint32_t a, uint32_t& x, uint32_t& y) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(a));
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// d += a (16 x 16) b (16 x 8); f16 operands for an e4m3 cache, bf16 otherwise.
template <bool kF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// Two e4m3 codes (16 bits) to two f16 values; every e4m3 value is an f16 value.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return h;
}
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  lo = e4m3x2_to_f16x2((uint16_t)w);
  hi = e4m3x2_to_f16x2((uint16_t)(w >> 16));
}
template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kF16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tmap, uint32_t bar,
                                            int x, int y, int z, int w, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"((uint64_t)tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > kDrainNs) return false;
  return true;
}

// Blocks of kBlk cache rows that a sequence of L rows reads, and the first
// of them: all rows, or those inside the window of the first new position
// (the one that sees furthest back). A length of 0 marks an unused batch
// slot; *bad reports lengths that the cache cannot hold.
template <int kBlk>
__device__ __forceinline__ int seq_blocks(const CacheAttnLaunch& A, int L, int& first, bool& bad) {
  bad = L != 0 && (L < A.n_new || L > A.Lmax);
  first = 0;
  if (L == 0 || bad) return 0;
  if (A.window > 0) first = max(0, L - A.n_new - A.window + 1) / kBlk;
  return (L + kBlk - 1) / kBlk - first;
}

// The part of the block run that CTA c of n takes.
__device__ __forceinline__ long long part_begin(long long total, int c, int n) {
  return total * c / n;
}

// One warp: the number of block units in the batch, and where unit `at` lies:
// sequence b and offset inside it (b = B when at >= total).
template <int kBlk>
__device__ __forceinline__ long long total_units(const CacheAttnLaunch& A, int lane, bool& any_bad) {
  long long sum = 0;
  bool bad_seen = false;
  for (int b = lane; b < A.B; b += 32) {
    int first;
    bool bad;
    sum += seq_blocks<kBlk>(A, A.seq_lens[b], first, bad);
    bad_seen |= bad;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  any_bad = __any_sync(0xffffffffu, bad_seen);
  return sum * A.Hkv * A.n_groups;
}
template <int kBlk>
__device__ __forceinline__ void locate_unit(const CacheAttnLaunch& A, int lane, long long at, int& b_out,
                                            long long& off_out) {
  const long long per = (long long)A.Hkv * A.n_groups;
  long long before = 0;
  b_out = A.B;
  off_out = 0;
  for (int b0 = 0; b0 < A.B; b0 += 32) {
    const int b = b0 + lane;
    int first;
    bool bad;
    const long long mine = b < A.B ? per * seq_blocks<kBlk>(A, A.seq_lens[b], first, bad) : 0;
    long long run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, at < before + run);
    if (hit) {
      const int l = __ffs(hit) - 1;
      b_out = b0 + l;
      off_out = at - before - __shfl_sync(0xffffffffu, run - mine, l);
      return;
    }
    before += __shfl_sync(0xffffffffu, run, 31);
  }
}

// Walks the tiles of a part: (b, h, group) and the block range inside each.
template <int kBlk>
struct Walk {
  int b, h, g;        // tile
  int blk, n_here;    // first block inside the tile, blocks of this part
  int nb, first, L;   // the tile's blocks, its first cache block, its length
  long long u, end;

  __device__ __forceinline__ void load(const CacheAttnLaunch& A) {
    bool bad;
    L = A.seq_lens[b];
    nb = seq_blocks<kBlk>(A, L, first, bad);
  }
  __device__ __forceinline__ void start(const CacheAttnLaunch& A, int b0, long long off, long long u0,
                                        long long u1) {
    u = u0;
    end = u1;
    b = b0;
    if (u >= end) return;
    load(A);
    blk = (int)(off % nb);
    const int t = (int)(off / nb);
    g = t % A.n_groups;
    h = t / A.n_groups;
    n_here = (int)min((long long)(nb - blk), end - u);
  }
  __device__ __forceinline__ bool done() const { return u >= end; }
  __device__ __forceinline__ void next(const CacheAttnLaunch& A) {
    u += n_here;
    if (u >= end) return;
    blk = 0;
    if (++g == A.n_groups) {
      g = 0;
      if (++h == A.Hkv) {
        h = 0;
        do {
          ++b;
          load(A);
        } while (nb == 0);
      }
    }
    n_here = (int)min((long long)nb, end - u);
  }
};

template <bool kE4m3, int kD, int kMt, bool kExtra>
__global__ void __launch_bounds__(kThreads, 2)
    cache_attn_kernel(const __grid_constant__ CacheAttnLaunch A, const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v) {
  using S = Shape<kE4m3, kD, kMt>;
  constexpr int kBlk = S::kBlk, kNt = S::kNt, kNd = S::kNd;
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t slot0 = (raw + 1023u) & ~1023u;
  const uint32_t qs = slot0 + S::kSlots * S::kSlotBytes;
  const uint32_t ps = qs + S::kQBytes;
  const uint32_t red = ps + S::kPBytes;                  // [kRows][4] fp32
  const uint32_t tab = red + S::kRows * 16;              // pos, index, scale, slope: [kRows] each
  const uint32_t tree = tab + 4 * S::kRows * 4;          // [128][4] ancestor words, then depth [128]
  const uint32_t bars = tree + 128 * 16 + 128 * 4;
  auto full_bar = [&](int s) { return bars + 8u * (uint32_t)s; };
  auto empty_bar = [&](int s) { return bars + 8u * (uint32_t)(S::kSlots + s); };
  uint8_t* gen = smem_raw - raw;                         // generic address of a shared offset
  volatile int* abort = reinterpret_cast<volatile int*>(gen + bars + 16 * S::kSlots);
  volatile int* shared_b = abort + 1;
  volatile long long* shared_u = reinterpret_cast<volatile long long*>(gen + bars + 16 * S::kSlots + 8);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), kConsumers);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (A.tree) {
    for (int e = threadIdx.x; e < A.n_new; e += kThreads) {
      sts128(tree + e * 16, A.anc[e][0], A.anc[e][1], A.anc[e][2], A.anc[e][3]);
      sts32(tree + 128 * 16 + e * 4, A.depth[e]);
    }
  }
  grid_dependency_wait();
  if (warp == 0) {
    bool any_bad;
    const long long total = total_units<kBlk>(A, lane, any_bad);
    const long long u0 = part_begin(total, blockIdx.x, gridDim.x);
    const long long u1 = part_begin(total, blockIdx.x + 1, gridDim.x);
    int b0 = A.B;
    long long off = 0;
    if (u0 < u1) locate_unit<kBlk>(A, lane, u0, b0, off);
    if (lane == 0) {
      *shared_b = b0;
      shared_u[0] = off;
      shared_u[1] = u0;
      shared_u[2] = u1;
      if (blockIdx.x == 0) *A.status = any_bad ? SPECDEC_ERR_INVALID_ARG : SPECDEC_OK;
    }
  }
  __syncthreads();
  Walk<kBlk> w;
  w.start(A, *shared_b, shared_u[0], shared_u[1], shared_u[2]);
  const long long part0 = shared_u[1];

  uint32_t issued_mask = 0, issued_phase = 0;
  if (warp == kConsumers) {
    // ---------------------------------------------------------- producer --
    if (lane == 0) {
      const uint64_t pol = policy_evict_first();
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (; ok && !w.done(); w.next(A)) {
        for (int i = 0; ok && i < 2 * w.n_here; ++i) {
          if (!mbar_wait(empty_bar(s), ph ^ 1u, abort, A.status)) {
            ok = false;
            break;
          }
          const int j0 = (w.first + w.blk + (i >> 1)) * kBlk;
          mbar_arrive_expect_tx(full_bar(s), (uint32_t)S::kSlotBytes);
          const uint32_t st = slot0 + (uint32_t)s * S::kSlotBytes;
#pragma unroll
          for (int p = 0; p < S::kPanels; ++p)
            tma_load_4d(st + p * kBlk * S::kPanelBytes, (i & 1) ? &tmap_v : &tmap_k, full_bar(s),
                        p * (S::kPanelBytes / S::kElem), w.h, j0, w.b, pol);
          issued_mask |= 1u << s;
          issued_phase = (issued_phase & ~(1u << s)) | (ph << s);
          if (++s == S::kSlots) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else {
    // --------------------------------------------------------- consumers --
    const int g = lane >> 2, t = lane & 3;
    int s = 0;
    uint32_t ph = 0;
    bool dead = false;      // a wait ran out: keep to the barriers, compute nothing
    auto advance = [&]() {
      if (++s == S::kSlots) {
        s = 0;
        ph ^= 1u;
      }
    };
    // Address of 16-byte chunk c of row r of a slot (the TMA swizzle: chunk
    // index XOR the row inside 8 rows of 128 bytes, or 4 pairs of rows of 64).
    auto chunk = [&](uint32_t base, int r, int c) {
      constexpr int per = S::kPanelBytes / 16;
      const int p = c / per, cc = c % per;
      const int x = S::kPanelBytes == 128 ? (r & 7) : ((r >> 1) & 3);
      return base + (uint32_t)(p * kBlk * S::kPanelBytes + r * S::kPanelBytes + ((cc ^ x) << 4));
    };
    for (; !w.done(); w.next(A)) {
      const int P0 = w.L - A.n_new;              // cache row (and position) of the first new row
      const int row_base = w.g * A.group_rows;
      const int rows_here = min(A.group_rows, A.R - row_base);
      // ---- queries into fragment order, with the rows' tables ----
      constexpr int kCh = kD / 8;                // 16-byte chunks of a query row
      for (int e = threadIdx.x; e < S::kRows * kCh; e += 32 * kConsumers) {
        const int r = e / kCh, c = e % kCh;
        uint4 val = make_uint4(0u, 0u, 0u, 0u);
        int i = 0, gq = 0;
        if (r < rows_here) {
          i = (row_base + r) / A.G;
          gq = (row_base + r) % A.G;
          val = __ldg(reinterpret_cast<const uint4*>(A.q + ((size_t)w.b * A.n_new + i) * A.q_stride +
                                                     (size_t)(w.h * A.G + gq) * kD + c * 8));
        }
        const uint32_t wv[4] = {val.x, val.y, val.z, val.w};
        uint32_t out[4];
        float q_scale = 1.f;
        if constexpr (kE4m3) {
          float f[8], amax = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[2 * k] = __uint_as_float(wv[k] << 16);
            f[2 * k + 1] = __uint_as_float(wv[k] & 0xffff0000u);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float a = fabsf(f[k]);
            if (a < INFINITY) amax = fmaxf(amax, a);
          }
          // the row's kCh lanes are neighbours in the warp
#pragma unroll
          for (int o = kCh / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // amax -> [2^14, 2^15): the exponent field moves to 127 + 14
          const int ex = (int)(__float_as_uint(amax) >> 23);
          const int down = amax > 0.f ? min(max(ex - 141, -100), 113) : 0;
          const float mul = __uint_as_float((uint32_t)(127 - down) << 23);
          q_scale = __uint_as_float((uint32_t)(127 + down) << 23);
#pragma unroll
          for (int k = 0; k < 4; ++k) out[k] = pack2<true>(f[2 * k] * mul, f[2 * k + 1] * mul);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) out[k] = wv[k];
        }
        const int mt = r >> 4, rr = r & 15;
        const uint32_t hi_row = rr >= 8 ? 4u : 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // dims 8c + 2k, +1: step, lane column and word of the A fragment
          int step, tt, word;
          if constexpr (kE4m3) {
            // lane column tt owns whole 16-byte code chunks (see the K loads)
            const int cc = c >> 1;
            const int ci = kD == 64 ? 0 : (cc & 1) + 2 * (cc >> 3);
            tt = kD == 64 ? cc : (cc & 7) >> 1;
            step = ci * 4 + (c & 1) * 2 + (k >> 1);
            word = (k & 1) * 2;
          } else {
            step = c >> 1;
            tt = k;
            word = (c & 1) * 2;
          }
          sts32(qs + (uint32_t)((mt * S::kKs + step) * 32 + (rr & 7) * 4 + tt) * 16 + word * 4 + hi_row,
                out[k]);
        }
        if (c == 0) {
          const int dep = A.tree ? (int)lds32(tree + 128 * 16 + i * 4) : i;
          sts32(tab + r * 4, (uint32_t)dep);
          sts32(tab + S::kRows * 4 + r * 4, (uint32_t)i);
          sts32(tab + 2 * S::kRows * 4 + r * 4, __float_as_uint(A.scale * q_scale));
          if (kExtra)
            sts32(tab + 3 * S::kRows * 4 + r * 4,
                  __float_as_uint(A.slopes && r < rows_here ? A.slopes[w.h * A.G + gq] * kLog2e : 0.f));
        }
      }
      named_bar_sync(1, 32 * kConsumers);

      float m_run[kMt][2], l_run[kMt][2], o[kMt][kNd][4], cq[kMt][2];
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          m_run[mt][h] = -INFINITY;
          l_run[mt][h] = 0.f;
          cq[mt][h] = __uint_as_float(lds32(tab + 2 * S::kRows * 4 + (mt * 16 + g + 8 * h) * 4));
        }
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int n = 0; n < kNd; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;

      // Whether row r of the group sees cache row j (j in [0, L) or beyond).
      auto sees = [&](int r, int j) {
        if (j >= w.L) return false;
        const int dep = (int)lds32(tab + r * 4);
        if (j < P0) return A.window <= 0 || P0 + dep - j < A.window;
        const int a = j - P0, i = (int)lds32(tab + S::kRows * 4 + r * 4);
        if (!A.tree) return a <= i && (A.window <= 0 || i - a < A.window);
        if (!((lds32(tree + i * 16 + (a >> 5) * 4) >> (a & 31)) & 1u)) return false;
        return A.window <= 0 || dep - (int)lds32(tree + 128 * 16 + a * 4) < A.window;
      };

      const int key_w = warp * (kBlk / kConsumers);      // this warp's first key in a block
      const float* ksp = nullptr;
      const float* vsp = nullptr;
      float sk_next = 1.f, sv_next = 1.f;
      auto load_scales = [&](int j) {                    // of the 32-row block that holds row j
        if constexpr (kE4m3) {
          if (j < w.L) {
            sk_next = __ldg(ksp + j / SPECDEC_KV8_BLOCK);
            sv_next = __ldg(vsp + j / SPECDEC_KV8_BLOCK);
          } else {
            sk_next = sv_next = 1.f;
          }
        }
      };
      if constexpr (kE4m3) {
        const size_t so = ((size_t)w.b * A.Hkv + w.h) * A.n_scale;
        ksp = A.k_scale + so;
        vsp = A.v_scale + so;
      }
      load_scales((w.first + w.blk) * kBlk + key_w);

      for (int ib = 0; ib < w.n_here; ++ib) {
        const int j0 = (w.first + w.blk + ib) * kBlk;
        const float sk = sk_next, sv = sv_next;
        if (ib + 1 < w.n_here) load_scales(j0 + kBlk + key_w);
        const bool clean = j0 + kBlk <= P0 + 1 &&
                           (A.window <= 0 || j0 > P0 + A.max_depth - A.window);
        // ---- S = Q K^T over this warp's keys ----
        float sc[kMt][kNt][4];
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int n = 0; n < kNt; ++n) sc[mt][n][0] = sc[mt][n][1] = sc[mt][n][2] = sc[mt][n][3] = 0.f;
        if (!dead && !mbar_wait(full_bar(s), ph, abort, A.status)) dead = true;
        if (!dead) {
          const uint32_t kb = slot0 + (uint32_t)s * S::kSlotBytes;
          if constexpr (kE4m3) {
            // Lane (g, t) takes key g of every n-tile, and of it whole 16-byte
            // chunks: 2t, 2t + 1 of every 128-byte panel (t at 64 dims). The
            // dims of a k step are spread over the lanes accordingly, alike
            // for Q; eight lanes of a load phase then hit all 32 banks.
#pragma unroll
            for (int ci = 0; ci < kD / 64; ++ci) {
              uint4 kw[kNt];
#pragma unroll
              for (int n = 0; n < kNt; ++n)
                kw[n] = lds128(chunk(kb, key_w + n * 8 + g,
                                     kD == 64 ? t : 2 * t + (ci & 1) + 8 * (ci >> 1)));
#pragma unroll
              for (int k4 = 0; k4 < 4; ++k4) {
                uint4 a[kMt];
#pragma unroll
                for (int mt = 0; mt < kMt; ++mt)
                  a[mt] = lds128(qs + (uint32_t)((mt * S::kKs + ci * 4 + k4) * 32 + lane) * 16);
#pragma unroll
                for (int n = 0; n < kNt; ++n) {
                  const uint32_t word = k4 == 0 ? kw[n].x : k4 == 1 ? kw[n].y : k4 == 2 ? kw[n].z : kw[n].w;
                  uint32_t b0, b1;
                  widen4(word, b0, b1);
#pragma unroll
                  for (int mt = 0; mt < kMt; ++mt) mma16816<true>(sc[mt][n], a[mt], b0, b1);
                }
              }
            }
          } else {
#pragma unroll
            for (int ks = 0; ks < S::kKs; ++ks) {
              uint4 a[kMt];
#pragma unroll
              for (int mt = 0; mt < kMt; ++mt)
                a[mt] = lds128(qs + (uint32_t)((mt * S::kKs + ks) * 32 + lane) * 16);
#pragma unroll
              for (int n = 0; n < kNt; n += 2) {
                uint32_t r[4];
                ldsm_x4(chunk(kb, key_w + n * 8 + (lane & 7) + ((lane >> 4) << 3),
                              ks * 2 + ((lane >> 3) & 1)), r);
#pragma unroll
                for (int mt = 0; mt < kMt; ++mt) {
                  mma16816<false>(sc[mt][n], a[mt], r[0], r[1]);
                  mma16816<false>(sc[mt][n + 1], a[mt], r[2], r[3]);
                }
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(empty_bar(s));
        }
        advance();

        // ---- exponents, masks, row maxima ----
        const float lv = kE4m3 ? __log2f(sv) : 0.f;
        const float inv_sv = kE4m3 ? rcp(sv) : 1.f;
        float bmax[kMt][2];
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = mt * 16 + g + 8 * h;
            float m = -INFINITY;
            if constexpr (kExtra) {
              const float ck = cq[mt][h] * sk;
              const float slope = __uint_as_float(lds32(tab + 3 * S::kRows * 4 + r * 4));
              const int dep = (int)lds32(tab + r * 4);
#pragma unroll
              for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float y = sc[mt][n][2 * h + e] * ck;
                  // cap * tanh(y / cap) = cap * (1 - 2 / (1 + e^(2 y / cap)))
                  if (A.cap > 0.f) y = A.cap * (1.f - 2.f * rcp(1.f + ex2(y * A.cap_exp)));
                  int pj = j0 + key_w + n * 8 + 2 * t + e;
                  if (A.tree && pj >= P0 && pj < w.L) pj = P0 + (int)lds32(tree + 128 * 16 + (pj - P0) * 4);
                  y = fmaf(y, kLog2e, lv) - slope * (float)(P0 + dep - pj);
                  sc[mt][n][2 * h + e] = y;
                }
            } else {
              const float ck = cq[mt][h] * sk * kLog2e;
#pragma unroll
              for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) sc[mt][n][2 * h + e] = fmaf(sc[mt][n][2 * h + e], ck, lv);
            }
            if (!clean) {
#pragma unroll
              for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (!sees(r, j0 + key_w + n * 8 + 2 * t + e)) sc[mt][n][2 * h + e] = -INFINITY;
            }
#pragma unroll
            for (int n = 0; n < kNt; ++n) m = fmaxf(m, fmaxf(sc[mt][n][2 * h], sc[mt][n][2 * h + 1]));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            bmax[mt][h] = m;
            if (t == 0) sts32(red + r * 16 + warp * 4, __float_as_uint(m));
          }
        named_bar_sync(1, 32 * kConsumers);

        // ---- probabilities to shared memory, in fragment order ----
        bool moved = false;
        float alpha[kMt][2];
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt) {
          float mu[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 m4 = lds128(red + (mt * 16 + g + 8 * h) * 16);
            const float m_new =
                fmaxf(fmaxf(m_run[mt][h], fmaxf(__uint_as_float(m4.x), __uint_as_float(m4.y))),
                      fmaxf(__uint_as_float(m4.z), __uint_as_float(m4.w)));
            mu[h] = m_new == -INFINITY ? 0.f : m_new;          // nothing seen yet
            alpha[mt][h] = ex2(m_run[mt][h] - mu[h]);
            m_run[mt][h] = m_new;
            moved |= alpha[mt][h] != 1.f;
            // f16 probabilities fill the range up to 2^15: small weights keep their bits
            if constexpr (kE4m3) mu[h] -= 15.f;
          }
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
          for (int n = 0; n < kNt; n += 2) {
            uint32_t pk[4];                    // rows g, g + 8 of n-tile n, then of n + 1
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float lo = ex2(sc[mt][n + (x >> 1)][(x & 1) * 2] - mu[x & 1]);
              const float hi = ex2(sc[mt][n + (x >> 1)][(x & 1) * 2 + 1] - mu[x & 1]);
              pk[x] = pack2<kE4m3>(lo, hi);
              // The sum takes bf16 weights as rounded: their error then moves
              // the output by w (v - o) only. The f16 rounding is left out of it.
              const float sum = kE4m3 ? lo + hi
                                      : __uint_as_float(pk[x] << 16) + __uint_as_float(pk[x] & 0xffff0000u);
              if (x & 1) sum1 += sum; else sum0 += sum;
            }
            sts128(ps + (uint32_t)(((key_w / 16 + n / 2) * kMt + mt) * 32 + lane) * 16, pk[0], pk[1], pk[2], pk[3]);
          }
          l_run[mt][0] = fmaf(l_run[mt][0], alpha[mt][0], sum0 * inv_sv);
          l_run[mt][1] = fmaf(l_run[mt][1], alpha[mt][1], sum1 * inv_sv);
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
            for (int n = 0; n < kNd; ++n) {
              o[mt][n][0] *= alpha[mt][0];
              o[mt][n][1] *= alpha[mt][0];
              o[mt][n][2] *= alpha[mt][1];
              o[mt][n][3] *= alpha[mt][1];
            }
        }
        named_bar_sync(1, 32 * kConsumers);

        // ---- O += P V over this warp's dims ----
        if (!dead && !mbar_wait(full_bar(s), ph, abort, A.status)) dead = true;
        if (!dead) {
          const uint32_t vb = slot0 + (uint32_t)s * S::kSlotBytes;
          // Rows past the sequence hold anything and a row that not every
          // query sees may hold an infinity or a NaN, which a zero
          // probability would not silence: both are kept out of the product.
          uint32_t odd = 0;
          auto guard = [&](uint32_t v, int j) {          // values of rows j (low half) and j + 1
            constexpr uint32_t ex = kE4m3 ? 0x7c00u : 0x7f80u;
            if (j >= w.L) v &= 0xffff0000u;
            if (j + 1 >= w.L) v &= 0x0000ffffu;
            if ((v & ex) == ex) {
              v &= 0xffff0000u;
              odd = 1;
            }
            if ((v & (ex << 16)) == (ex << 16)) {
              v &= 0x0000ffffu;
              odd = 1;
            }
            return v;
          };
#pragma unroll
          for (int kk = 0; kk < S::kKk; ++kk) {
            uint4 a[kMt];
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt)
              a[mt] = lds128(ps + (uint32_t)((kk * kMt + mt) * 32 + lane) * 16);
            uint32_t b0[kNd], b1[kNd];
            if constexpr (kE4m3) {
              // Lane (g, t): kNd neighbouring dims of keys 2t, 2t + 1 and
              // 8 further; bytes of the two keys pair up into f16x2.
              const int d0 = warp * S::kDw + g * kNd;
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                const int r0 = kk * 16 + hf * 8 + 2 * t;
                uint32_t x[2], y[2];
                const uint32_t a0 = chunk(vb, r0, d0 >> 4) + (d0 & 15);
                const uint32_t a1 = chunk(vb, r0 + 1, d0 >> 4) + (d0 & 15);
                if constexpr (kNd == 8) {
                  lds64(a0, x[0], x[1]);
                  lds64(a1, y[0], y[1]);
                } else if constexpr (kNd == 4) {
                  x[0] = lds32(a0);
                  y[0] = lds32(a1);
                } else {
                  x[0] = lds16(a0);
                  y[0] = lds16(a1);
                }
                uint32_t(&b)[kNd] = hf ? b1 : b0;
#pragma unroll
                for (int q4 = 0; q4 < (kNd + 3) / 4; ++q4) {
                  widen4(__byte_perm(x[q4], y[q4], 0x5140), b[q4 * 4], b[q4 * 4 + 1]);
                  if constexpr (kNd >= 4)
                    widen4(__byte_perm(x[q4], y[q4], 0x7362), b[q4 * 4 + 2], b[q4 * 4 + 3]);
                }
              }
            } else {
#pragma unroll
              for (int n = 0; n < kNd; n += 2) {
                uint32_t r[4];
                ldsm_x4_t(chunk(vb, kk * 16 + (lane & 7) + (((lane >> 3) & 1) << 3),
                                warp * (S::kDw / 8) + n + (lane >> 4)), r);
                b0[n] = r[0];
                b1[n] = r[1];
                b0[n + 1] = r[2];
                b1[n + 1] = r[3];
              }
            }
            if (!clean) {
#pragma unroll
              for (int n = 0; n < kNd; ++n) {
                b0[n] = guard(b0[n], j0 + kk * 16 + 2 * t);
                b1[n] = guard(b1[n], j0 + kk * 16 + 8 + 2 * t);
              }
            }
#pragma unroll
            for (int n = 0; n < kNd; ++n)
#pragma unroll
              for (int mt = 0; mt < kMt; ++mt) mma16816<kE4m3>(o[mt][n], a[mt], b0[n], b1[n]);
          }
          if (!clean && __any_sync(0xffffffffu, odd)) {
            // Rare: the infinities and NaN left out above, for the rows that see them.
            for (int key = 0; key < kBlk && j0 + key < w.L; ++key) {
#pragma unroll
              for (int n = 0; n < kNd; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int d = kE4m3 ? warp * S::kDw + (2 * t + e) * kNd + n
                                      : warp * S::kDw + n * 8 + 2 * t + e;
                  const int byte = d * S::kElem;
                  const uint32_t at = chunk(vb, key, byte >> 4) + (byte & 15);
                  float v;
                  bool is_odd;
                  if constexpr (kE4m3) {
                    is_odd = (lds8(at) & 0x7fu) == 0x7fu;
                    v = __uint_as_float(0x7fffffffu);
                  } else {
                    const uint32_t u = lds16(at);
                    is_odd = (u & 0x7f80u) == 0x7f80u;
                    v = __uint_as_float(u << 16);
                  }
                  if (!is_odd) continue;
#pragma unroll
                  for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                      const int r = mt * 16 + g + 8 * h;
                      if (r >= rows_here || !sees(r, j0 + key)) continue;
                      const uint32_t pu =
                          lds16(ps + (uint32_t)(((key >> 4) * kMt + mt) * 32 + g * 4 + ((key & 7) >> 1)) * 16 +
                                (h + ((key >> 3) & 1) * 2) * 4 + (key & 1) * 2);
                      const float pv = kE4m3 ? __half2float(__ushort_as_half((unsigned short)pu))
                                             : __uint_as_float(pu << 16);
                      o[mt][n][2 * h + e] += pv * v;
                    }
                }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(empty_bar(s));
        }
        advance();
      }

      // ---- the tile's sums over the warps, then the output or a partial ----
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          l_run[mt][h] += __shfl_xor_sync(0xffffffffu, l_run[mt][h], 1);
          l_run[mt][h] += __shfl_xor_sync(0xffffffffu, l_run[mt][h], 2);
          if (t == 0) sts32(red + (mt * 16 + g + 8 * h) * 16 + warp * 4, __float_as_uint(l_run[mt][h]));
        }
      named_bar_sync(1, 32 * kConsumers);
      const bool whole = w.blk == 0 && w.n_here == w.nb;
      const size_t slot = (size_t)blockIdx.x * 2 + (w.u == part0 ? 0 : 1);
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = mt * 16 + g + 8 * h;
          if (r >= rows_here || dead) continue;
          const uint4 l4 = lds128(red + r * 16);
          const float l = (__uint_as_float(l4.x) + __uint_as_float(l4.y)) +
                          (__uint_as_float(l4.z) + __uint_as_float(l4.w));
          if (whole) {
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // NaN stays
            const int i = (row_base + r) / A.G, gq = (row_base + r) % A.G;
            __nv_bfloat16* dst =
                A.out + (((size_t)w.b * A.n_new + i) * A.Hq + (size_t)w.h * A.G + gq) * kD + warp * S::kDw;
            if constexpr (kE4m3) {
              // dims (2t) kNd .. (2t + 2) kNd - 1 are this lane's
              uint32_t pk[kNd];
#pragma unroll
              for (int n = 0; n < kNd; n += 2) {
                pk[n / 2] = pack2<false>(o[mt][n][2 * h] * inv, o[mt][n + 1][2 * h] * inv);
                pk[kNd / 2 + n / 2] = pack2<false>(o[mt][n][2 * h + 1] * inv, o[mt][n + 1][2 * h + 1] * inv);
              }
              uint32_t* d32 = reinterpret_cast<uint32_t*>(dst + 2 * t * kNd);
              if constexpr (kNd >= 4) {
#pragma unroll
                for (int n = 0; n < kNd; n += 4)
                  *reinterpret_cast<uint4*>(d32 + n) = make_uint4(pk[n], pk[n + 1], pk[n + 2], pk[n + 3]);
              } else {
                *reinterpret_cast<uint2*>(d32) = make_uint2(pk[0], pk[1]);
              }
            } else {
#pragma unroll
              for (int n = 0; n < kNd; ++n)
                *reinterpret_cast<uint32_t*>(dst + n * 8 + 2 * t) =
                    pack2<false>(o[mt][n][2 * h] * inv, o[mt][n][2 * h + 1] * inv);
            }
          } else {
            float* po = A.part_o + (slot * S::kRows + r) * kD + warp * S::kDw;
#pragma unroll
            for (int n = 0; n < kNd; ++n) {
              if constexpr (kE4m3) {
                po[2 * t * kNd + n] = o[mt][n][2 * h];
                po[(2 * t + 1) * kNd + n] = o[mt][n][2 * h + 1];
              } else {
                *reinterpret_cast<float2*>(po + n * 8 + 2 * t) = make_float2(o[mt][n][2 * h], o[mt][n][2 * h + 1]);
              }
            }
            if (warp == 0 && t == 0)
              *reinterpret_cast<float2*>(A.part_ml + (slot * S::kRows + r) * 2) = make_float2(m_run[mt][h], l);
          }
        }
    }
  }
  __syncthreads();   // every role has left its loop
  if (*abort && warp == kConsumers && lane == 0)
    // A wait gave up: let every copy already issued land before the CTA exits.
    for (int s = 0; s < S::kSlots; ++s)
      if (issued_mask & (1u << s)) wait_drain(full_bar(s), (issued_phase >> s) & 1u);
}

// Merges the partials of the tiles that more than one CTA worked on, and
// zeroes the outputs of sequences without blocks. One warp per query row:
// blockIdx.x = tile, blockIdx.y * 8 + warp = row of its group.
template <bool kE4m3, int kD, int kMt>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ CacheAttnLaunch A, int n_ctas) {
  using S = Shape<kE4m3, kD, kMt>;
  __shared__ long long sh_before[8], sh_total[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x;
  const int grp = tile % A.n_groups;
  const int h = tile / A.n_groups % A.Hkv;
  const int b = tile / A.n_groups / A.Hkv;
  grid_dependency_wait();
  long long before = 0, total = 0;
  for (int x = threadIdx.x; x < A.B; x += 256) {
    int first;
    bool bad;
    const int nb = seq_blocks<S::kBlk>(A, A.seq_lens[x], first, bad);
    total += nb;
    if (x < b) before += nb;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) {
    sh_before[warp] = before;
    sh_total[warp] = total;
  }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    before += sh_before[x];
    total += sh_total[x];
  }
  int first;
  bool bad;
  const int nb = seq_blocks<S::kBlk>(A, A.seq_lens[b], first, bad);
  const long long per = (long long)A.Hkv * A.n_groups;
  total *= per;
  const long long u0 = before * per + (long long)(h * A.n_groups + grp) * nb;
  const int r = blockIdx.y * 8 + warp;
  const int rr = grp * A.group_rows + r;
  if (r >= A.group_rows || rr >= A.R) return;
  constexpr int kPer = kD / 32;
  __nv_bfloat16* dst =
      A.out + (((size_t)b * A.n_new + rr / A.G) * A.Hq + (size_t)h * A.G + rr % A.G) * kD + lane * kPer;
  float acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  float inv = 0.f;
  if (nb > 0) {
    // CTA c owns unit u iff part_begin(c) <= u < part_begin(c + 1)
    const int c0 = (int)(((u0 + 1) * n_ctas - 1) / total);
    const int c1 = (int)(((u0 + nb) * n_ctas - 1) / total);
    if (c0 == c1) return;                        // its CTA wrote the output
    float M = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) {
      const long long pb = part_begin(total, c, n_ctas);
      if (pb == part_begin(total, c + 1, n_ctas)) continue;
      const size_t slot = (size_t)c * 2 + (c == c0 && pb != u0 ? 1 : 0);
      M = fmaxf(M, A.part_ml[(slot * S::kRows + r) * 2]);
    }
    M = warp_max(M);
    const float mu = M == -INFINITY ? 0.f : M;
    float l = 0.f;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      const long long pb = part_begin(total, c, n_ctas);
      if (pb == part_begin(total, c + 1, n_ctas)) continue;
      const size_t slot = (size_t)c * 2 + (c == c0 && pb != u0 ? 1 : 0);
      const float2 ml = *reinterpret_cast<const float2*>(A.part_ml + (slot * S::kRows + r) * 2);
      const float wgt = ex2(ml.x - mu);
      l += ml.y * wgt;
      const float* po = A.part_o + (slot * S::kRows + r) * kD + lane * kPer;
#pragma unroll
      for (int k = 0; k < kPer; k += 2) {
        const float2 v = *reinterpret_cast<const float2*>(po + k);
        acc[k] = fmaf(v.x, wgt, acc[k]);
        acc[k + 1] = fmaf(v.y, wgt, acc[k + 1]);
      }
    }
    inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  }
#pragma unroll
  for (int k = 0; k < kPer; k += 2)
    *reinterpret_cast<uint32_t*>(dst + k) = pack2<false>(acc[k] * inv, acc[k + 1] * inv);
}

template <bool kE4m3, int kD, int kMt, bool kExtra>
cudaError_t launch_one(const CacheAttnLaunch& A, const CUtensorMap& tk, const CUtensorMap& tv,
                       cudaStream_t stream) {
  using S = Shape<kE4m3, kD, kMt>;
  static std::atomic<int> smem_set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !smem_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(cache_attn_kernel<kE4m3, kD, kMt, kExtra>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) smem_set[dev].store(1, std::memory_order_release);
  }
  const long long tiles = (long long)A.B * A.Hkv * A.n_groups;
  const long long most = tiles * ((A.Lmax + S::kBlk - 1) / S::kBlk);
  const int grid = (int)(most < kCacheAttnCtas ? most : kCacheAttnCtas);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, cache_attn_kernel<kE4m3, kD, kMt, kExtra>, A, tk, tv);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)tiles, (A.group_rows + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, combine_kernel<kE4m3, kD, kMt>, A, grid);
}

template <bool kE4m3, int kD, int kMt>
cudaError_t launch_extra(const CacheAttnLaunch& A, const CUtensorMap& tk, const CUtensorMap& tv,
                         cudaStream_t stream) {
  return A.cap > 0.f || A.slopes ? launch_one<kE4m3, kD, kMt, true>(A, tk, tv, stream)
                                 : launch_one<kE4m3, kD, kMt, false>(A, tk, tv, stream);
}

// Row tiles per CTA: the fewest of 1, 2 and 4 (2 at 256 dims) that hold a group.
template <bool kE4m3, int kD>
cudaError_t launch_rows(const CacheAttnLaunch& A, const CUtensorMap& tk, const CUtensorMap& tv,
                        cudaStream_t stream) {
  if (A.group_rows <= 16) return launch_extra<kE4m3, kD, 1>(A, tk, tv, stream);
  if constexpr (kD == 256)
    return launch_extra<kE4m3, kD, 2>(A, tk, tv, stream);
  else
    return A.group_rows <= 32 ? launch_extra<kE4m3, kD, 2>(A, tk, tv, stream)
                              : launch_extra<kE4m3, kD, 4>(A, tk, tv, stream);
}

}  // namespace cache_attn
}  // namespace specdec
