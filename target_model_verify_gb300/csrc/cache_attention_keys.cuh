// The cache attention (cache_attention.cuh) over an e4m3 cache of head dim
// 128 for up to 24 query rows per KV head, with the cache on the M side of
// both products.
//
// With few query rows the row-per-lane form pays for 128 of them: its products
// and their operand reads, and widening V to f16, take as long as the cache
// takes to arrive. Here
//   S^T = K Q^T:   M = 128 keys, N = 48: the rows' two e4m3 query terms side
//                  by side (K is read from shared memory once; the terms'
//                  scores are added in registers);
//   O^T += V^T P^T: M = 128 dims, N = 96: the rows' probabilities as four
//                  e5m2 terms, p = t0 + t1 / 8 + t2 / 64 + t3 / 512, with an
//                  accumulator each, and V is multiplied as it lies in the
//                  cache. A term has three significant bits and f16's exponents,
//                  so the four are p rounded to f16, exactly, at every size.
//                  (Three e4m3 terms hold as many bits but end 2^28 below
//                  their top: the small weights beside one dominant key
//                  vanished from outputs whose sum counted them.)
// Lane = key in the softmax, so a row's statistics run over lanes and warps.
// Only its reference (the exponent of p = 2^15, the most of which a term can
// hold eight times the rest) does not follow every maximum: it is set 2^6
// above one when a block's largest p would pass 2^15, and to 2^24 below its
// highest when that would stay below 2^-14, where f16's normal numbers end. So a weight is off by at most 2^-11
// of itself, or below those by half of f16's last step, 2^-25: 2^-34 of the
// row's largest and 2^-11 of the largest among its own 128 rows. (A key that
// takes nearly all of a row's weight, as the first one does in many models,
// leaves the small ones their precision, down to 2^-45 of it.) They go no
// further down, so that sums and outputs stay finite. One barrier per
// block, with votes, finds out whether one has to move; sums stay with the
// keys' threads until the tile ends.
//
// Two CTAs per SM (256 tensor memory columns each) of six warps, so that a
// thread may have 168 registers: 0-3 softmax, 4 loads (K and V blocks,
// queries and row tables, the check of V blocks that not every query sees
// whole), 5 issues both products.
//
// Measured (64 x 4096 rows, 5 positions, 32 query / 8 KV heads): 105 us for
// 543 MB, 5170 GB/s or 0.76 of the copy peak (the other form: 121 us); scores
// of twice and four times the spread 107 and 140 us, where references move and
// are looked at more often. What is left is the start (6 us until the first
// block's products), the first block's pass for its references, the SMs'
// unequal ends and the merge (4 us).
#pragma once

#include "cache_attention.cuh"

namespace specdec {
namespace cache_attn {

constexpr int kKeyThreads = 192;
constexpr int kKeyD = 128, kKeyBlk = 128;
constexpr int kKeyRows = kCacheAttnKeyRows, kKeyLanes = 32;     // query rows, and their tables' and partials' pitch
constexpr int kKeyTerms = 4;
constexpr int kKeyRingK = 2, kKeyRingV = 3;             // blocks of each in flight: V's are held longer
constexpr int kKeySlot = kKeyBlk * kKeyD;
constexpr int kKeyPanel = kKeyBlk * 32, kKeyPanels = kKeyRows / 8;      // [keys][4 terms][8 rows] codes
static_assert(kKeyRows % 8 == 0 && kKeyTerms == 4 && kKeyRows <= kKeyLanes, "eight rows' terms to a panel");
constexpr int kKeyQBytes = 2 * kKeyRows * kKeyD;        // [hi rows, lo rows][dims]
constexpr int kKeyColS = 0, kKeyColO = 128;
// log2: p at the reference; how far above a row's maximum that is set; how far
// below it a block's maximum may lie (kDeep and kReach as in the other form)
constexpr float kBase = 15.f, kLift = 6.f, kFall = 29.f;
// tables per query buffer: of every row its score factor, slope, depth and
// place in the output [32]; of every new position the rows that see it [128]
constexpr int kKeyTab = 4 * kKeyLanes * 4 + 128 * 4;
constexpr int kKeySmem = 1024 + (kKeyRingK + kKeyRingV) * kKeySlot + kKeyPanels * kKeyPanel + 2 * kKeyQBytes +
                         2 * kKeyTab + 8 * kKeyLanes * 4 + 128 * 4 + 64 + 256;
static_assert(2 * (kKeySmem + 1024) <= 228 * 1024, "two CTAs per SM");

// MN-major operand of 32-byte rows (32 codes along N), 32-byte swizzle.
__device__ __forceinline__ uint64_t operand_desc32(uint32_t saddr, uint32_t lead) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(lead >> 4) << 16;
  d |= (uint64_t)((8u * 32) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)6 << 61;
  return d;
}
// A barrier that counts the threads with x.
__device__ __forceinline__ int bar_count(int id, int nthreads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.popc.u32 %0, %2, %3, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "r"(nthreads)
      : "memory");
  return (int)r;
}
__device__ __forceinline__ uint32_t f16x2_to_e5m2x2(uint32_t h) {
  uint16_t c;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
  return c;
}
// (h - code) * 8, elementwise; exact for code the e5m2 rounding of h (whose
// bytes are the upper ones of f16 values), and at most 2^15 for h up to that.
__device__ __forceinline__ uint32_t rest8(uint32_t h, uint32_t code) {
  const uint32_t back = __byte_perm(code, 0, 0x1404);
  const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&back)),
                            __float2half2_rn(8.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&x)[48]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
      "}, [%48];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47"
      "}, [%49];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]),
        "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]),
        "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]), "=r"(x[16]), "=r"(x[17]),
        "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]),
        "=r"(x[24]), "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]),
        "=r"(x[30]), "=r"(x[31]), "=r"(x[32]), "=r"(x[33]), "=r"(x[34]), "=r"(x[35]),
        "=r"(x[36]), "=r"(x[37]), "=r"(x[38]), "=r"(x[39]), "=r"(x[40]), "=r"(x[41]),
        "=r"(x[42]), "=r"(x[43]), "=r"(x[44]), "=r"(x[45]), "=r"(x[46]), "=r"(x[47])
      : "r"(taddr + 0), "r"(taddr + 32)
      : "memory");
}
// Halves the rows a lane carries five times: lane r returns the warp's
// join of row r (rows past the last: `none`).
template <typename Join>
__device__ __forceinline__ float rows_to_lanes(const float (&x)[kKeyRows], int lane, float none, Join join) {
  float y[kKeyLanes];
#pragma unroll
  for (int r = 0; r < kKeyLanes; ++r) y[r] = r < kKeyRows ? x[r] : none;
#pragma unroll
  for (int o = 16, cnt = 16; o; o >>= 1, cnt >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int k = 0; k < cnt; ++k) {
      const float give = up ? y[k] : y[k + cnt], keep = up ? y[k + cnt] : y[k];
      y[k] = join(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  return y[0];
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float m;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
__device__ __forceinline__ float min_or_nan(float a, float b) {
  float m;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

template <bool kExtra>
__global__ void __launch_bounds__(kKeyThreads, 2)
    cache_attn_keys_kernel(const __grid_constant__ CacheAttnLaunch A, const __grid_constant__ CUtensorMap tmap_k,
                           const __grid_constant__ CUtensorMap tmap_v) {
  constexpr int kBlk = kKeyBlk, kD = kKeyD, kRows = kKeyRows, kLanes = kKeyLanes;
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring_k = (raw + 1023u) & ~1023u;
  const uint32_t ring_v = ring_k + kKeyRingK * kKeySlot;
  const uint32_t pb = ring_v + kKeyRingV * kKeySlot;       // probabilities: all terms
  const uint32_t qb = pb + kKeyPanels * kKeyPanel;
  const uint32_t tab = qb + 2 * kKeyQBytes;
  const uint32_t ref = tab + 2 * kKeyTab;                  // references, then factors for what moved
  const uint32_t zeros = ref + 2 * kLanes * 4;             // [32]
  const uint32_t red = zeros + kLanes * 4;                 // [4 warps][32 rows]
  const uint32_t depths = red + 4 * kLanes * 4;            // of the tree's nodes [128]
  const uint32_t marks = depths + 128 * 4;                 // [2 blocks][4 warps][2] rows, see below
  const uint32_t peaks = marks + 64;                       // the rows' highest references
  const uint32_t bars = peaks + kLanes * 4;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  auto k_full = [&](int s) { return bar(s); };
  auto k_empty = [&](int s) { return bar(2 + s); };
  auto s_full = [&](int s) { return bar(4 + s); };
  auto p_full = [&](int s) { return bar(6 + s); };
  auto o_done = [&](int s) { return bar(8 + s); };
  auto q_full = [&](int s) { return bar(10 + s); };
  auto q_empty = [&](int s) { return bar(12 + s); };
  auto v_full = [&](int s) { return bar(14 + s); };
  auto v_empty = [&](int s) { return bar(17 + s); };
  auto v_clean = [&](int s) { return bar(20 + s); };
  const uint32_t drained = bar(23);
  uint8_t* const words = smem_raw + (bar(24) - raw);
  volatile int* const abort = reinterpret_cast<volatile int*>(words);
  volatile int* const odd = abort + 1;
  volatile uint32_t* const tmem_slot = reinterpret_cast<volatile uint32_t*>(words) + 2;
  volatile int* const place = abort + 4;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), kSoftWarps);
      mbar_init(o_done(s), 1);
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 1 + kSoftWarps);
    }
    for (int s = 0; s < kKeyRingV; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 1);
      mbar_init(v_clean(s), 1);
    }
    mbar_init(drained, 1);
    *abort = 0;
    *odd = 0;
    fence_mbar_init();
  }
  if (warp == 0) sts32(zeros + lane * 4, 0u);
  if (warp == 5) tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 256);
  if (A.tree)                        // not by warp 0, which looks for its part meanwhile
    for (int e = (int)threadIdx.x - 32; e >= 0 && e < A.n_new; e += kKeyThreads - 32) sts32(depths + e * 4, A.depth[e]);
  grid_dependency_wait();
  grid_launch_dependents();          // the merge may get ready on idle SMs
  if (warp == 0) {
    const Place pl = find_part<kBlk>(A, lane, blockIdx.x / A.head_lanes, gridDim.x / A.head_lanes);
    if (lane == 0) {
      place[0] = pl.b;
      place[1] = pl.off;
      place[2] = pl.u0;
      place[3] = pl.u1;
      place[4] = pl.total;
      place[5] = pl.parts;
      if (blockIdx.x == 0) *reinterpret_cast<int2*>(A.status) = make_int2(SPECDEC_OK, pl.any_bad);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int part0 = place[2];
  Walk<kBlk> w;
  w.start(A, place[0], place[1], part0, place[3]);
  auto warp_wait = [&](uint32_t b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait<true>(b, parity, abort, A.status));
  };
  uint32_t issued_k = 0, issued_v = 0, phase_k = 0, phase_v = 0;   // producer: copies in flight

  if (warp == 4) {
    // ------------------------------------------------------------- loads --
    const uint64_t pol = policy_evict_first();
    uint32_t n = 0, nt = 0;
    bool ok = true;
    auto load_queries = [&](const Walk<kBlk>& t, uint32_t nt) {
      const uint32_t qs = nt & 1;
      if (!warp_wait(q_empty(qs), ((nt >> 1) & 1) ^ 1u)) return false;
      // lane = row: two e4m3 terms of its 128 dims
      const int pos0 = t.g * A.group_pos, row = lane;
      const bool mine = row < min(A.group_pos, A.n_new - pos0) * A.G;
      const int idx = mine ? pos0 + row / A.G : 0, head = t.h * A.G + (mine ? row % A.G : 0);
      const uint4* src = reinterpret_cast<const uint4*>(A.q + ((size_t)t.b * A.n_new + idx) * A.q_stride +
                                                        (size_t)head * kD);
      uint32_t wv[kD / 2];
#pragma unroll
      for (int c = 0; c < kD / 8; ++c) {
        const uint4 v = mine ? __ldcg(src + c) : make_uint4(0u, 0u, 0u, 0u);
        wv[4 * c] = v.x;
        wv[4 * c + 1] = v.y;
        wv[4 * c + 2] = v.z;
        wv[4 * c + 3] = v.w;
      }
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < kD / 2; ++k) top = max(top, max(wv[k] & 0x7fffu, (wv[k] >> 16) & 0x7fffu));
      const bool fine = top < 0x7f80u;
      const int down = top > 0 && fine ? min(max((int)(top >> 7) - 134, -100), 120) : 0;
      const float mul = __uint_as_float((uint32_t)(127 - down) << 23);
      const uint32_t hi_row = qb + qs * kKeyQBytes + row * kD, lo_row = hi_row + kRows * kD;
#pragma unroll
      for (int c = 0; c < kD / 16; ++c) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t ph[2], pl[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t u = wv[8 * c + 2 * k + x];
            const float a = __uint_as_float(u << 16) * mul, b = __uint_as_float(u & 0xffff0000u) * mul;
            ph[x] = f32_to_e4m3x2(a, b);
            const uint32_t back = e4m3x2_to_f16x2((uint16_t)ph[x]);
            const float2 r2 = __half22float2(*reinterpret_cast<const __half2*>(&back));
            pl[x] = f32_to_e4m3x2(a - r2.x, b - r2.y);
          }
          hi[k] = ph[0] | (ph[1] << 16);
          lo[k] = pl[0] | (pl[1] << 16);
        }
        const uint32_t to = (uint32_t)((c ^ (row & 7)) << 4);
        if (row < kRows) {
          sts128(hi_row + to, hi[0], hi[1], hi[2], hi[3]);
          sts128(lo_row + to, lo[0], lo[1], lo[2], lo[3]);
        }
      }
      const uint32_t at = tab + qs * kKeyTab + row * 4;
      const float q_scale = fine ? __uint_as_float((uint32_t)(127 + down) << 23) : __uint_as_float(0x7fffffffu);
      sts32(at, __float_as_uint(A.scale * q_scale * (kExtra ? 1.f : kLog2e)));
      sts32(at + kLanes * 4, __float_as_uint(kExtra && A.slopes ? A.slopes[head] * kLog2e : 0.f));
      const int dep = A.tree ? (int)lds32(depths + idx * 4) : idx;
      sts32(at + 2 * kLanes * 4, __float_as_uint((float)dep));
      sts32(at + 3 * kLanes * 4, (uint32_t)(idx * A.Hq + head));
      for (int a0 = 0; a0 < A.n_new; a0 += 32) {
        uint32_t sees = 0, of_mine = 0;          // new positions a0 .. a0 + 31 that this row sees
        if (A.tree)
          sees = A.anc[idx][a0 >> 5];
        else if (idx >= a0)
          sees = idx - a0 >= 31 ? 0xffffffffu : (2u << (idx - a0)) - 1u;
#pragma unroll
        for (int a = 0; a < 32; ++a) {
          bool see = (sees >> a) & 1u;
          if (A.window > 0) {
            const int da = A.tree ? (int)lds32(depths + (a0 + a) * 4) : a0 + a;
            see = see && dep - da < A.window;
          }
          const uint32_t rows = __ballot_sync(0xffffffffu, see);
          if (lane == a) of_mine = rows;
        }
        sts32(tab + qs * kKeyTab + 4 * kLanes * 4 + (a0 + lane) * 4, of_mine);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(qs));
      return true;
    };
    // A block that not every query sees whole, before V^T P^T takes it.
    int check_j0 = -1, check_L = 0;      // the last block loaded: its first row (-1: nothing to do), its sequence
    auto check_values = [&](uint32_t nb) {
      if (check_j0 < 0) return true;
      const uint32_t s = nb % kKeyRingV;
      if (!warp_wait(v_full(s), (nb / kKeyRingV) & 1)) return false;
      // Rows past the sequence hold anything, and a NaN in a row that not
      // every query sees would pass a zero probability: neither stays in
      // the product. The epilogue adds the NaN where seen.
      for (int e = lane; e < kKeySlot / 16; e += 32) {
        const uint32_t a = ring_v + s * kKeySlot + e * 16;
        const uint4 v = lds128(a);
        uint32_t x[4] = {v.x, v.y, v.z, v.w};
        bool put = false;
        if (check_j0 + (e >> 3) >= check_L) {
          x[0] = x[1] = x[2] = x[3] = 0u;
          put = true;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // bytes whose low seven bits are all ones
          const uint32_t nan = __vcmpeq4(x[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
          if (nan) {
            x[k] &= ~nan;
            put = true;
            *odd = 1;
          }
        }
        if (put) sts128(a, x[0], x[1], x[2], x[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_clean(s));
      return true;
    };
    if (!w.done()) ok = load_queries(w, 0);
    for (; ok && !w.done(); w.next(A), ++nt) {
      for (int i = 0; i < w.n_here; ++i, ++n) {
        const uint32_t s = n & 1, ph = (n >> 1) & 1;
        const int j0 = w.row(i);
        if (!(ok = warp_wait(k_empty(s), ph ^ 1u))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(k_full(s), kKeySlot);
          tma_load_4d(ring_k + s * kKeySlot, &tmap_k, k_full(s), 0, w.h, j0, w.b, pol);
        }
        __syncwarp();
        issued_k |= 1u << s;
        phase_k = (phase_k & ~(1u << s)) | (ph << s);
        const uint32_t sv = n % kKeyRingV, phv = (n / kKeyRingV) & 1;
        if (!(ok = warp_wait(v_empty(sv), phv ^ 1u))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(v_full(sv), kKeySlot);
          tma_load_4d(ring_v + sv * kKeySlot, &tmap_v, v_full(sv), 0, w.h, j0, w.b, pol);
        }
        __syncwarp();
        issued_v |= 1u << sv;
        phase_v = (phase_v & ~(1u << sv)) | (phv << sv);
        // the check runs a block behind, when its values are likely there
        if (!(ok = check_values(n - 1))) break;
        check_j0 = w.clean(i) ? -1 : j0;
        check_L = w.L;
        if (i == w.n_here / 2) {
          // halfway, when the last tile's buffer is free: the next one's queries
          Walk<kBlk> then = w;
          then.next(A);
          if (!then.done() && !(ok = load_queries(then, nt + 1))) break;
        }
      }
    }
    if (ok) check_values(n - 1);
  } else if (warp == 5) {
    // ------------------------------------------------------------ issuer --
    // Scores run a block ahead of the values' product.
    constexpr uint32_t id_s = instr_desc(0, false, 2 * kRows);
    constexpr uint32_t id_o = instr_desc(0, true, kKeyTerms * kRows) | (1u << 15)     // A (V^T) is M-major too,
                              | (1u << 10);                                         // B is e5m2
    const uint64_t k_desc = operand_desc<128>(ring_k, 16), q_desc = operand_desc<128>(qb, 16);
    const uint64_t v_desc = operand_desc<128>(ring_v, 16), p_desc = operand_desc32(pb, kKeyPanel);
    Walk<kBlk> wq = w;
    uint32_t nq = 0, tq = 0, n = 0, clean_ph = 0;
    int iq = 0;
    auto issue_scores = [&]() {
      const uint32_t qs = tq & 1, s = nq & 1;
      if (iq == 0 && !warp_wait(q_full(qs), (tq >> 1) & 1)) return false;
      if (!warp_wait(k_full(s), (nq >> 1) & 1)) return false;
      tc_fence_after();
      const uint64_t kd = k_desc + (uint64_t)(s * (kKeySlot >> 4)), qd = q_desc + (uint64_t)(qs * (kKeyQBytes >> 4));
      const bool last = iq + 1 == wq.n_here;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kD / 32; ++k) mma_ss<true>(tmem + kKeyColS + s * 64, kd + 2 * k, qd + 2 * k, id_s, k > 0);
        tc_commit(s_full(s));
        tc_commit(k_empty(s));
        if (last) tc_commit(q_empty(qs));
      }
      __syncwarp();
      ++nq;
      ++iq;
      if (last) {
        iq = 0;
        ++tq;
        wq.next(A);
      }
      return true;
    };
    bool ok = w.done() || issue_scores();
    for (; ok && !w.done(); w.next(A))
      for (int i = 0; i < w.n_here; ++i, ++n) {
        // the other buffer's scores were read before the last product was issued
        if (!wq.done() && !(ok = issue_scores())) break;
        const uint32_t s = n & 1, sv = n % kKeyRingV;
        if (!(ok = warp_wait(v_full(sv), (n / kKeyRingV) & 1))) break;
        if (!w.clean(i)) {
          if (!(ok = warp_wait(v_clean(sv), (clean_ph >> sv) & 1))) break;
          clean_ph ^= 1u << sv;
        }
        if (!(ok = warp_wait(p_full(s), (n >> 1) & 1))) break;
        tc_fence_after();
        const uint64_t vd = v_desc + (uint64_t)(sv * (kKeySlot >> 4));
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBlk / 32; ++k)
            mma_ss<true>(tmem + kKeyColO, vd + k * (32 * 128 >> 4), p_desc + k * (32 * 32 >> 4), id_o, i > 0 || k > 0);
          tc_commit(o_done(s));
          tc_commit(v_empty(sv));
        }
        __syncwarp();
      }
    // every product has to be done before the tensor memory is given back
    if (elect_one()) tc_commit(drained);
    wait_drain(drained, 0);
  } else {
    // ----------------------------------------------------------- softmax --
    const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
    const int kl = warp * 32 + lane;         // this thread's key of a block, and its dim of the output
    bool dead = false, noted = false;
    uint32_t n = 0, nt = 0;
    for (; !w.done(); w.next(A), ++nt) {
      const int P0 = w.L - A.n_new, pos0 = w.g * A.group_pos;
      const int rows_here = min(A.group_pos, A.n_new - pos0) * A.G;
      const uint32_t qs = nt & 1, t0 = tab + qs * kKeyTab;
      const size_t so = ((size_t)w.b * A.Hkv + w.h) * A.n_scale;
      const float* ks = A.k_scale + so;
      const float* vs = A.v_scale + so;
      float sk_next, sv_next;
      auto load_scales = [&](int jw) {
        sk_next = jw < w.L ? __ldcg(ks + jw / SPECDEC_KV8_BLOCK) : 1.f;
        sv_next = jw < w.L ? __ldcg(vs + jw / SPECDEC_KV8_BLOCK) : 1.f;
      };
      load_scales(w.row(0) + warp * 32);
      // The rows that see cache row jj: those that see its new position, or,
      // before the new rows, those whose window reaches it.
      auto seen_by = [&](int jj) {
        const int a = jj - P0;
        if (jj >= w.L) return 0u;
        if (a >= 0) return lds32(t0 + 4 * kLanes * 4 + a * 4);
        if (A.window <= 0) return 0xffffffffu;
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < kRows; r += 4) {
          const float4 d = lds128f(t0 + 2 * kLanes * 4 + r * 4);
          m |= ((int)d.x - a < A.window ? 1u : 0u) << r | ((int)d.y - a < A.window ? 2u : 0u) << r |
               ((int)d.z - a < A.window ? 4u : 0u) << r | ((int)d.w - a < A.window ? 8u : 0u) << r;
        }
        return m;
      };
      float l[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) l[r] = 0.f;
      if (warp == 0) {
        sts32(ref + lane * 4, __float_as_uint(INFINITY));      // negated: none yet
        sts32(peaks + lane * 4, __float_as_uint(-INFINITY));
      }
      if (!dead && !warp_wait(q_full(qs), (nt >> 1) & 1)) dead = true;
      named_bar_sync(1, 32 * kSoftWarps);

      for (int ib = 0; ib < w.n_here; ++ib, ++n) {
        const int j = w.row(ib) + kl;                  // this thread's cache row
        const bool clean = w.clean(ib);
        const float sk = sk_next, lvb = __log2f(sv_next) + kBase, inv_sv = rcp(sv_next);
        if (ib + 1 < w.n_here) load_scales(w.row(ib + 1) + warp * 32);
        if (!dead && !warp_wait(s_full(n & 1), (n >> 1) & 1)) dead = true;
        tc_fence_after();
        float y[kRows];
        // The tile's first block begins with its rows' maxima, other blocks
        // with exponents against the references; one of those too high, or
        // a row without one high enough, brings in the maxima as well.
        // (`from_ref` points at the negated references, or at zeros: one piece
        // of code for both.)
        bool maxima = ib == 0, settled = ib == 0;
        for (;;) {
          const uint32_t from_ref = maxima ? zeros : ref;
          if (!dead) {
            uint32_t u[2 * kRows];
            tmem_load(tl + kKeyColS + (n & 1) * 64, u);
#pragma unroll
            for (int r = 0; r < kRows; r += 2) {
              y[r] = __uint_as_float(u[r]);
              y[r + 1] = __uint_as_float(u[r + 1]);
              add2(y[r], y[r + 1], __uint_as_float(u[kRows + r]), __uint_as_float(u[kRows + 1 + r]));
            }
          }
          float pj = 0.f;
          if (kExtra && A.slopes) {
            int p = j - P0;                            // position from the first new one's
            if (A.tree && p >= 0) p = (int)lds32(depths + min(p, A.n_new - 1) * 4);
            pj = (float)p;
          }
#pragma unroll
          for (int r = 0; r < kRows; r += 4) {
            const float4 c = lds128f(t0 + r * 4);
            float4 b = lds128f(from_ref + r * 4);
            add2(b.x, b.y, lvb, lvb);
            add2(b.z, b.w, lvb, lvb);
            // The product with the row's factor is rounded before anything is
            // added, so that exponents of any size agree with their reference.
            mul2(y[r], y[r + 1], c.x, c.y);
            mul2(y[r + 2], y[r + 3], c.z, c.w);
            if constexpr (kExtra) {
              const float4 sl = lds128f(t0 + kLanes * 4 + r * 4), dp = lds128f(t0 + 2 * kLanes * 4 + r * 4);
              mul2(y[r], y[r + 1], sk, sk);
              mul2(y[r + 2], y[r + 3], sk, sk);
              if (A.cap > 0.f) {
#pragma unroll
                for (int k = 0; k < 4; ++k) y[r + k] = capped(y[r + k] * A.cap_exp, A.cap * kLog2e, A.cap * kLog2e);
              } else {
                mul2(y[r], y[r + 1], kLog2e, kLog2e);
                mul2(y[r + 2], y[r + 3], kLog2e, kLog2e);
              }
              // bias slope * (pos_j - pos_i)
              float4 away = make_float4(-dp.x, -dp.y, -dp.z, -dp.w);
              add2(away.x, away.y, pj, pj);
              add2(away.z, away.w, pj, pj);
              fma2(away.x, away.y, sl.x, sl.y, b.x, b.y);
              fma2(away.z, away.w, sl.z, sl.w, b.z, b.w);
              add2(y[r], y[r + 1], away.x, away.y);
              add2(y[r + 2], y[r + 3], away.z, away.w);
            } else {
              fma2(y[r], y[r + 1], sk, sk, b.x, b.y);
              fma2(y[r + 2], y[r + 3], sk, sk, b.z, b.w);
            }
          }
          if (!clean) {
            const uint32_t m = seen_by(j);
#pragma unroll
            for (int r = 0; r < kRows; ++r) y[r] = (m >> r) & 1u ? y[r] : -INFINITY;
          }
          if (!maxima) {
            if (settled) {
              // exponents of 2^24 and more are whole steps from their reference
#pragma unroll
              for (int r = 0; r < kRows; ++r) y[r] = min_or_nan(y[r], kBase);
              break;
            }
            float top = -INFINITY, bot = INFINITY;
            if (!dead) {
#pragma unroll
              for (int r = 0; r < kRows; r += 4) {
                top = max3(max3(top, y[r], y[r + 1]), y[r + 2], y[r + 3]);
                bot = min3(min3(bot, y[r], y[r + 1]), y[r + 2], y[r + 3]);
              }
            }
            // Votes: 16 for a warp with an exponent too high, 1 for one with a
            // key that every row holds high enough, which settles it in most blocks.
            const bool high = __any_sync(0xffffffffu, top > kBase), even = __any_sync(0xffffffffu, bot > kBase - kFall);
            const int votes = bar_count(1, 32 * kSoftWarps, lane < 16 ? high : lane == 16 && even);
            if (__builtin_expect((votes & 15) && votes < 16, 1)) break;
            if (votes < 16) {
              // The rows with a key high enough, over the block's keys, and those
              // with one that a lower reference would serve. (Two blocks' marks: a
              // warp may still read the last one's.)
              uint32_t loud = 0, worth = 0;
#pragma unroll
              for (int r = 0; r < kRows; r += 4) {
                // how far each reference is below its highest: one at its end is not moved
                const float4 p = lds128f(peaks + r * 4), m = lds128f(ref + r * 4);
                const float down[4] = {p.x + m.x, p.y + m.y, p.z + m.z, p.w + m.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  loud |= (y[r + k] > kBase - kFall ? 1u : 0u) << (r + k);
                  worth |= (down[k] < kDeep && y[r + k] > down[k] + (kBase - kLift - kReach) ? 1u : 0u) << (r + k);
                }
              }
              loud = __reduce_or_sync(0xffffffffu, loud);
              worth = __reduce_or_sync(0xffffffffu, worth);
              const uint32_t mark = marks + (n & 1) * 32;
              if (lane == 0) sts64(mark + warp * 8, dead ? 0u : loud, dead ? 0u : worth);
              named_bar_sync(1, 32 * kSoftWarps);
              const uint4 a = lds128(mark), b = lds128(mark + 16);
              loud = a.x | a.z | b.x | b.z;
              worth = a.y | a.w | b.y | b.w;
              // rows of padding have no say
              if ((worth & ~loud & (0xffffffffu >> (32 - rows_here))) == 0) break;
            }
            maxima = settled = true;
            continue;
          }
          // ---- some row's reference has to move ----
          if (dead) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) y[r] = -INFINITY;
          }
          const float mine = rows_to_lanes(y, lane, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
          sts32(red + kl * 4, __float_as_uint(mine - kBase));
          named_bar_sync(1, 32 * kSoftWarps);
          if (warp == 0) {
            float M = __uint_as_float(lds32(red + lane * 4));
#pragma unroll
            for (int x = 1; x < kSoftWarps; ++x) M = fmaxf(M, __uint_as_float(lds32(red + (x * 32 + lane) * 4)));
            const float was = -__uint_as_float(lds32(ref + lane * 4));
            const float peak = __uint_as_float(lds32(peaks + lane * 4));
            const bool down = M < was - kFall && M > peak - kLift - kReach && was > peak - kDeep;
            const bool move = M > was || down;
            const float to = down ? peak - kDeep : M + kLift;
            if (move) sts32(peaks + lane * 4, __float_as_uint(fmaxf(peak, to)));
            sts32(ref + lane * 4, __float_as_uint(-(move ? to : was)));
            sts32(ref + kLanes * 4 + lane * 4, __float_as_uint(move ? ex2(was - to) : 1.f));
          }
          named_bar_sync(1, 32 * kSoftWarps);
          if (!dead) {
            const uint32_t al = ref + kLanes * 4;
#pragma unroll
            for (int r = 0; r < kRows; r += 4) {
              const float4 f = lds128f(al + r * 4);
              mul2(l[r], l[r + 1], f.x, f.y);
              mul2(l[r + 2], l[r + 3], f.z, f.w);
            }
            if (ib > 0) {
              if (!warp_wait(o_done((n - 1) & 1), ((n - 1) >> 1) & 1)) dead = true;
              if (!dead) {
                tc_fence_after();
#pragma unroll 1
                for (int g = 0; g < kKeyPanels; ++g) {
                  const float4 lo = lds128f(al + g * 32), hi = lds128f(al + g * 32 + 16);
                  const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                  uint32_t v[32];
                  tmem_load(tl + kKeyColO + 32 * g, v);
#pragma unroll
                  for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f[k % 8]);
                  tmem_store(tl + kKeyColO + 32 * g, v, Cols<32>{});
                }
                tmem_wait_store();
              }
            }
          }
          maxima = false;
        }
        // ---- probabilities, as four e5m2 terms ----
        // the last block's product has read its own
        if (!dead && n > 0 && !warp_wait(o_done((n - 1) & 1), ((n - 1) >> 1) & 1)) dead = true;
        if (dead) continue;
        const uint32_t to = pb + kl * 32, half = ((uint32_t)kl >> 2 & 1) << 4;   // halves trade places every four keys
#pragma unroll
        for (int g = 0; g < kKeyPanels; ++g) {
          uint32_t code[kKeyTerms][2];                 // [term][rows 4x .. 4x + 3 of the panel's]
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t part[kKeyTerms][2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int r = 8 * g + 4 * x + 2 * z;
              const float p0 = ex2(y[r]), p1 = ex2(y[r + 1]);
              uint32_t h = pack2<true>(p0, p1);
              acc2(l[r], l[r + 1], p0, p1, inv_sv);
#pragma unroll
              for (int t = 0; t < kKeyTerms; ++t) {
                part[t][z] = f16x2_to_e5m2x2(h);
                if (t + 1 < kKeyTerms) h = rest8(h, part[t][z]);
              }
            }
#pragma unroll
            for (int t = 0; t < kKeyTerms; ++t) code[t][x] = part[t][0] | (part[t][1] << 16);
          }
          sts128(to + g * kKeyPanel + half, code[0][0], code[0][1], code[1][0], code[1][1]);
          sts128(to + g * kKeyPanel + (half ^ 16), code[2][0], code[2][1], code[3][0], code[3][1]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(n & 1));
      }

      // ---- sums over the keys, then the output or this part's share ----
      const float sum = rows_to_lanes(l, lane, 0.f, [](float a, float b) { return a + b; });
      sts32(red + kl * 4, __float_as_uint(sum));
      named_bar_sync(1, 32 * kSoftWarps);
      const bool whole = w.blk == 0 && w.n_here == w.nb;
      const size_t slot = (size_t)blockIdx.x * 2 + (w.u == part0 ? 0 : 1);
      if (warp == 0) {
        float lt = 0.f;
#pragma unroll
        for (int x = 0; x < kSoftWarps; ++x) lt += __uint_as_float(lds32(red + (x * 32 + lane) * 4));
        // the output's factor per row, where the references' factors were
        const float inv = lt > 0.f ? 1.f / lt : (lt == 0.f ? 0.f : lt);    // NaN stays
        sts32(ref + kLanes * 4 + lane * 4, __float_as_uint(whole ? inv : 1.f));
        if (!whole && lane < rows_here && !dead)
          *reinterpret_cast<float2*>(A.part_ml + (slot * kLanes + lane) * 2) =
              make_float2(-__uint_as_float(lds32(ref + lane * 4)), lt);
      }
      named_bar_sync(1, 32 * kSoftWarps);
      if (!dead && !warp_wait(o_done((n - 1) & 1), ((n - 1) >> 1) & 1)) dead = true;
      tc_fence_after();
      if (!dead) {
        float o[kRows];
#pragma unroll
        for (int g = 0; g < kKeyPanels; ++g) {
          uint32_t v[32];
          tmem_load(tl + kKeyColO + 32 * g, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            auto term = [&](int t) { return __uint_as_float(v[8 * t + k]); };
            o[8 * g + k] = fmaf(term(3), 1.f / 512, fmaf(term(2), 1.f / 64, fmaf(term(1), 1.f / 8, term(0))));
          }
        }
        if (*odd) {
          // NaN that were held back from the product (rare), for the rows that see them
          for (int ib = 0; ib < w.n_here; ++ib) {
            if (w.clean(ib)) continue;
            const int jb = w.row(ib);
            for (int k = 0; k < kBlk && jb + k < w.L; ++k) {
              const uint8_t code =
                  static_cast<const uint8_t*>(A.v)[(((size_t)w.b * A.Lmax + jb + k) * A.Hkv + w.h) * kD + kl];
              if ((code & 0x7fu) != 0x7fu) continue;
              const uint32_t m = seen_by(jb + k);
#pragma unroll
              for (int r = 0; r < kRows; ++r)
                if ((m >> r) & 1u) o[r] = __uint_as_float(0x7fffffffu);
            }
          }
        }
        __nv_bfloat16* out = A.out + (size_t)w.b * A.n_new * A.Hq * kD + kl;
        float* part = A.part_o + slot * kLanes * kD + kl;
#pragma unroll
        for (int r = 0; r < kRows; r += 4) {
          if (r >= rows_here) break;
          const float4 f = lds128f(ref + kLanes * 4 + r * 4);
          const uint4 at = lds128(t0 + 3 * kLanes * 4 + r * 4);
          const float ff[4] = {f.x, f.y, f.z, f.w};
          const uint32_t to[4] = {at.x, at.y, at.z, at.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (r + k >= rows_here) break;
            if (whole)
              out[(size_t)to[k] * kD] = __float2bfloat16(o[r + k] * ff[k]);
            else
              part[(r + k) * kD] = o[r + k];
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty(qs));
      tc_fence_before();
      named_bar_sync(1, 32 * kSoftWarps);    // the tables are free for the next tile
      if (w.blk == 0 && (!whole || A.note_tiles) && threadIdx.x == 0) {
        write_note(A, w.b, w.h, w.g, whole, last_part(w, place[4], place[5]), (int)(slot & 1));
        noted = true;
      }
    }
    if (!noted && !A.note_tiles && threadIdx.x == 0) A.notes[blockIdx.x].x = -1;
    zero_empty<kD, kBlk>(A);
  }
  tc_fence_before();
  __syncthreads();   // every role has left its loop
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, 256);
  if (*abort && warp == 4 && lane == 0)
    // A wait gave up: let every copy already issued land before the CTA exits.
    for (int s = 0; s < kKeyRingV; ++s) {
      if (issued_k & (1u << s)) wait_drain(k_full(s), (phase_k >> s) & 1u);
      if (issued_v & (1u << s)) wait_drain(v_full(s), (phase_v >> s) & 1u);
    }
}

template <bool kExtra>
cudaError_t launch_keys(const CacheAttnLaunch& A, const CUtensorMap& tk, const CUtensorMap& tv,
                        cudaStream_t stream) {
  static std::atomic<int> smem_set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !smem_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(cache_attn_keys_kernel<kExtra>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeySmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) smem_set[dev].store(1, std::memory_order_release);
  }
  const long long tiles = (long long)A.B * A.Hkv * A.n_groups;
  const long long most = tiles * ((A.Lmax + kKeyBlk - 1) / kKeyBlk + kTileCost);
  const int parts = cache_attn_parts(A, kCacheAttnMaxCtas, most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts * A.head_lanes);
  cfg.blockDim = dim3(kKeyThreads);
  cfg.dynamicSmemBytes = kKeySmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  CacheAttnLaunch L = A;
  L.note_tiles = note_tiles(A, parts);
  e = cudaLaunchKernelEx(&cfg, cache_attn_keys_kernel<kExtra>, L, tk, tv);
  if (e != cudaSuccess) return e;
  return launch_combine<kKeyD, kKeyLanes>(L, parts, cfg);
}

}  // namespace cache_attn
}  // namespace specdec
