// Verify-step attention with caps, distance biases, windows and token trees,
// over a bf16 cache or over an e4m3 cache with block scales.
//
// For new position i (row r = i * G + gq of KV head h) and cache row j:
//   s_rj = scale * q_r . k_j            (k_j = s_k code_j for an e4m3 cache)
//   s_rj = cap * tanh(s_rj / cap)       when a cap is set
//   x_rj = log2(e) * (s_rj - slope_h * (pos_i - pos_j))
//   o_r  = sum_j 2^x_rj v_j / sum_j 2^x_rj   over the rows j that i sees
// with one pass over the cache and the softmax statistics in fp32. The scale
// of an e4m3 value block enters the exponent: with y_rj = x_rj + log2(s_v),
// o = sum 2^(y - M) code_j / sum (2^(y - M) / s_v), M a reference near the
// running maximum of y, so weights of every block share one range.
//
// Bound: HBM (each K and V row is read once per group of up to 128 query
// rows).
//
// Schedule. The (sequence, KV head, row group) tiles, each a run of cache
// blocks as long as its own sequence (or window), are laid end to end and
// the run of blocks is cut into equal parts, one per CTA (one CTA per SM), on
// the device from seq_lens, so ragged batches keep every SM busy to the end.
// A tile that lies inside one part is finished by its CTA; the others leave
// (maximum, sum, unnormalised output) partials that combine_kernel merges.
//
// CTA: warps 0-3 softmax, 4-7 auxiliary, 8 TMA producer, 9 tcgen05 issuer.
//   S = Q K^T: tcgen05.mma, M = 128 query rows, N = a block of keys, into one
//     of two tensor-memory buffers, a block ahead of the softmax. bf16:
//     kind::f16. e4m3: kind::f8f6f4 on the codes as they lie; the query row,
//     scaled by a power of two to below 256, is the sum of two e4m3 terms
//     (4 + 4 significant bits hold a bf16 value exactly down to 2^-10 of the
//     row's largest, and to 2^-18 of it below), so two products accumulate.
//   softmax: lane = query row, so maxima and sums need no exchange. With
//     R <= 64 query rows the 128 lanes hold 128 / RP copies of the rows (RP =
//     32 or 64) and each copy takes its own share of every block's keys; its
//     probabilities go to its share's columns of the P operand, whose other
//     columns stay zero, so the copies are independent online softmaxes,
//     merged once per tile. The reference M moves only when a row's maximum
//     passes it by 2^8 (the exponents have that headroom), so the output in
//     tensor memory is rarely rescaled.
//   O += P V: P from tensor memory, V the MN-major operand, kind::f16. e4m3
//     values are widened to f16 (exact) by the auxiliary warps into a second
//     shared-memory tile, since P needs f16's 11 bits and both operands share
//     a type; bf16 values are used as they land.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "kernels.h"

namespace specdec {
namespace cache_attn {

constexpr int kSoftWarps = 4;
constexpr int kAuxWarps = 4;
constexpr int kProducer = 8, kIssuer = 9;     // warp indices
constexpr int kThreads = 320;
constexpr unsigned long long kDrainNs = 1000000000ull;
constexpr float kHeadroom = 8.f;              // log2 by which a maximum may pass its reference
constexpr int kSmemLimit = 227 * 1024;

template <bool kE4m3, int kD, int kRP>
struct Shape {
  static constexpr int kElem = kE4m3 ? 1 : 2;
  static constexpr int kBlk = cache_attn_block(kE4m3, kD);   // keys per block
  static constexpr int kRowBytes = kD * kElem;
  static constexpr int kPanelBytes = kRowBytes < 128 ? kRowBytes : 128;   // one TMA box row
  static constexpr int kPanels = kRowBytes / kPanelBytes;
  static constexpr int kSlotBytes = kBlk * kRowBytes;        // a block of K, or of V, as it lands
  static constexpr int kCopies = 128 / kRP;                  // copies of the query rows
  static constexpr int kKpl = kBlk / kCopies;                // keys per lane and block
  static constexpr int kTerms = kE4m3 ? 2 : 1;
  static constexpr int kQTerm = 128 * kRowBytes;             // 128 query rows in the K operand's type
  static constexpr int kQBytes = kTerms * kQTerm;
  static constexpr int kQBufs = kElem * kD >= (kE4m3 ? 128 : 512) ? 1 : 2;
  static constexpr int kV16Bytes = kE4m3 ? kBlk * kD * 2 : 0;   // widened V, two of them
  static constexpr int kStageBytes = kCopies > 1 ? 128 * 33 * 4 : 0;   // merge of the copies
  static constexpr int kTabBytes = 2 * 128 * 4 + 128 * 8 + 128 * 16 + 128 * 4;  // q scales, (m, l), tree
  static constexpr int kFixed = 1024 + 2 * kV16Bytes + kQBufs * kQBytes + kStageBytes + kTabBytes + 512;
  static constexpr int kRingMax = (kSmemLimit - kFixed) / (2 * kSlotBytes);
  static constexpr int kRing = kRingMax < 6 ? kRingMax : 6;  // K blocks (and V blocks) in flight
  static constexpr int kSmem = kFixed + 2 * kRing * kSlotBytes;
  static_assert(kRing >= 2, "two K and two V blocks must fit");
  // tensor memory columns: two score buffers, the output, two P operands
  static constexpr int kColS = 0, kColO = 2 * kBlk, kColP = kColO + kD;
  static_assert(kColP + kBlk <= 512, "tensor memory");
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
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
// Two e4m3 codes (16 bits) to two f16 values; every e4m3 value is an f16 value.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return h;
}
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
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

// Shared-memory operand descriptor, swizzled rows of kPanel = 128 or 64
// bytes in groups of 8. K-major: the k extent of one MMA lies inside a row.
// MN-major (V): a row is one k, its bytes run along N; `lead` is the distance
// to the next panel of N and 8 k rows follow every 8 * kPanel bytes.
template <int kPanel>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, uint32_t lead) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(lead >> 4) << 16;
  d |= (uint64_t)((8u * kPanel) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)(kPanel == 128 ? 2 : 4) << 61;
  return d;
}
// Instruction descriptor fields: D fp32; operand types (f16 0, bf16 1 under
// kind::f16; e4m3 0 under kind::f8f6f4); B transposed (MN-major).
__host__ __device__ constexpr uint32_t instr_desc(int type, bool b_mn, int N) {
  return (1u << 4) | ((uint32_t)type << 7) | ((uint32_t)type << 10) | (b_mn ? 1u << 16 : 0u) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// D (+)= A B^T with A and B in shared memory.
template <bool kF8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (kF8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    tc_mma_bf16(d, a, b, idesc, acc);
}
// The same with A in tensor memory (f16 or bf16 pairs, one row per lane).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Tensor memory: each thread of a warp reads or writes consecutive 32-bit
// columns of its lane. Loads return with the values there.
template <int kN>
struct Cols {};
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
      "}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]),
        "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]),
        "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
      : "r"(taddr + 0)
      : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&x)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
      "}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]),
        "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]),
        "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]), "=r"(x[16]), "=r"(x[17]),
        "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]),
        "=r"(x[24]), "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]),
        "=r"(x[30]), "=r"(x[31])
      : "r"(taddr + 0)
      : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&x)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
      "}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63"
      "}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]),
        "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]),
        "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]), "=r"(x[16]), "=r"(x[17]),
        "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]),
        "=r"(x[24]), "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]),
        "=r"(x[30]), "=r"(x[31]), "=r"(x[32]), "=r"(x[33]), "=r"(x[34]), "=r"(x[35]),
        "=r"(x[36]), "=r"(x[37]), "=r"(x[38]), "=r"(x[39]), "=r"(x[40]), "=r"(x[41]),
        "=r"(x[42]), "=r"(x[43]), "=r"(x[44]), "=r"(x[45]), "=r"(x[46]), "=r"(x[47]),
        "=r"(x[48]), "=r"(x[49]), "=r"(x[50]), "=r"(x[51]), "=r"(x[52]), "=r"(x[53]),
        "=r"(x[54]), "=r"(x[55]), "=r"(x[56]), "=r"(x[57]), "=r"(x[58]), "=r"(x[59]),
        "=r"(x[60]), "=r"(x[61]), "=r"(x[62]), "=r"(x[63])
      : "r"(taddr + 0), "r"(taddr + 32)
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t* x, Cols<8>) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8};"
      ::"r"(taddr), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]),
        "r"(x[6]), "r"(x[7])
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t* x, Cols<16>) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(taddr), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]),
        "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]), "r"(x[10]), "r"(x[11]),
        "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t* x, Cols<32>) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      ::"r"(taddr), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]),
        "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]), "r"(x[10]), "r"(x[11]),
        "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]), "r"(x[16]), "r"(x[17]),
        "r"(x[18]), "r"(x[19]), "r"(x[20]), "r"(x[21]), "r"(x[22]), "r"(x[23]),
        "r"(x[24]), "r"(x[25]), "r"(x[26]), "r"(x[27]), "r"(x[28]), "r"(x[29]),
        "r"(x[30]), "r"(x[31])
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t* x, Cols<64>) {
  tmem_store(taddr, x, Cols<32>{});
  tmem_store(taddr + 32, x + 32, Cols<32>{});
}
__device__ __forceinline__ void tmem_wait_store() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
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

// The visible rows among 32 of the cache, for one query row: the cached
// prefix (rows below P0, bounded below by the window) and the new rows' own
// mask, 128 bits from row P0 on.
struct Sight {
  int P0, low;            // first new row; lowest prefix row seen
  uint32_t v[4];
  __device__ __forceinline__ uint32_t word(int k) const {
    return k == 0 ? v[0] : k == 1 ? v[1] : k == 2 ? v[2] : k == 3 ? v[3] : 0u;
  }
  __device__ __forceinline__ uint32_t mask(int j) const {
    const int p = P0 - j, lo = low - j;
    uint32_t m = p <= 0 ? 0u : p >= 32 ? 0xffffffffu : (1u << p) - 1u;
    if (lo > 0) m &= lo >= 32 ? 0u : 0xffffffffu << lo;
    const int off = -p;
    if (off > -32 && off < 128) {
      if (off < 0)
        m |= v[0] << -off;
      else
        m |= __funnelshift_r(word(off >> 5), word((off >> 5) + 1), off & 31);
    }
    return m;
  }
};

template <bool kE4m3, int kD, int kRP, bool kExtra>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CacheAttnLaunch A, const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_q) {
  using S = Shape<kE4m3, kD, kRP>;
  constexpr int kBlk = S::kBlk, kKpl = S::kKpl, kR = S::kRing, kNq = S::kQBufs;
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring_k = (raw + 1023u) & ~1023u;
  const uint32_t ring_v = ring_k + kR * S::kSlotBytes;
  const uint32_t v16 = ring_v + kR * S::kSlotBytes;
  const uint32_t qb = v16 + 2 * S::kV16Bytes;
  const uint32_t stage = qb + kNq * S::kQBytes;
  const uint32_t q_tab = stage + S::kStageBytes;           // query row scales [kNq][128]
  const uint32_t ml_tab = q_tab + 2 * 128 * 4;             // (reference, sum) of every lane
  const uint32_t tree = ml_tab + 128 * 8;                  // [128][4] ancestor words, then depth [128]
  const uint32_t bars = tree + 128 * 16 + 128 * 4;
  auto k_full = [&](int s) { return bars + 8u * (uint32_t)s; };
  auto k_empty = [&](int s) { return bars + 8u * (uint32_t)(kR + s); };
  auto v_full = [&](int s) { return bars + 8u * (uint32_t)(2 * kR + s); };
  auto v_empty = [&](int s) { return bars + 8u * (uint32_t)(3 * kR + s); };
  auto v_clean = [&](int s) { return bars + 8u * (uint32_t)(4 * kR + s); };
  const uint32_t bars2 = bars + 8u * 5 * kR;
  auto s_full = [&](int s) { return bars2 + 8u * (uint32_t)s; };
  auto p_full = [&](int s) { return bars2 + 8u * (uint32_t)(2 + s); };
  auto q_full = [&](int s) { return bars2 + 8u * (uint32_t)(4 + s); };
  auto q_empty = [&](int s) { return bars2 + 8u * (uint32_t)(6 + s); };
  auto v16_full = [&](int s) { return bars2 + 8u * (uint32_t)(8 + s); };
  auto v16_empty = [&](int s) { return bars2 + 8u * (uint32_t)(10 + s); };
  // One per block parity: when a block's scores are there, the product two
  // blocks back is done, so a wait for the one before it is never a phase off.
  auto o_done = [&](int s) { return bars2 + 8u * (uint32_t)(12 + s); };
  const uint32_t drained = bars2 + 8u * 14;
  uint8_t* const words = smem_raw + (bars2 + 8u * 16 - raw);
  volatile int* const abort = reinterpret_cast<volatile int*>(words);
  volatile int* const odd = abort + 1;                     // a value that is no number was held back
  volatile uint32_t* const tmem_slot = reinterpret_cast<volatile uint32_t*>(words) + 2;
  volatile int* const shared_b = abort + 3;
  volatile long long* const shared_u = reinterpret_cast<volatile long long*>(words + 16);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kR; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), kE4m3 ? kAuxWarps : 1 + kAuxWarps);   // bf16: the product reads it too
      mbar_init(v_clean(s), kAuxWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(o_done(s), 1);
      mbar_init(p_full(s), kSoftWarps);
      mbar_init(q_full(s), kE4m3 ? kAuxWarps : 1);
      mbar_init(q_empty(s), kE4m3 ? 1 + kSoftWarps : 1);
      mbar_init(v16_full(s), kAuxWarps);
      mbar_init(v16_empty(s), 1);
    }
    mbar_init(drained, 1);
    *abort = 0;
    *odd = 0;
    fence_mbar_init();
  }
  if (warp == kIssuer) tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk<kBlk> w;
  w.start(A, *shared_b, shared_u[0], shared_u[1], shared_u[2]);
  const long long part0 = shared_u[1];
  // A warp's wait: all lanes agree on whether it ran out.
  auto warp_wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, A.status));
  };
  // Whether every new position sees every row of block ib of the walk's tile.
  auto is_clean = [&](const Walk<kBlk>& t, int ib) {
    const int j0 = (t.first + t.blk + ib) * kBlk, P0 = t.L - A.n_new;
    return j0 + kBlk <= P0 + 1 && (A.window <= 0 || j0 > P0 + A.max_depth - A.window);
  };
  uint32_t issued[3] = {0, 0, 0}, issued_phase[3] = {0, 0, 0};   // producer: K, V, Q copies in flight

  if (warp == kProducer) {
    // ---------------------------------------------------------- producer --
    if (lane == 0) {
      const uint64_t pol = policy_evict_first();
      auto mark = [&](int what, int s, uint32_t ph) {
        issued[what] |= 1u << s;
        issued_phase[what] = (issued_phase[what] & ~(1u << s)) | (ph << s);
      };
      int s = 0;
      uint32_t ph = 0, nt = 0;
      bool ok = true;
      for (; ok && !w.done(); w.next(A), ++nt) {
        if constexpr (!kE4m3) {
          // the tile's query rows, once per copy
          const int qs = nt % kNq;
          const uint32_t qph = (nt / kNq) & 1;
          if (!(ok = mbar_wait(q_empty(qs), qph ^ 1u, abort, A.status))) break;
          const uint32_t box = (uint32_t)(A.group_pos * A.G) * 128u;
          mbar_arrive_expect_tx(q_full(qs), box * (kD / 64) * S::kCopies);
          for (int c = 0; c < S::kCopies; ++c)
            for (int p = 0; p < kD / 64; ++p)
              tma_load_4d(qb + qs * S::kQBytes + p * 128 * 128 + c * kRP * 128, &tmap_q, q_full(qs), p * 64,
                          w.h * A.G, w.g * A.group_pos, w.b, policy_evict_normal());
          mark(2, qs, qph);
        }
        for (int i = 0; i < w.n_here; ++i) {
          const int j0 = (w.first + w.blk + i) * kBlk;
          if (!(ok = mbar_wait(k_empty(s), ph ^ 1u, abort, A.status))) break;
          mbar_arrive_expect_tx(k_full(s), (uint32_t)S::kSlotBytes);
#pragma unroll
          for (int p = 0; p < S::kPanels; ++p)
            tma_load_4d(ring_k + s * S::kSlotBytes + p * kBlk * S::kPanelBytes, &tmap_k, k_full(s),
                        p * (S::kPanelBytes / S::kElem), w.h, j0, w.b, pol);
          mark(0, s, ph);
          if (!(ok = mbar_wait(v_empty(s), ph ^ 1u, abort, A.status))) break;
          mbar_arrive_expect_tx(v_full(s), (uint32_t)S::kSlotBytes);
#pragma unroll
          for (int p = 0; p < S::kPanels; ++p)
            tma_load_4d(ring_v + s * S::kSlotBytes + p * kBlk * S::kPanelBytes, &tmap_v, v_full(s),
                        p * (S::kPanelBytes / S::kElem), w.h, j0, w.b, pol);
          mark(1, s, ph);
          if (++s == kR) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ issuer --
    if (lane == 0 && !w.done()) {
      constexpr uint32_t id_qk = instr_desc(kE4m3 ? 0 : 1, false, kBlk);
      constexpr uint32_t id_pv = instr_desc(kE4m3 ? 0 : 1, true, kD);
      Walk<kBlk> wq = w;                 // the tile whose scores come next
      int iq = 0, sq = 0;
      uint32_t phq = 0, nq = 0, tq = 0;
      auto issue_scores = [&]() {
        const int qs = tq % kNq;
        if (iq == 0 && !mbar_wait<true>(q_full(qs), (tq / kNq) & 1, abort, A.status)) return false;
        if (!mbar_wait<true>(k_full(sq), phq, abort, A.status)) return false;
        tc_fence_after();
        const uint32_t d = tmem + S::kColS + (nq & 1) * kBlk;
#pragma unroll
        for (int term = 0; term < S::kTerms; ++term)
#pragma unroll
          for (int p = 0; p < S::kPanels; ++p)
#pragma unroll
            for (int k = 0; k < S::kPanelBytes / 32; ++k)
              mma_ss<kE4m3>(d,
                            operand_desc<S::kPanelBytes>(qb + qs * S::kQBytes + term * S::kQTerm +
                                                             p * 128 * S::kPanelBytes + k * 32, 16),
                            operand_desc<S::kPanelBytes>(ring_k + sq * S::kSlotBytes +
                                                             p * kBlk * S::kPanelBytes + k * 32, 16),
                            id_qk, term + p + k > 0);
        tc_commit(k_empty(sq));
        tc_commit(s_full(nq & 1));
        if (++sq == kR) {
          sq = 0;
          phq ^= 1u;
        }
        ++nq;
        if (++iq == wq.n_here) {
          tc_commit(q_empty(qs));
          iq = 0;
          ++tq;
          wq.next(A);
        }
        return true;
      };
      bool ok = issue_scores();
      int s = 0;
      uint32_t ph = 0, n = 0, clean_ph = 0;
      for (; ok && !w.done(); w.next(A))
        for (int i = 0; i < w.n_here; ++i, ++n) {
          // Scores run a block ahead. Into a new tile they do so only with a
          // second query buffer: with one, they would wait for the refill.
          const bool more = !wq.done(), early = more && (kNq == 2 || iq != 0);
          if (early && !(ok = issue_scores())) break;
          if (!(ok = mbar_wait<true>(p_full(n & 1), (n >> 1) & 1, abort, A.status))) break;
          uint32_t vb;
          if constexpr (kE4m3) {
            vb = v16 + (n & 1) * S::kV16Bytes;
            if (!(ok = mbar_wait<true>(v16_full(n & 1), (n >> 1) & 1, abort, A.status))) break;
          } else {
            vb = ring_v + s * S::kSlotBytes;
            if (!(ok = mbar_wait<true>(v_full(s), ph, abort, A.status))) break;
            if (!is_clean(w, i)) {
              if (!(ok = mbar_wait<true>(v_clean(s), (clean_ph >> s) & 1, abort, A.status))) break;
              clean_ph ^= 1u << s;
            }
          }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kBlk / 16; ++k)
            mma_ts(tmem + S::kColO, tmem + S::kColP + (n & 1) * (kBlk / 2) + k * 8,
                   operand_desc<128>(vb + k * 2048, kBlk * 128), id_pv, i > 0 || k > 0);
          tc_commit(kE4m3 ? v16_empty(n & 1) : v_empty(s));
          tc_commit(o_done(n & 1));
          if (more && !early && !(ok = issue_scores())) break;
          if (++s == kR) {
            s = 0;
            ph ^= 1u;
          }
        }
      // every product has to be done before the tensor memory is given back
      tc_commit(drained);
      wait_drain(drained, 0);
    }
  } else if (warp >= kSoftWarps) {
    // --------------------------------------------------------- auxiliary --
    const int at = threadIdx.x - 32 * kSoftWarps;      // 0 .. 127
    bool ok = true;
    if constexpr (kE4m3) {
      Walk<kBlk> wl = w;                               // the tile whose queries come next
      uint32_t tl = 0;
      auto load_queries = [&]() {
        const int qs = tl % kNq;
        if (!warp_wait(q_empty(qs), ((tl / kNq) & 1) ^ 1u)) return false;
        constexpr int kCh = kD / 8;                    // lanes per row, 8 dims each
        const int pos0 = wl.g * A.group_pos;
        const int rows = min(A.group_pos, A.n_new - pos0) * A.G;
        for (int e = at; e < kRP * kCh; e += 32 * kAuxWarps) {
          const int r = e / kCh, c = e % kCh;
          uint4 val = make_uint4(0u, 0u, 0u, 0u);
          if (r < rows)
            val = __ldg(reinterpret_cast<const uint4*>(
                A.q + ((size_t)wl.b * A.n_new + pos0 + r / A.G) * A.q_stride +
                (size_t)(wl.h * A.G + r % A.G) * kD + c * 8));
          const uint32_t wv[4] = {val.x, val.y, val.z, val.w};
          float f[8], amax = 0.f;
          bool fine = true;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            f[k] = __uint_as_float(k & 1 ? wv[k >> 1] & 0xffff0000u : wv[k >> 1] << 16);
            amax = fmaxf(amax, fabsf(f[k]));
            fine &= fabsf(f[k]) < INFINITY;
          }
#pragma unroll
          for (int o = kCh / 2; o; o >>= 1) {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            fine &= __shfl_xor_sync(0xffffffffu, (int)fine, o) != 0;
          }
          // largest magnitude -> [2^7, 2^8); a row that holds no numbers is NaN
          const int down = amax > 0.f && fine ? min(max((int)(__float_as_uint(amax) >> 23) - 134, -100), 120) : 0;
          const float mul = __uint_as_float((uint32_t)(127 - down) << 23);
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t ph[2], pl[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float a = f[4 * k + 2 * x] * mul, b = f[4 * k + 2 * x + 1] * mul;
              ph[x] = f32_to_e4m3x2(a, b);
              const uint32_t back = e4m3x2_to_f16x2((uint16_t)ph[x]);
              const float2 r2 = __half22float2(*reinterpret_cast<const __half2*>(&back));
              pl[x] = f32_to_e4m3x2(a - r2.x, b - r2.y);
            }
            hi[k] = ph[0] | (ph[1] << 16);
            lo[k] = pl[0] | (pl[1] << 16);
          }
          const int d0 = c * 8, p = d0 / S::kPanelBytes, cc = (d0 % S::kPanelBytes) / 16;
#pragma unroll
          for (int copy = 0; copy < S::kCopies; ++copy) {
            const int rr = copy * kRP + r;
            const int x = S::kPanelBytes == 128 ? (rr & 7) : ((rr >> 1) & 3);
            const uint32_t dst = qb + qs * S::kQBytes + p * 128 * S::kPanelBytes + rr * S::kPanelBytes +
                                 ((cc ^ x) << 4) + (d0 & 8);
            sts64(dst, hi[0], hi[1]);
            sts64(dst + S::kQTerm, lo[0], lo[1]);
          }
          if (c == 0)
            sts32(q_tab + (qs * 128 + r) * 4,
                  fine ? (uint32_t)(127 + down) << 23 : 0x7fffffffu);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full(qs));
        ++tl;
        wl.next(A);
        return true;
      };
      for (int k = 0; k < kNq; ++k)
        if (ok && !wl.done()) ok = load_queries();
      int s = 0;
      uint32_t ph = 0, n = 0;
      for (; ok && !w.done(); w.next(A)) {
        for (int i = 0; i < w.n_here; ++i, ++n) {
          const bool clean = is_clean(w, i);
          const int j0 = (w.first + w.blk + i) * kBlk;
          if (!(ok = warp_wait(v_full(s), ph))) break;
          if (!(ok = warp_wait(v16_empty(n & 1), ((n >> 1) & 1) ^ 1u))) break;
          // A warp takes 8 keys x 4 chunks of 16 codes at a time: rows p and
          // p ^ 5 side by side keep both the reads and the writes free of
          // bank conflicts under their swizzles.
          const uint32_t src = ring_v + s * S::kSlotBytes, dst = v16 + (n & 1) * S::kV16Bytes;
          const int pr = lane >> 3, row8 = (lane & 4) ? pr ^ 5 : pr;
          constexpr int kQuads = kD / 64;
#pragma unroll 4
          for (int e = warp - kSoftWarps; e < kBlk / 8 * kQuads; e += kAuxWarps) {
            const int j = (e / kQuads) * 8 + row8, c = (e % kQuads) * 4 + (lane & 3);
            constexpr int per = S::kPanelBytes / 16;
            const int x = S::kPanelBytes == 128 ? (j & 7) : ((j >> 1) & 3);
            const uint4 v = lds128(src + (c / per) * kBlk * S::kPanelBytes + j * S::kPanelBytes +
                                   (((c % per) ^ x) << 4));
            const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              h[2 * k] = e4m3x2_to_f16x2((uint16_t)wv[k]);
              h[2 * k + 1] = e4m3x2_to_f16x2((uint16_t)(wv[k] >> 16));
            }
            if (!clean) {
              // Rows past the sequence hold anything, and a NaN in a row that
              // not every query sees would pass a zero probability: neither
              // enters the product. The epilogue adds the NaN where seen.
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                if (j0 + j >= w.L) h[k] = 0u;
                if ((h[k] & 0x7c00u) == 0x7c00u) {
                  h[k] &= 0xffff0000u;
                  *odd = 1;
                }
                if ((h[k] & 0x7c000000u) == 0x7c000000u) {
                  h[k] &= 0x0000ffffu;
                  *odd = 1;
                }
              }
            }
            const uint32_t to = dst + (c >> 2) * kBlk * 128 + j * 128;
            const int c2 = (2 * c) & 7;
            sts128(to + ((c2 ^ (j & 7)) << 4), h[0], h[1], h[2], h[3]);
            sts128(to + (((c2 + 1) ^ (j & 7)) << 4), h[4], h[5], h[6], h[7]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(v_empty(s));
            mbar_arrive(v16_full(n & 1));
          }
          if (++s == kR) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (ok && !wl.done()) ok = load_queries();
      }
    } else {
      // bf16 values are multiplied as they land; only blocks with rows that
      // not every query sees are gone over first (see above).
      int s = 0;
      uint32_t ph = 0;
      for (; ok && !w.done(); w.next(A))
        for (int i = 0; i < w.n_here; ++i) {
          // every block is waited for, and released, so that this loop and the
          // ring never part by more than the ring's length
          if (!(ok = warp_wait(v_full(s), ph))) break;
          if (!is_clean(w, i)) {
            const int j0 = (w.first + w.blk + i) * kBlk;
            for (int e = at; e < S::kSlotBytes / 16; e += 32 * kAuxWarps) {
              const int j = (e >> 3) % kBlk;
              const uint32_t a = ring_v + s * S::kSlotBytes + e * 16;
              uint4 v = lds128(a);
              uint32_t wv[4] = {v.x, v.y, v.z, v.w};
              bool put = false;
              if (j0 + j >= w.L) {
                wv[0] = wv[1] = wv[2] = wv[3] = 0u;
                put = true;
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((wv[k] & 0x7f80u) == 0x7f80u) {
                  wv[k] &= 0xffff0000u;
                  put = true;
                  *odd = 1;
                }
                if ((wv[k] & 0x7f800000u) == 0x7f800000u) {
                  wv[k] &= 0x0000ffffu;
                  put = true;
                  *odd = 1;
                }
              }
              if (put) sts128(a, wv[0], wv[1], wv[2], wv[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(v_clean(s));
          }
          if (lane == 0) mbar_arrive(v_empty(s));
          if (++s == kR) {
            s = 0;
            ph ^= 1u;
          }
        }
    }
  } else {
    // ----------------------------------------------------------- softmax --
    const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);      // this warp's lanes
    const int row = (warp * 32 + lane) % kRP, copy = warp * 32 / kRP;
    constexpr int kSub = kKpl > 32 ? kKpl / 32 : 1;                // 32-row pieces of a lane's keys
    constexpr int kSubKeys = kKpl / kSub;
    bool dead = false;                   // a wait ran out: keep to the barriers, compute nothing
    uint32_t n = 0, nt = 0;
    if constexpr (S::kCopies > 1) {
      const uint32_t zero[32] = {};
#pragma unroll
      for (int c = 0; c < kBlk; c += 32) tmem_store(tl + S::kColP + c, zero, Cols<32>{});
      tmem_wait_store();
    }
    for (; !w.done(); w.next(A), ++nt) {
      const int P0 = w.L - A.n_new, pos0 = w.g * A.group_pos;
      const int rows_here = min(A.group_pos, A.n_new - pos0) * A.G;
      const bool mine = row < rows_here;
      const int idx = mine ? pos0 + row / A.G : 0, gq = mine ? row % A.G : 0;
      const int dep = A.tree ? (int)lds32(tree + 128 * 16 + idx * 4) : idx;
      Sight sight;
      sight.P0 = P0;
      sight.low = A.window > 0 ? P0 + dep - A.window + 1 : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (A.tree) {
          sight.v[k] = lds32(tree + idx * 16 + k * 4);
        } else {
          const int top = idx - 32 * k, low = A.window > 0 ? idx - A.window + 1 - 32 * k : 0;
          uint32_t m = top < 0 ? 0u : top >= 31 ? 0xffffffffu : (2u << top) - 1u;
          if (low > 0) m &= low >= 32 ? 0u : 0xffffffffu << low;
          sight.v[k] = m;
        }
      }
      if (A.tree && A.window > 0 && A.window <= A.max_depth) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          for (int a = 0; a < 32 && 32 * k + a < A.n_new; ++a)
            if (dep - (int)lds32(tree + 128 * 16 + (32 * k + a) * 4) >= A.window) sight.v[k] &= ~(1u << a);
      }
      float ck = A.scale;
      if constexpr (kE4m3) {
        const int qs = nt % kNq;
        if (!dead && !warp_wait(q_full(qs), (nt / kNq) & 1)) dead = true;
        ck *= __uint_as_float(lds32(q_tab + (qs * 128 + row) * 4));
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty(qs));
      }
      if (!kExtra) ck *= kLog2e;
      const float slope = kExtra && A.slopes ? A.slopes[w.h * A.G + gq] * kLog2e : 0.f;

      float m_ref = -INFINITY, l = 0.f;
      const int key0 = copy * kKpl;                                // this copy's first key of a block
      float sk_next[kSub], sv_next[kSub];
      auto load_scales = [&](int j) {
        if constexpr (kE4m3) {
          const size_t so = ((size_t)w.b * A.Hkv + w.h) * A.n_scale;
#pragma unroll
          for (int x = 0; x < kSub; ++x) {
            const int jj = j + x * kSubKeys;
            sk_next[x] = jj < w.L ? __ldg(A.k_scale + so + jj / SPECDEC_KV8_BLOCK) : 1.f;
            sv_next[x] = jj < w.L ? __ldg(A.v_scale + so + jj / SPECDEC_KV8_BLOCK) : 1.f;
          }
        }
      };
      load_scales((w.first + w.blk) * kBlk + key0);

      for (int ib = 0; ib < w.n_here; ++ib, ++n) {
        const int j0 = (w.first + w.blk + ib) * kBlk + key0;
        const bool clean = is_clean(w, ib);
        float sk[kSub], sv[kSub];
        if constexpr (kE4m3) {
#pragma unroll
          for (int x = 0; x < kSub; ++x) {
            sk[x] = sk_next[x];
            sv[x] = sv_next[x];
          }
          if (ib + 1 < w.n_here) load_scales(j0 + kBlk);
        }
        if (!dead && !warp_wait(s_full(n & 1), (n >> 1) & 1)) dead = true;
        if (dead) continue;
        tc_fence_after();
        // ---- this lane's scores, as exponents ----
        union {
          uint32_t u[kKpl];
          float f[kKpl];
        } x;
        {
          const uint32_t from = tl + S::kColS + (n & 1) * kBlk + key0;
          if constexpr (kKpl == 128) {
            tmem_load(from, *reinterpret_cast<uint32_t(*)[64]>(&x.u[0]));
            tmem_load(from + 64, *reinterpret_cast<uint32_t(*)[64]>(&x.u[64]));
          } else {
            tmem_load(from, x.u);
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
          float* const y = x.f + sub * kSubKeys;
          const float lv = kE4m3 ? __log2f(sv[sub]) : 0.f;
          const float c = kE4m3 ? ck * sk[sub] : ck;
          const int js = j0 + sub * kSubKeys;
          if constexpr (kExtra) {
#pragma unroll
            for (int k = 0; k < kSubKeys; ++k) {
              float z = y[k] * c;
              // cap * tanh(z / cap) = cap * (1 - 2 / (1 + e^(2 z / cap)))
              if (A.cap > 0.f) z = A.cap * (1.f - 2.f * rcp(1.f + ex2(z * A.cap_exp)));
              y[k] = fmaf(z, kLog2e, lv);
            }
            if (A.slopes) {
              // bias slope * (pos_j - pos_i); tree nodes stand at their depth
              const float base = (float)(js - P0 - dep);
              if (clean || !A.tree) {
#pragma unroll
                for (int k = 0; k < kSubKeys; ++k) y[k] = fmaf(slope, base + (float)k, y[k]);
              } else {
#pragma unroll
                for (int k = 0; k < kSubKeys; ++k) {
                  int pj = js + k - P0;
                  if (pj >= 0) pj = (int)lds32(tree + 128 * 16 + min(pj, A.n_new - 1) * 4);
                  y[k] = fmaf(slope, (float)(pj - dep), y[k]);
                }
              }
            }
          } else if constexpr (kE4m3) {
#pragma unroll
            for (int k = 0; k < kSubKeys; ++k) y[k] = fmaf(y[k], c, lv);
          } else {
#pragma unroll
            for (int k = 0; k < kSubKeys; ++k) y[k] *= c;
          }
          if (!clean) {
            const uint32_t m = sight.mask(js);
#pragma unroll
            for (int k = 0; k < kSubKeys; ++k) y[k] = (m >> k) & 1u ? y[k] : -INFINITY;
          }
          float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < kSubKeys; ++k) t4[k & 3] = fmaxf(t4[k & 3], y[k]);
          top = fmaxf(top, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])));
        }
        // ---- the reference follows the maximum when it has to ----
        const bool need = mine && top > m_ref + kHeadroom;
        if (__any_sync(0xffffffffu, need)) {
          const float to = need ? top : m_ref;
          const float alpha = need ? ex2(m_ref - to) : 1.f;
          l *= alpha;
          m_ref = to;
          if (ib > 0) {
            if (!warp_wait(o_done((n - 1) & 1), ((n - 1) >> 1) & 1)) {
              dead = true;
              continue;
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < kD; c += 32) {
              uint32_t v[32];
              tmem_load(tl + S::kColO + c, v);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
              tmem_store(tl + S::kColO + c, v, Cols<32>{});
            }
            tmem_wait_store();
          }
        }
        // ---- probabilities ----
        // f16 ones are kept 2^7 high: the headroom's 2^8 above that still fits,
        // and small weights stay normal numbers down to 2^-21.
        const float mu = (m_ref == -INFINITY ? 0.f : m_ref) - (kE4m3 ? 7.f : 0.f);
        uint32_t pk[kKpl / 2];
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
          float sum[2] = {0.f, 0.f};
#pragma unroll
          for (int k = 0; k < kSubKeys; k += 2) {
            const float p0 = ex2(x.f[sub * kSubKeys + k] - mu), p1 = ex2(x.f[sub * kSubKeys + k + 1] - mu);
            const uint32_t u = pack2<kE4m3>(p0, p1);
            pk[(sub * kSubKeys + k) / 2] = u;
            // The sum takes bf16 weights as rounded: their error then moves
            // the output by w (v - o) only. The f16 rounding is left out of it.
            if constexpr (kE4m3) {
              sum[0] += p0;
              sum[1] += p1;
            } else {
              sum[0] += __uint_as_float(u << 16);
              sum[1] += __uint_as_float(u & 0xffff0000u);
            }
          }
          if constexpr (kE4m3)
            l = fmaf(sum[0] + sum[1], rcp(sv[sub]), l);
          else
            l += sum[0] + sum[1];
        }
        tmem_store(tl + S::kColP + (n & 1) * (kBlk / 2) + key0 / 2, pk, Cols<kKpl / 2>{});
        tmem_wait_store();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(n & 1));
      }

      // ---- the tile's output, or this part's share of it ----
      if (!dead && !warp_wait(o_done((n - 1) & 1), ((n - 1) >> 1) & 1)) dead = true;
      tc_fence_after();
      const bool whole = w.blk == 0 && w.n_here == w.nb;
      const size_t slot = (size_t)blockIdx.x * 2 + (w.u == part0 ? 0 : 1);
      // Infinities and NaN that were held back from the product (rare), for
      // the rows that see them.
      auto add_odd = [&](float (&v)[32], int c0) {
        for (int ib = 0; ib < w.n_here; ++ib) {
          if (is_clean(w, ib)) continue;
          const int j0 = (w.first + w.blk + ib) * kBlk + key0;
          for (int k = 0; k < kKpl && j0 + k < w.L; ++k) {
            const bool seen = mine && (sight.mask(j0 + k) & 1u);
            const size_t from = (((size_t)w.b * A.Lmax + j0 + k) * A.Hkv + w.h) * kD + c0;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              float val;
              if constexpr (kE4m3) {
                const uint8_t code = static_cast<const uint8_t*>(A.v)[from + c];
                val = (code & 0x7fu) == 0x7fu ? __uint_as_float(0x7fffffffu) : 0.f;
              } else {
                const uint32_t u = static_cast<const uint16_t*>(A.v)[from + c];
                val = (u & 0x7f80u) == 0x7f80u ? __uint_as_float(u << 16) : 0.f;
              }
              if (seen && val != 0.f) v[c] += val;
            }
          }
        }
      };
      const bool has_odd = *odd != 0;
      if constexpr (S::kCopies == 1) {
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);       // NaN stays
        const size_t at_row =
            (((size_t)w.b * A.n_new + idx) * A.Hq + (size_t)w.h * A.G + gq) * kD;
#pragma unroll 1
        for (int c0 = 0; c0 < kD; c0 += 32) {
          if (dead) break;
          uint32_t u[32];
          tmem_load(tl + S::kColO + c0, u);
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(u[k]);
          if (has_odd) add_odd(v, c0);
          if (!mine) continue;
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(A.out + at_row + c0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[k] = make_uint4(pack2<false>(v[8 * k] * inv, v[8 * k + 1] * inv),
                                  pack2<false>(v[8 * k + 2] * inv, v[8 * k + 3] * inv),
                                  pack2<false>(v[8 * k + 4] * inv, v[8 * k + 5] * inv),
                                  pack2<false>(v[8 * k + 6] * inv, v[8 * k + 7] * inv));
          } else {
            float4* dst = reinterpret_cast<float4*>(A.part_o + (slot * kRP + row) * kD + c0);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          }
        }
        if (!whole && mine && !dead)
          *reinterpret_cast<float2*>(A.part_ml + (slot * kRP + row) * 2) = make_float2(m_ref, l);
      } else {
        // Merge the copies through shared memory, 32 columns at a time.
        const int lg = warp * 32 + lane;
        sts64(ml_tab + lg * 8, __float_as_uint(m_ref), __float_as_uint(l));
        named_bar_sync(1, 32 * kSoftWarps);
        float M = -INFINITY, lt = 0.f;
#pragma unroll
        for (int c = 0; c < S::kCopies; ++c)
          M = fmaxf(M, __uint_as_float(lds32(ml_tab + (c * kRP + row) * 8)));
        const float Mu = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int c = 0; c < S::kCopies; ++c)
          lt += __uint_as_float(lds32(ml_tab + (c * kRP + row) * 8 + 4)) *
                ex2(__uint_as_float(lds32(ml_tab + (c * kRP + row) * 8)) - Mu);
        const float wgt = ex2(m_ref - Mu);
        const float inv = lt > 0.f ? 1.f / lt : (lt == 0.f ? 0.f : lt);
        constexpr int kPer = 32 / S::kCopies;                    // columns a thread sums
        const size_t at_row =
            (((size_t)w.b * A.n_new + idx) * A.Hq + (size_t)w.h * A.G + gq) * kD;
#pragma unroll 1
        for (int c0 = 0; c0 < kD; c0 += 32) {
          if (!dead) {
            uint32_t u[32];
            tmem_load(tl + S::kColO + c0, u);
            float v[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(u[k]);
            if (has_odd) add_odd(v, c0);
#pragma unroll
            for (int k = 0; k < 32; ++k) sts32(stage + (lg * 33 + k) * 4, __float_as_uint(v[k] * wgt));
          }
          named_bar_sync(1, 32 * kSoftWarps);
          // thread (row, copy) sums columns copy * kPer ..
          float v[kPer];
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            v[k] = 0.f;
#pragma unroll
            for (int c = 0; c < S::kCopies; ++c)
              v[k] += __uint_as_float(lds32(stage + ((c * kRP + row) * 33 + copy * kPer + k) * 4));
          }
          if (mine && !dead) {
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(A.out + at_row + c0 + copy * kPer);
#pragma unroll
              for (int k = 0; k < kPer / 8; ++k)
                dst[k] = make_uint4(pack2<false>(v[8 * k] * inv, v[8 * k + 1] * inv),
                                    pack2<false>(v[8 * k + 2] * inv, v[8 * k + 3] * inv),
                                    pack2<false>(v[8 * k + 4] * inv, v[8 * k + 5] * inv),
                                    pack2<false>(v[8 * k + 6] * inv, v[8 * k + 7] * inv));
            } else {
              float4* dst =
                  reinterpret_cast<float4*>(A.part_o + (slot * kRP + row) * kD + c0 + copy * kPer);
#pragma unroll
              for (int k = 0; k < kPer / 4; ++k)
                dst[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
          }
          named_bar_sync(1, 32 * kSoftWarps);
        }
        if (!whole && mine && !dead && copy == 0)
          *reinterpret_cast<float2*>(A.part_ml + (slot * kRP + row) * 2) = make_float2(M, lt);
      }
    }
  }
  tc_fence_before();
  __syncthreads();   // every role has left its loop
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
  if (*abort && warp == kProducer && lane == 0)
    // A wait gave up: let every copy already issued land before the CTA exits.
    for (int s = 0; s < kR; ++s) {
      if (issued[0] & (1u << s)) wait_drain(k_full(s), (issued_phase[0] >> s) & 1u);
      if (issued[1] & (1u << s)) wait_drain(v_full(s), (issued_phase[1] >> s) & 1u);
      if (!kE4m3 && s < kNq && (issued[2] & (1u << s))) wait_drain(q_full(s), (issued_phase[2] >> s) & 1u);
    }
}

// Merges the partials of the tiles that more than one CTA worked on, and
// zeroes the outputs of sequences without blocks. One warp per query row:
// blockIdx.x = tile, blockIdx.y * 8 + warp = row of its group.
template <bool kE4m3, int kD, int kRP>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ CacheAttnLaunch A, int n_ctas) {
  constexpr int kBlk = cache_attn_block(kE4m3, kD);
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
    const int nb = seq_blocks<kBlk>(A, A.seq_lens[x], first, bad);
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
  const int nb = seq_blocks<kBlk>(A, A.seq_lens[b], first, bad);
  const long long per = (long long)A.Hkv * A.n_groups;
  total *= per;
  const long long u0 = before * per + (long long)(h * A.n_groups + grp) * nb;
  const int pos0 = grp * A.group_pos;
  const int r = blockIdx.y * 8 + warp;
  if (r >= min(A.group_pos, A.n_new - pos0) * A.G) return;
  constexpr int kPer = kD / 32;
  __nv_bfloat16* dst = A.out +
                       (((size_t)b * A.n_new + pos0 + r / A.G) * A.Hq + (size_t)h * A.G + r % A.G) * kD +
                       lane * kPer;
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
      M = fmaxf(M, A.part_ml[(slot * kRP + r) * 2]);
    }
    M = warp_max(M);
    const float mu = M == -INFINITY ? 0.f : M;
    float l = 0.f;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      const long long pb = part_begin(total, c, n_ctas);
      if (pb == part_begin(total, c + 1, n_ctas)) continue;
      const size_t slot = (size_t)c * 2 + (c == c0 && pb != u0 ? 1 : 0);
      const float2 ml = *reinterpret_cast<const float2*>(A.part_ml + (slot * kRP + r) * 2);
      const float wgt = ex2(ml.x - mu);
      l += ml.y * wgt;
      const float* po = A.part_o + (slot * kRP + r) * kD + lane * kPer;
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

template <bool kE4m3, int kD, int kRP, bool kExtra>
cudaError_t launch_one(const CacheAttnLaunch& A, const CUtensorMap& tk, const CUtensorMap& tv,
                       const CUtensorMap& tq, cudaStream_t stream) {
  using S = Shape<kE4m3, kD, kRP>;
  static std::atomic<int> smem_set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !smem_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(cache_attn_kernel<kE4m3, kD, kRP, kExtra>,
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
  e = cudaLaunchKernelEx(&cfg, cache_attn_kernel<kE4m3, kD, kRP, kExtra>, A, tk, tv, tq);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)tiles, (A.group_pos * A.G + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, combine_kernel<kE4m3, kD, kRP>, A, grid);
}

template <bool kE4m3, int kD, int kRP>
cudaError_t launch_extra(const CacheAttnLaunch& A, const CUtensorMap& tk, const CUtensorMap& tv,
                         const CUtensorMap& tq, cudaStream_t stream) {
  return A.cap > 0.f || A.slopes ? launch_one<kE4m3, kD, kRP, true>(A, tk, tv, tq, stream)
                                 : launch_one<kE4m3, kD, kRP, false>(A, tk, tv, tq, stream);
}

// Rows per copy: the fewest of 32, 64 and 128 lanes that hold a group.
template <bool kE4m3, int kD>
cudaError_t launch_rows(const CacheAttnLaunch& A, const CUtensorMap& tk, const CUtensorMap& tv,
                        const CUtensorMap& tq, cudaStream_t stream) {
  switch (cache_attn_rows(A.group_pos * A.G)) {
    case 32: return launch_extra<kE4m3, kD, 32>(A, tk, tv, tq, stream);
    case 64: return launch_extra<kE4m3, kD, 64>(A, tk, tv, tq, stream);
    default: return launch_extra<kE4m3, kD, 128>(A, tk, tv, tq, stream);
  }
}

}  // namespace cache_attn
}  // namespace specdec
