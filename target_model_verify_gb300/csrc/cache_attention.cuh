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
// rows). Measured on a GB300 (graph replays; copy peak 6771 GB/s): 64 x 4096
// bf16 rows, 5 positions, 32 query / 8 KV heads of 128: 160 us for 1074 MB,
// 0.99 of the copy peak (16 positions: 160 us); a tree of 26 over 8 x 4096:
// 35 us for 136 MB, where starting, the softmax of 128 lanes and the merge
// show; the tree over 32 x 4096 e4m3 rows: 103 us for 268 MB (131 with a
// bias), bound by the softmax (one warp per scheduler takes 0.9 us for a
// lane's 64 scores).
//
// Schedule. A tile is a (sequence, KV head, row group), a run of cache blocks
// as long as its own sequence (or window). A head's tiles are laid end to end
// and cut into equal parts, on the device from seq_lens, so ragged batches
// keep every SM busy to the end. Part p of head h goes to CTA p * Hkv + h:
// the heads' CTAs go through the same cache rows at the same time, and since
// a row of the cache holds all its heads side by side, DRAM pages are read
// whole. A tile that lies inside one part is finished by its CTA; of the
// others every CTA leaves a partial (maximum, sum, unnormalised output), and
// the one with its first block a note of who shares it, from which
// combine_kernel merges.
// (The last CTA of a tile merging in place, counted in by an atomic, was
// slower in every case measured, by 1 to 12 us a call: its four warps take
// the rows one batch after another while the grid waits.)
//
// CTA: warps 0-3 softmax, 4-7 auxiliary, 8 and 9 TMA producers (K with Q,
// and V, whose slots free up at different times), 10 and 11 tcgen05 issuers
// (one per product: a thread takes 50 to 100 cycles for each MMA, as long as
// the MMA itself, and more for each wait). What an earlier kernel may have
// written (queries, scales) is not read with ld.global.nc: this kernel can
// begin before that one ends.
//   S = Q K^T: tcgen05.mma, M = 128 query rows, N = a block of keys, into one
//     of two tensor-memory buffers, a block ahead of the softmax. bf16:
//     kind::f16. e4m3: kind::f8f6f4 on the codes as they lie; the query row,
//     scaled by a power of two to below 256, is the sum of two e4m3 terms
//     (4 + 4 significant bits hold a bf16 value exactly down to 2^-9 of the
//     row's largest, and to within 2^-17 of it below), so two products accumulate.
//   softmax: lane = query row, so maxima and sums need no exchange. With
//     R <= 64 query rows the 128 lanes hold 128 / RP copies of the rows (RP =
//     32 or 64) and each copy takes its own share of every block's keys; its
//     probabilities go to its share's columns of the P operand, whose other
//     columns stay zero, so the copies are independent online softmaxes,
//     merged once per tile. The reference M moves only when a row's maximum
//     passes it by 2^8 (the exponents have that headroom), so the output in
//     tensor memory is rarely rescaled. f16 probabilities (e4m3 caches) have
//     normal numbers down to 2^-21 of M: a block that stays below that moves M
//     to 2^24 below its highest, so that the many small weights beside a
//     dominant one keep their precision, down to 2^-45 of it; no further, so
//     that sums and outputs stay finite. bf16 ones have fp32's exponents. Code for rare blocks (masks, moving
//     references, huge exponents) stands outside the loop's line: the loop is
//     longer than the nearest instruction cache, and jumps over unrolled code
//     cost 500 cycles a block with a bias.
//   O += P V: P from tensor memory, V the MN-major operand, kind::f16. e4m3
//     values are widened to f16 (exact) by the auxiliary warps into a second
//     shared-memory tile, since P needs f16's 11 bits and both operands share
//     a type; bf16 values are used as they land, and P is bf16 for the same
//     reason (the sum takes it as rounded, see below).
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "kernels.h"

namespace specdec {
namespace cache_attn {

constexpr int kSoftWarps = 4;
constexpr int kAuxWarps = 4;
constexpr int kProducer = 8, kProducerV = 9, kIssuerS = 10, kIssuerO = 11;   // warp indices
constexpr int kThreads = 384;
constexpr unsigned long long kDrainNs = 1000000000ull;
constexpr int kStagePitch = 36 * 4;           // bytes: 32 floats, 16-byte accesses free of bank conflicts
constexpr float kHeadroom = 8.f;              // log2 by which a maximum may pass its reference,
constexpr float kBelow = 21.f;                // and stay below it (f16 probabilities)
constexpr float kNear = 17.f;                 // (this far, when its warp rescales anyway)
constexpr float kDeep = 24.f;                 // log2 by which a reference goes below its highest,
constexpr float kReach = 45.f;                // for blocks no further below that than this
constexpr int kSmemLimit = 227 * 1024;
constexpr int kTileCost = 3;                  // units of work that a tile costs besides its blocks

template <bool kE4m3, int kD, int kRP>
struct Shape {
  static constexpr int kElem = kE4m3 ? 1 : 2;
  static constexpr int kBlk = cache_attn_block(kD, kRP);   // keys per block
  static constexpr int kRowBytes = kD * kElem;
  static constexpr int kPanelBytes = kRowBytes < 128 ? kRowBytes : 128;   // one TMA box row
  static constexpr int kPanels = kRowBytes / kPanelBytes;
  static constexpr int kSlotBytes = kBlk * kRowBytes;        // a block of K, or of V, as it lands
  static constexpr int kCopies = 128 / kRP;                  // copies of the query rows
  static constexpr int kKpl = kBlk / kCopies;                // keys per lane and block
  static constexpr int kTerms = kE4m3 ? 2 : 1;
  // Queries: e4m3 terms sit in tensor memory where it has room for them
  // (shared memory bandwidth is what the e4m3 products compete for), else
  // 128 rows in the K operand's layout in shared memory.
  static constexpr bool kQTmem = kE4m3 && kD <= 128;
  static constexpr int kQTerm = 128 * kRowBytes;
  static constexpr int kQBytes = kQTmem ? 0 : kTerms * kQTerm;
  static constexpr int kQBufs = !kE4m3 && kD <= 128 ? 2 : 1;
  // two P buffers where tensor memory has room for them
  static constexpr int kPBufs = 3 * kBlk + kD + (kQTmem ? kTerms * (kD / 4) : 0) <= 512 ? 2 : 1;
  static constexpr int kV16Bytes = kE4m3 ? kBlk * kD * 2 : 0;   // widened V, two of them
  static constexpr int kStageBytes = 128 * kStagePitch;      // 32 output columns of every lane
  static constexpr int kTabBytes = 128 * 4 + 128 * 8 + 128 * 4 + 128 * 16 + 128 * 4;  // q scales, (m, l), places, tree
  static constexpr int kFixed = 1024 + 2 * kV16Bytes + kQBufs * kQBytes + kStageBytes + kTabBytes + 512;
  static constexpr int kRingMax = (kSmemLimit - kFixed) / (2 * kSlotBytes);
  static constexpr int kRing = kRingMax < 6 ? kRingMax : 6;  // K blocks (and V blocks) in flight
  static constexpr int kSmem = kFixed + 2 * kRing * kSlotBytes;
  static_assert(kRing >= 2, "two K and two V blocks must fit");
  // tensor memory columns: two score buffers, the output, P, the query terms
  static constexpr int kColS = 0, kColO = 2 * kBlk, kColP = kColO + kD, kColQ = kColP + kPBufs * (kBlk / 2);
  static_assert(kColQ + (kQTmem ? kTerms * (kD / 4) : 0) <= 512, "tensor memory");
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
// log2(e) cap tanh(z / cap), cap * tanh(z / cap) = cap * (1 - 2 / (1 + e^(2 z / cap))),
// from 2 log2(e) z / cap. Off by about 2^-22 cap, less than the probabilities'
// rounding for the caps allowed (up to 1000).
__device__ __forceinline__ float capped(float z_cap_exp, float cap_log2e, float plus) {   // plus = the cap + a bias
  return fmaf(-2.f * cap_log2e, rcp(1.f + ex2(z_cap_exp)), plus);
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
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
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
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
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
// The same with A in tensor memory: a row per lane, 32-bit columns of two
// 16-bit or four 8-bit elements along k.
template <bool kF8>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (kF8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ void fma2(float& a, float& b, float c, float d, float e, float f) {   // a c + e, b d + f
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tmov.b64 z, {%4, %5};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d), "f"(e), "f"(f));
}
__device__ __forceinline__ void fma2(float& a, float& b, float c, float d) { fma2(a, b, c, c, d, d); }
__device__ __forceinline__ void acc2(float& a, float& b, float c, float d, float e) {   // a += c e, b += d e
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tmov.b64 z, {%4, %4};\n\t"
      "fma.rn.f32x2 x, y, z, x;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d), "f"(e));
}
__device__ __forceinline__ void mul2(float& a, float& b, float c, float d) {   // a *= c, b *= d
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {   // a += c, b += d
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
template <int kN>
__device__ __forceinline__ float largest(const float* y) {      // kN = 16 or 32
  float a = max3(y[0], y[1], y[2]), b = max3(y[3], y[4], y[5]);
#pragma unroll
  for (int k = 6; k + 3 < kN; k += 4) {
    a = max3(a, y[k], y[k + 1]);
    b = max3(b, y[k + 2], y[k + 3]);
  }
  return fmaxf(max3(a, y[kN - 2], y[kN - 1]), b);
}
__device__ __forceinline__ float4 lds128f(uint32_t a) {
  const uint4 v = lds128(a);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
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
__device__ __forceinline__ void tmem_wait_store() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// What the schedule knows of a sequence: the blocks of kBlk cache rows it
// reads, all or those inside the window of its first new position (the one
// that sees furthest back), and the first of them. A length of 0 marks an
// unused batch slot; bad: a length that the cache cannot hold.
template <int kBlk>
__device__ __forceinline__ int seq_blocks(const CacheAttnLaunch& A, int L, int& first, bool& bad) {
  bad = L != 0 && (L < A.n_new || L > A.Lmax);
  first = 0;
  if (L == 0 || bad) return 0;
  if (A.window > 0) first = max(0, L - A.n_new - A.window + 1) / kBlk;
  return (L + kBlk - 1) / kBlk - first;
}

// Units of work of a tile of nb blocks: starting and writing out a tile
// costs about kTileCost blocks, which come first.
__device__ __forceinline__ int tile_units(int nb) { return nb > 0 ? nb + kTileCost : 0; }

// The first unit of CTA c's part, of n: equal parts to within a unit.
__device__ __forceinline__ int part_begin(int total, int c, int n) {
  return total / n * c + (int)((unsigned)(total % n) * (unsigned)c / (unsigned)n);
}

// CTAs beside each other on one part: one per KV head, or, with too many heads
// for that, one that takes all heads' tiles.
__device__ __forceinline__ int heads_of(const CacheAttnLaunch& A) { return A.head_lanes > 1 ? 1 : A.Hkv; }

// One warp: the units of a head lane, and where unit part_begin(c) lies:
// sequence b (B when there is none) and offset inside it.
struct Place {
  int total, parts, u0, u1, b, off;      // parts: those with units, of n
  bool any_bad;
};
template <int kBlk>
__device__ __forceinline__ Place find_part(const CacheAttnLaunch& A, int lane, int c, int n) {
  const int per = heads_of(A) * A.n_groups;
  Place p;
  int first, units0 = 0, sum = 0;
  bool bad, bad_seen = false;
  for (int b = lane; b < A.B; b += 32) {
    const int u = per * tile_units(seq_blocks<kBlk>(A, A.seq_lens[b], first, bad));
    if (b < 32) units0 = u;                    // the first 32 sequences stay at hand
    sum += u;
    bad_seen |= bad;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  p.any_bad = __any_sync(0xffffffffu, bad_seen);
  p.total = sum;
  p.parts = min(n, sum);
  p.u0 = p.u1 = 0;
  p.b = A.B;
  p.off = 0;
  if (c >= p.parts) return p;
  p.u0 = part_begin(sum, c, p.parts);
  p.u1 = part_begin(sum, c + 1, p.parts);
  int before = 0;
  for (int b0 = 0; b0 < A.B; b0 += 32) {
    const int b = b0 + lane;
    const int mine = b0 == 0 ? units0
                     : b < A.B ? per * tile_units(seq_blocks<kBlk>(A, A.seq_lens[b], first, bad)) : 0;
    int run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, p.u0 < before + run);
    if (hit) {
      const int l = __ffs(hit) - 1;
      p.b = b0 + l;
      p.off = p.u0 - before - __shfl_sync(0xffffffffu, run - mine, l);
      return p;
    }
    before += __shfl_sync(0xffffffffu, run, 31);
  }
  return p;
}

// Walks the tiles of a part: (b, h, group) and the block range inside each.
template <int kBlk>
struct Walk {
  int b, h, g, h0;    // tile, the part's first head
  int blk, n_here;    // first block inside the tile, blocks of this part
  int nb, first, L;   // the tile's blocks, its first cache block, its length
  int clean_lo, clean_hi;   // the tile's blocks that every new position sees whole
  bool backward;            // the order of the blocks: see at()
  int u, end, tile0;  // this part's first unit in the tile, the part's end, the tile's first unit

  __device__ __forceinline__ void load(const CacheAttnLaunch& A) {
    bool bad;
    L = A.seq_lens[b];
    nb = seq_blocks<kBlk>(A, L, first, bad);
    const int P0 = L - A.n_new;               // row and position of the first new one
    clean_hi = (P0 + 1) / kBlk - first;
    clean_lo = A.window > 0 ? (max(0, P0 + A.max_depth - A.window + 1) + kBlk - 1) / kBlk - first : 0;
  }
  __device__ __forceinline__ void cut() {
    const int to = min(tile0 + tile_units(nb), end);
    blk = max(0, u - tile0 - kTileCost);
    n_here = max(0, to - tile0 - kTileCost) - blk;
  }
  __device__ __forceinline__ void start(const CacheAttnLaunch& A, int b0, int off, int u0, int u1) {
    u = u0;
    end = u1;
    b = b0;
    backward = A.slopes != nullptr;
    if (u >= end) return;
    load(A);
    const int units = tile_units(nb), t = off / units;
    tile0 = u - (off - t * units);
    g = t % A.n_groups;
    h0 = A.head_lanes > 1 ? (int)blockIdx.x % A.head_lanes : 0;
    h = h0 + t / A.n_groups;
    cut();
    if (n_here == 0) next(A);
  }
  __device__ __forceinline__ bool done() const { return u >= end; }
  // To the next tile, and past one of which this part has only the leading units.
  __device__ __forceinline__ void next(const CacheAttnLaunch& A) {
    do {
      u = tile0 = tile0 + tile_units(nb);
      if (u >= end) return;
      if (++g == A.n_groups) {
        g = 0;
        if (++h == h0 + heads_of(A)) {
          h = h0;
          do {
            ++b;
            load(A);
          } while (nb == 0);
        }
      }
      cut();
    } while (n_here == 0);
  }
  // This part's block i, in the order in which they are taken: from the
  // sequence's start, but from its end with a bias by distance, which makes
  // the last rows' exponents the largest: the references then move at the
  // tile's first block only. 23.7 against 24.5 us in this order for a tree of
  // 26 over 8 ragged sequences of up to 3001 rows (e4m3, 64 dims), 10.1 against
  // 10.5 for a chain of 3 over 3 of 1003 (bf16).
  __device__ __forceinline__ int at(int i) const { return blk + (backward ? n_here - 1 - i : i); }
  __device__ __forceinline__ int row(int i) const { return (first + at(i)) * kBlk; }
  __device__ __forceinline__ bool clean(int i) const { return at(i) >= clean_lo && at(i) < clean_hi; }
};

// What the CTA with a tile's first block notes for the merge: the sequence
// (-1: nothing to merge), KV head and row group, the last part with blocks of
// it, its own part and which of its two partials is the tile's.
__device__ __forceinline__ void write_note(const CacheAttnLaunch& A, int b, int h, int g, bool whole, int last,
                                           int slot) {
  A.notes[A.note_tiles ? (b * A.Hkv + h) * A.n_groups + g : blockIdx.x] =
      make_int4(whole ? -1 : b, h * A.n_groups + g, last, (int)(blockIdx.x / A.head_lanes) * 2 + slot);
}
// The part that holds the walk's tile's last unit.
template <int kBlk>
__device__ __forceinline__ int last_part(const Walk<kBlk>& w, int total, int parts) {
  // part c holds unit u iff part_begin(c) <= u < part_begin(c + 1)
  return (int)(((unsigned long long)(w.tile0 + tile_units(w.nb)) * parts - 1) / total);
}

// Outputs of sequences without blocks are zero: the softmax warps of the grid
// share them out.
template <int kD, int kBlk>
__device__ __forceinline__ void zero_empty(const CacheAttnLaunch& A) {
  for (int b = blockIdx.x; b < A.B; b += gridDim.x) {
    int first;
    bool bad;
    if (seq_blocks<kBlk>(A, A.seq_lens[b], first, bad) > 0) continue;
    if (A.note_tiles)
      for (int e = threadIdx.x; e < A.Hkv * A.n_groups; e += 32 * kSoftWarps)
        A.notes[b * A.Hkv * A.n_groups + e].x = -1;
    uint4* dst = reinterpret_cast<uint4*>(A.out + (size_t)b * A.n_new * A.Hq * kD);
    const long long chunks = (long long)A.n_new * A.Hq * (kD / 8);
    for (long long e = threadIdx.x; e < chunks; e += 32 * kSoftWarps) dst[e] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// Merges the partials of the tiles that more than one CTA worked on.
// blockIdx.x = the note, blockIdx.y: rows. `wpr` of the eight warps share the
// partials of kRows rows, which they take together, so that eight loads are in
// flight either way.
template <int kD, int kRP>
struct MergeShape {
  static constexpr int kRows = kRP / 32;                    // 1, 2 or 4
  static constexpr int kParts = 8 / kRows;
};
template <int kD, int kRP>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ CacheAttnLaunch A, int wpr) {
  constexpr int kPer = kD / 32, kRows = MergeShape<kD, kRP>::kRows, kParts = MergeShape<kD, kRP>::kParts;
  __shared__ float part[8][kRows][kD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  const int4 note = __ldcg(A.notes + blockIdx.x);
  // A bad length's code comes now, when a wait that ran out has left its own,
  // which spoils every output and stays.
  const int bad_lens = blockIdx.x == 0 && blockIdx.y == 0 ? __ldcg(A.status + 1) : 0;
  if (bad_lens && threadIdx.x == 0) set_status(A.status, SPECDEC_ERR_INVALID_ARG);
  if (note.x < 0) return;
  const int b = note.x, grp = note.y % A.n_groups, h = note.y / A.n_groups;
  const int pos0 = grp * A.group_pos, rows = min(A.group_pos, A.n_new - pos0) * A.G;
  const int r0 = (blockIdx.y * (8 / wpr) + warp / wpr) * kRows, slice = warp % wpr;
  const int first = note.w >> 1, head_lane = A.head_lanes > 1 ? h : 0;
  float acc[kRows][kPer], l[kRows], M[kRows];
#pragma unroll
  for (int y = 0; y < kRows; ++y) {
    l[y] = 0.f;
    M[y] = -INFINITY;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[y][k] = 0.f;
  }
  if (r0 < rows) {
    // a lane looks after every 32nd part's statistics and kPer dims
    for (int cb = first; cb <= note.z; cb += 32) {
      const int c = min(cb + lane, note.z), here = min(32, note.z - cb + 1);
      const bool none = cb + lane > note.z;
      const int slot = 2 * (c * A.head_lanes + head_lane) + (c == first ? note.w & 1 : 0);
      float2 ml[kRows];
      float wgt[kRows];
#pragma unroll
      for (int y = 0; y < kRows; ++y)
        ml[y] = __ldcg(reinterpret_cast<const float2*>(A.part_ml) + (size_t)slot * kRP + min(r0 + y, rows - 1));
#pragma unroll
      for (int y = 0; y < kRows; ++y) {
        if (none) ml[y] = make_float2(-INFINITY, 0.f);
        const float m_new = fmaxf(M[y], warp_max(ml[y].x));
        const float mu = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = ex2(M[y] - mu);
        wgt[y] = none ? 0.f : ex2(ml[y].x - mu);
        l[y] = fmaf(l[y], alpha, warp_sum(none ? 0.f : ml[y].y * wgt[y]));
        M[y] = m_new;
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[y][k] *= alpha;
      }
      for (int x0 = slice; x0 < here; x0 += kParts * wpr) {
        float2 v[kParts][kRows][kPer / 2];
#pragma unroll
        for (int x = 0; x < kParts; ++x) {
          const int s = __shfl_sync(0xffffffffu, slot, min(x0 + x * wpr, here - 1));
#pragma unroll
          for (int y = 0; y < kRows; ++y) {
            const float2* po = reinterpret_cast<const float2*>(
                A.part_o + ((size_t)s * kRP + min(r0 + y, rows - 1)) * kD + lane * kPer);
#pragma unroll
            for (int k = 0; k < kPer / 2; ++k)
              v[x][y][k] = x0 + x * wpr < here ? __ldcg(po + k) : make_float2(0.f, 0.f);
          }
        }
#pragma unroll
        for (int x = 0; x < kParts; ++x)
#pragma unroll
          for (int y = 0; y < kRows; ++y) {
            const float w = __shfl_sync(0xffffffffu, wgt[y], min(x0 + x * wpr, here - 1));
            const float f = x0 + x * wpr < here ? w : 0.f;
#pragma unroll
            for (int k = 0; k < kPer / 2; ++k) {
              acc[y][2 * k] = fmaf(v[x][y][k].x, f, acc[y][2 * k]);
              acc[y][2 * k + 1] = fmaf(v[x][y][k].y, f, acc[y][2 * k + 1]);
            }
          }
      }
    }
  }
  if (wpr > 1) {
#pragma unroll
    for (int y = 0; y < kRows; ++y)
#pragma unroll
      for (int k = 0; k < kPer; ++k) part[warp][y][lane * kPer + k] = acc[y][k];
    __syncthreads();
    if (slice) return;
    for (int x = 1; x < wpr; ++x)
#pragma unroll
      for (int y = 0; y < kRows; ++y)
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[y][k] += part[warp + x][y][lane * kPer + k];
  }
#pragma unroll
  for (int y = 0; y < kRows; ++y) {
    const int r = r0 + y;
    if (r >= rows) return;
    const float inv = l[y] > 0.f ? 1.f / l[y] : (l[y] == 0.f ? 0.f : l[y]);       // NaN stays
    uint32_t* dst = reinterpret_cast<uint32_t*>(
        A.out + (((size_t)b * A.n_new + pos0 + r / A.G) * A.Hq + (size_t)h * A.G + r % A.G) * kD + lane * kPer);
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k) dst[k] = pack2<false>(acc[y][2 * k] * inv, acc[y][2 * k + 1] * inv);
  }
}

// Parts of the schedule: as many as the CTAs (or the work, `most` units in
// all heads at the longest) allow.
inline int cache_attn_parts(const CacheAttnLaunch& A, int ctas, long long most) {
  const long long by_work = (most + A.head_lanes - 1) / A.head_lanes, by_ctas = ctas / A.head_lanes;
  return (int)(by_work < by_ctas ? by_work : by_ctas);
}

// A note per tile where there are no more tiles than CTAs (the merge then has
// fewer CTAs that find nothing to do), else a note per CTA.
inline int note_tiles(const CacheAttnLaunch& A, int parts) {
  const long long tiles = (long long)A.B * A.Hkv * A.n_groups;
  return tiles <= (long long)parts * A.head_lanes ? (int)tiles : 0;
}

// The merge, after the attention kernel on the same stream. Warps per row:
// as many as a tile has parts when the parts are dealt out evenly, and more
// where the grid stays within two CTAs per SM (8 ragged sequences of 256 dims
// with a window: 17.4 -> 16.8 us), at most 8.
template <int kD, int kRP>
cudaError_t launch_combine(const CacheAttnLaunch& A, int parts, cudaLaunchConfig_t& cfg) {
  const long long tiles = (long long)A.B * A.n_groups * (A.head_lanes > 1 ? 1 : A.Hkv);
  const long long each = parts / tiles;
  const int rows = A.group_pos * A.G;
  int wpr = each >= 8 ? 8 : each >= 4 ? 4 : each >= 2 ? 2 : 1;
  auto row_ctas = [&](int w) {
    const int per_cta = 8 / w * MergeShape<kD, kRP>::kRows;
    return (rows + per_cta - 1) / per_cta;
  };
  while (A.note_tiles && wpr < 8 && A.note_tiles * row_ctas(2 * wpr) <= 2 * kCacheAttnCtas) wpr *= 2;
  cfg.gridDim = dim3(A.note_tiles ? A.note_tiles : parts * A.head_lanes, row_ctas(wpr));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, combine_kernel<kD, kRP>, A, wpr);
}

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
  const uint32_t q_tab = stage + S::kStageBytes;           // query row scales, by lane
  const uint32_t ml_tab = q_tab + 128 * 4;                 // (reference, sum) of every lane
  const uint32_t place_tab = ml_tab + 128 * 8;             // a row's place in the output, by lane
  const uint32_t tree = place_tab + 128 * 4;               // [128][4] ancestor words, then depth [128]
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
  // One per block parity: the softmax takes note of every phase of each.
  auto o_done = [&](int s) { return bars2 + 8u * (uint32_t)(12 + s); };
  auto s_empty = [&](int s) { return bars2 + 8u * (uint32_t)(14 + s); };
  const uint32_t drained = bars2 + 8u * 16;
  uint8_t* const words = smem_raw + (bars2 + 8u * 18 - raw);
  volatile int* const abort = reinterpret_cast<volatile int*>(words);
  volatile int* const odd = abort + 1;                     // a value that is no number was held back
  volatile uint32_t* const tmem_slot = reinterpret_cast<volatile uint32_t*>(words) + 2;
  volatile int* const place = abort + 4;                   // find_part's answer

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
      mbar_init(s_empty(s), kSoftWarps);
      mbar_init(o_done(s), 1);
      mbar_init(p_full(s), kSoftWarps);
      mbar_init(q_full(s), kE4m3 ? kAuxWarps : 1);
      mbar_init(q_empty(s), kE4m3 ? 1 + kSoftWarps : 1);
      mbar_init(v16_full(s), kAuxWarps);
      mbar_init(v16_empty(s), 1);
    }
    mbar_init(drained, 2);
    *abort = 0;
    *odd = 0;
    fence_mbar_init();
  }
  if (warp == kIssuerO) tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
  if (A.tree) {
    // not by warp 0, which looks for its part meanwhile
    for (int e = (int)threadIdx.x - 32; e >= 0 && e < A.n_new; e += kThreads - 32) {
      sts128(tree + e * 16, A.anc[e][0], A.anc[e][1], A.anc[e][2], A.anc[e][3]);
      sts32(tree + 128 * 16 + e * 4, A.depth[e]);
    }
  }
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
  // A warp's wait: all lanes agree on whether it ran out.
  auto warp_wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait<true>(bar, parity, abort, A.status));
  };
  uint32_t issued = 0, issued_phase = 0, issued_q = 0, issued_q_phase = 0;   // producers: copies in flight

  if (warp == kProducer || warp == kProducerV) {
    // --------------------------------------- producers: K and Q; V --
    if (lane == 0) {
      const bool is_v = warp == kProducerV;
      const uint64_t pol = policy_evict_first();
      const CUtensorMap* const map = is_v ? &tmap_v : &tmap_k;
      const uint32_t ring = is_v ? ring_v : ring_k;
      int s = 0;
      uint32_t ph = 0, nt = 0;
      bool ok = true;
      for (; ok && !w.done(); w.next(A), ++nt) {
        if (!kE4m3 && !is_v) {
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
          issued_q |= 1u << qs;
          issued_q_phase = (issued_q_phase & ~(1u << qs)) | (qph << qs);
        }
        for (int i = 0; i < w.n_here; ++i) {
          const int j0 = w.row(i);
          const uint32_t full = is_v ? v_full(s) : k_full(s);
          if (!(ok = mbar_wait(is_v ? v_empty(s) : k_empty(s), ph ^ 1u, abort, A.status))) break;
          mbar_arrive_expect_tx(full, (uint32_t)S::kSlotBytes);
#pragma unroll
          for (int p = 0; p < S::kPanels; ++p)
            tma_load_4d(ring + s * S::kSlotBytes + p * kBlk * S::kPanelBytes, map, full,
                        p * (S::kPanelBytes / S::kElem), w.h, j0, w.b, pol);
          issued |= 1u << s;
          issued_phase = (issued_phase & ~(1u << s)) | (ph << s);
          if (++s == kR) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else if (warp == kIssuerS) {
    // --------------------------------------------------- issuer of Q K^T --
    // Scores run up to two blocks ahead of the softmax's answer.
    constexpr uint32_t id_qk = instr_desc(kE4m3 ? 0 : 1, false, kBlk);
    const uint64_t q_desc = operand_desc<S::kPanelBytes>(qb, 16);
    const uint64_t k_desc = operand_desc<S::kPanelBytes>(ring_k, 16);
    int s = 0;
    uint32_t ph = 0, n = 0, nt = 0;
    bool ok = true;
    for (; ok && !w.done(); w.next(A), ++nt) {
      const int qs = nt % kNq;
      if (!(ok = warp_wait(q_full(qs), (nt / kNq) & 1))) break;
      const uint64_t qd = q_desc + (uint64_t)((uint32_t)(qs * S::kQBytes) >> 4);
      for (int i = 0; i < w.n_here; ++i, ++n) {
        if (!(ok = warp_wait(k_full(s), ph))) break;
        // the buffer's previous scores are in the softmax's registers
        if (n >= 2 && !(ok = warp_wait(s_empty(n & 1), ((n - 2) >> 1) & 1))) break;
        tc_fence_after();
        const uint64_t kd = k_desc + (uint64_t)((uint32_t)(s * S::kSlotBytes) >> 4);
        const uint32_t d = tmem + S::kColS + (n & 1) * kBlk;
        if (elect_one()) {
#pragma unroll
          for (int term = 0; term < S::kTerms; ++term)
#pragma unroll
            for (int p = 0; p < S::kPanels; ++p)
#pragma unroll
              for (int k = 0; k < S::kPanelBytes / 32; ++k) {
                const uint64_t b = kd + (uint64_t)((p * kBlk * S::kPanelBytes + k * 32) >> 4);
                if constexpr (S::kQTmem)
                  mma_ts<true>(d, tmem + S::kColQ + term * (kD / 4) + p * (S::kPanelBytes / 4) + k * 8, b, id_qk,
                               term + p + k > 0);
                else
                  mma_ss<kE4m3>(d, qd + (uint64_t)((term * S::kQTerm + p * 128 * S::kPanelBytes + k * 32) >> 4), b,
                                id_qk, term + p + k > 0);
              }
          tc_commit(s_full(n & 1));
          tc_commit(k_empty(s));
          if (i + 1 == w.n_here) tc_commit(q_empty(qs));
        }
        __syncwarp();
        if (++s == kR) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (elect_one()) tc_commit(drained);
    wait_drain(drained, 0);
  } else if (warp == kIssuerO) {
    // ----------------------------------------------------- issuer of P V --
    constexpr uint32_t id_pv = instr_desc(kE4m3 ? 0 : 1, true, kD);
    const uint64_t v_desc = operand_desc<128>(kE4m3 ? v16 : ring_v, kBlk * 128);
    int s = 0;
    uint32_t ph = 0, n = 0, clean_ph = 0;
    bool ok = true;
    for (; ok && !w.done(); w.next(A))
      for (int i = 0; i < w.n_here; ++i, ++n) {
        uint64_t vd;
        if constexpr (kE4m3) {
          vd = v_desc + (uint64_t)((uint32_t)((n & 1) * S::kV16Bytes) >> 4);
          if (!(ok = warp_wait(v16_full(n & 1), (n >> 1) & 1))) break;
        } else {
          vd = v_desc + (uint64_t)((uint32_t)(s * S::kSlotBytes) >> 4);
          if (!(ok = warp_wait(v_full(s), ph))) break;
          if (!w.clean(i)) {
            if (!(ok = warp_wait(v_clean(s), (clean_ph >> s) & 1))) break;
            clean_ph ^= 1u << s;
          }
        }
        if (!(ok = warp_wait(p_full(n & 1), (n >> 1) & 1))) break;
        tc_fence_after();
        const uint32_t pa = tmem + S::kColP + (S::kPBufs == 2 ? (n & 1) * (kBlk / 2) : 0);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBlk / 16; ++k)
            mma_ts<false>(tmem + S::kColO, pa + k * 8, vd + (uint64_t)(k * 2048 >> 4), id_pv, i > 0 || k > 0);
          tc_commit(o_done(n & 1));
          tc_commit(kE4m3 ? v16_empty(n & 1) : v_empty(s));
        }
        __syncwarp();
        if (++s == kR) {
          s = 0;
          ph ^= 1u;
        }
      }
    // every product has to be done before the tensor memory is given back
    if (elect_one()) tc_commit(drained);
    wait_drain(drained, 0);
  } else if (warp >= kSoftWarps) {
    // --------------------------------------------------------- auxiliary --
    const int at = threadIdx.x - 32 * kSoftWarps;      // 0 .. 127
    bool ok = true;
    if constexpr (kE4m3) {
      // A tile's query rows as two e4m3 terms each. In tensor memory: thread
      // = lane = row, 16 dims at a time; its scale from all of the row first.
      uint32_t nt = 0;
      auto load_queries = [&](const Walk<kBlk>& t) {
        if (!warp_wait(q_empty(0), (nt & 1) ^ 1u)) return false;
        if constexpr (S::kQTmem) {
          tc_fence_after();                    // the last tile's products have read their terms
          const int row = at % kRP, pos0 = t.g * A.group_pos;
          const bool mine = row < min(A.group_pos, A.n_new - pos0) * A.G;
          const uint4* src = reinterpret_cast<const uint4*>(
              A.q + ((size_t)t.b * A.n_new + pos0 + (mine ? row / A.G : 0)) * A.q_stride +
              (size_t)(t.h * A.G + (mine ? row % A.G : 0)) * kD);
          uint32_t wv[kD / 2];
#pragma unroll
          for (int c = 0; c < kD / 8; ++c) {
            const uint4 v = mine ? __ldcg(src + c) : make_uint4(0u, 0u, 0u, 0u);
            wv[4 * c] = v.x;
            wv[4 * c + 1] = v.y;
            wv[4 * c + 2] = v.z;
            wv[4 * c + 3] = v.w;
          }
          uint32_t top = 0;                    // largest magnitude, as bf16 bits
#pragma unroll
          for (int k = 0; k < kD / 2; ++k)
            top = max(top, max(wv[k] & 0x7fffu, (wv[k] >> 16) & 0x7fffu));
          const bool fine = top < 0x7f80u;     // else the row holds no numbers: NaN
          // largest magnitude -> [2^7, 2^8)
          const int down = top > 0 && fine ? min(max((int)(top >> 7) - 134, -100), 120) : 0;
          const float mul = __uint_as_float((uint32_t)(127 - down) << 23);
#pragma unroll
          for (int c = 0; c < kD / 4; c += 8) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint32_t ph[2], pl[2];
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t u = wv[(c + k) * 2 + x];
                const float a = __uint_as_float(u << 16) * mul, b = __uint_as_float(u & 0xffff0000u) * mul;
                ph[x] = f32_to_e4m3x2(a, b);
                const uint32_t back = e4m3x2_to_f16x2((uint16_t)ph[x]);
                const float2 r2 = __half22float2(*reinterpret_cast<const __half2*>(&back));
                pl[x] = f32_to_e4m3x2(a - r2.x, b - r2.y);
              }
              hi[k] = ph[0] | (ph[1] << 16);
              lo[k] = pl[0] | (pl[1] << 16);
            }
            const uint32_t to = tmem + ((uint32_t)((warp & 3) * 32) << 16) + S::kColQ + c;
            tmem_store(to, hi, Cols<8>{});
            tmem_store(to + kD / 4, lo, Cols<8>{});
          }
          sts32(q_tab + at * 4, fine ? (uint32_t)(127 + down) << 23 : 0x7fffffffu);
          tmem_wait_store();
          tc_fence_before();
        } else {
          static_assert(S::kPanelBytes == 128, "256 dims");
          constexpr int kCh = kD / 8;                    // lanes per row, 8 dims each
          const int pos0 = t.g * A.group_pos;
          const int rows = min(A.group_pos, A.n_new - pos0) * A.G;
          for (int e = at; e < kRP * kCh; e += 32 * kAuxWarps) {
            const int r = e / kCh, c = e % kCh;
            uint4 val = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows)
              val = __ldcg(reinterpret_cast<const uint4*>(
                  A.q + ((size_t)t.b * A.n_new + pos0 + r / A.G) * A.q_stride +
                  (size_t)(t.h * A.G + r % A.G) * kD + c * 8));
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
            const int d0 = c * 8, p = d0 / 128, cc = (d0 % 128) / 16;
#pragma unroll
            for (int copy = 0; copy < S::kCopies; ++copy) {
              const int rr = copy * kRP + r;
              const uint32_t dst = qb + p * 128 * 128 + rr * 128 + ((cc ^ (rr & 7)) << 4) + (d0 & 8);
              sts64(dst, hi[0], hi[1]);
              sts64(dst + S::kQTerm, lo[0], lo[1]);
            }
            if (c == 0)
#pragma unroll
              for (int copy = 0; copy < S::kCopies; ++copy)
                sts32(q_tab + (copy * kRP + r) * 4, fine ? (uint32_t)(127 + down) << 23 : 0x7fffffffu);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full(0));
        ++nt;
        return true;
      };
      if (!w.done()) ok = load_queries(w);
      int s = 0;
      uint32_t ph = 0, n = 0;
      for (; ok && !w.done(); w.next(A)) {
        for (int i = 0; i < w.n_here; ++i, ++n) {
          const bool clean = w.clean(i);
          const int j0 = w.row(i);
          if (!(ok = warp_wait(v_full(s), ph))) break;
          if (!(ok = warp_wait(v16_empty(n & 1), ((n >> 1) & 1) ^ 1u))) break;
          // A warp takes 8 keys x 4 chunks of 16 codes at a time: rows p and
          // p ^ 5 side by side keep both the reads and the writes free of
          // bank conflicts under their swizzles.
          const uint32_t src = ring_v + s * S::kSlotBytes, dst = v16 + (n & 1) * S::kV16Bytes;
          const int pr = lane >> 3, row8 = (lane & 4) ? pr ^ 5 : pr;
          constexpr int kQuads = kD / 64, kPer = S::kPanelBytes / 16;
          constexpr int kSteps = kBlk / 8 * kQuads / kAuxWarps, kBatch = kSteps < 8 ? kSteps : 8;
#pragma unroll 1
          for (int e0 = warp - kSoftWarps; e0 < kBlk / 8 * kQuads; e0 += kAuxWarps * kBatch) {
            uint4 v[kBatch];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
              const int e = e0 + x * kAuxWarps, j = (e / kQuads) * 8 + row8, c = (e % kQuads) * 4 + (lane & 3);
              const int sw = S::kPanelBytes == 128 ? (j & 7) : ((j >> 1) & 3);
              v[x] = lds128(src + (c / kPer) * kBlk * S::kPanelBytes + j * S::kPanelBytes +
                            (((c % kPer) ^ sw) << 4));
            }
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
              const int e = e0 + x * kAuxWarps, j = (e / kQuads) * 8 + row8, c = (e % kQuads) * 4 + (lane & 3);
              const uint32_t wv[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
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
        if (!ok) break;
        Walk<kBlk> then = w;
        then.next(A);
        if (!then.done()) ok = load_queries(then);
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
          if (!w.clean(i)) {
            const int j0 = w.row(i);
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
    const int lg = warp * 32 + lane, row = lg % kRP, copy = warp * 32 / kRP;
    static_assert(kKpl >= 16 && kKpl <= 64, "a lane's scores of a block stay in registers");
    constexpr int kSubKeys = kKpl < 32 ? kKpl : 32, kSubs = kKpl / kSubKeys;   // runs with one scale
    constexpr int kRun = 16, kRuns = kExtra ? kKpl / kRun : 1;                 // runs with one bias start
    bool dead = false;                   // a wait ran out: keep to the barriers, compute nothing
    bool noted = false;
    uint32_t n = 0, nt = 0;
    bool s_ready = false;                // block n's scores were seen ready
    if constexpr (S::kCopies > 1) {
      const uint32_t zero[32] = {};
#pragma unroll
      for (int c = 0; c < S::kPBufs * (kBlk / 2); c += 32) tmem_store(tl + S::kColP + c, zero, Cols<32>{});
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
      sts32(place_tab + lg * 4, (uint32_t)(idx * A.Hq + w.h * A.G + gq));
      // Cap and bias: key k of a run adds kb[k], the run's start adds to all.
      const float slope = kExtra && A.slopes ? A.slopes[w.h * A.G + gq] * kLog2e : 0.f;
      const float cap_log2e = A.cap * kLog2e;
      float kb[kExtra ? kRun : 1];
      if constexpr (kExtra) {
#pragma unroll
        for (int k = 0; k < kRun; ++k) kb[k] = fmaf(slope, (float)k, cap_log2e);
      }
      const int key0 = copy * kKpl;                                // this copy's first key of a block
      const float* ks = nullptr;
      const float* vs = nullptr;
      float sk_next[kSubs], sv_next[kSubs];
      auto load_scales = [&](int j) {
        if constexpr (kE4m3) {
#pragma unroll
          for (int x = 0; x < kSubs; ++x) {
            const int jj = j + x * kSubKeys;
            sk_next[x] = jj < w.L ? __ldcg(ks + jj / SPECDEC_KV8_BLOCK) : 1.f;
            sv_next[x] = jj < w.L ? __ldcg(vs + jj / SPECDEC_KV8_BLOCK) : 1.f;
          }
        }
      };
      float ck = A.scale;
      if constexpr (kE4m3) {
        const size_t so = ((size_t)w.b * A.Hkv + w.h) * A.n_scale;
        ks = A.k_scale + so;
        vs = A.v_scale + so;
        load_scales(w.row(0) + key0);
        if (!dead && !warp_wait(q_full(0), nt & 1)) dead = true;
        ck *= __uint_as_float(lds32(q_tab + lg * 4));
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty(0));
      }
      if (!kExtra) ck *= kLog2e;

      // m_low: what a block's maximum has to pass for its reference to go down
      float m_ref = -INFINITY, m_peak = -INFINITY, m_low = INFINITY, l = 0.f;
      for (int ib = 0; ib < w.n_here; ++ib, ++n) {
        const int j0 = w.row(ib) + key0;
        const bool clean = w.clean(ib);
        float cs[kSubs], lv[kSubs], inv_sv[kSubs];                 // per run: score factor, log2 s_v, 1 / s_v
#pragma unroll
        for (int x = 0; x < kSubs; ++x) {
          cs[x] = ck;
          lv[x] = 0.f;
          inv_sv[x] = 1.f;
          if constexpr (kE4m3) {
            cs[x] = ck * sk_next[x];
            if (cs[x] < 1e-37f) cs[x] = 1e-37f;                    // -inf times it stays -inf (NaN stays too)
            lv[x] = __log2f(sv_next[x]);
            inv_sv[x] = rcp(sv_next[x]);
          }
        }
        if (kE4m3 && ib + 1 < w.n_here) load_scales(w.row(ib + 1) + key0);
        if (__builtin_expect(!__all_sync(0xffffffffu, s_ready), 0) && !dead &&
            !warp_wait(s_full(n & 1), (n >> 1) & 1))
          dead = true;
        if (dead) continue;
        tc_fence_after();
        union {
          uint32_t u[kKpl];
          float f[kKpl];
        } x;
        tmem_load(tl + S::kColS + (n & 1) * kBlk + key0, x.u);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty(n & 1));
        // ---- masks, cap and bias; the lane's largest exponent ----
        float top = -INFINITY, at[kRuns];
        if constexpr (kExtra) {
          if (A.cap > 0.f) {
#pragma unroll
            for (int k = 0; k < kKpl; ++k)
              x.f[k] = capped(x.f[k] * (cs[k / kSubKeys] * A.cap_exp), cap_log2e, kb[k % kRun]);
          } else {
#pragma unroll
            for (int k = 0; k < kKpl; k += 2) {
              const float c = cs[k / kSubKeys] * kLog2e;
              fma2(x.f[k], x.f[k + 1], c, c, kb[k % kRun], kb[k % kRun + 1]);
            }
          }
          // bias slope * (pos_j - pos_i), with rows at their index
#pragma unroll
          for (int run = 0; run < kRuns; ++run)
            at[run] = fmaf(slope, (float)(j0 + run * kRun - P0 - dep), lv[run * kRun / kSubKeys]);
        }
        if (__builtin_expect(!clean, 0)) {
          if (kExtra && A.tree && A.slopes) {
            // a tree's nodes stand at their depth instead
#pragma unroll
            for (int k = 0; k < kKpl; ++k) {
              const int jn = j0 + k - P0;
              if (jn >= 0 && jn < A.n_new)
                x.f[k] = fmaf(slope, (float)((int)lds32(tree + 128 * 16 + jn * 4) - jn), x.f[k]);
            }
          }
#pragma unroll
          for (int sub = 0; sub < kSubs; ++sub) {
            const uint32_t m = sight.mask(j0 + sub * kSubKeys);
#pragma unroll
            for (int k = 0; k < kSubKeys; ++k)
              x.f[sub * kSubKeys + k] = (m >> k) & 1u ? x.f[sub * kSubKeys + k] : -INFINITY;
          }
        }
        if constexpr (!kExtra) {
#pragma unroll
          for (int sub = 0; sub < kSubs; ++sub)
            top = fmaxf(top, fmaf(largest<kSubKeys>(x.f + sub * kSubKeys), cs[sub], lv[sub]));
        }
        if constexpr (kExtra) {
#pragma unroll
          for (int run = 0; run < kRuns; ++run) top = fmaxf(top, largest<kRun>(x.f + run * kRun) + at[run]);
        }
        // ---- the reference follows the maximum when it has to ----
        const bool up = mine && top > m_ref + kHeadroom, down = kE4m3 && top < m_ref - kBelow && top > m_low;
        if (__builtin_expect(__any_sync(0xffffffffu, up || down), 0)) {
          const float to = up ? top : kE4m3 && top < m_ref - kNear && top > m_low ? m_peak - kDeep : m_ref;
          const float alpha = to != m_ref ? ex2(m_ref - to) : 1.f;
          l *= alpha;
          m_ref = to;
          if constexpr (kE4m3) {
            m_peak = fmaxf(m_peak, to);
            m_low = to > m_peak - kDeep ? m_peak - kReach : INFINITY;
          }
          if (ib > 0) {
            if (!warp_wait(o_done((n - 1) & 1), ((n - 1) >> 1) & 1)) {
              dead = true;
              continue;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kD; c += 16) {
              uint32_t v[16];
              tmem_load(tl + S::kColO + c, v);
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
              tmem_store(tl + S::kColO + c, v, Cols<16>{});
            }
            tmem_wait_store();
          }
        }
        // ---- probabilities ----
        // f16 ones are kept 2^7 high: the headroom's 2^8 above that still fits,
        // and small weights stay normal numbers down to 2^-21.
        constexpr float kHigh = kE4m3 ? 7.f : 0.f;
        const float ref = m_ref == -INFINITY ? 0.f : m_ref, mu = ref - kHigh;
        // Exponents of 2^20 and more are rounded before the subtraction, as the
        // reference was: a fused one would bring out the reference's rounding.
        // The 2^7 come last: from 2^24 on, less than a step, they would be lost
        // or doubled in the reference, and 2^8 above it no f16 any more.
        float af[kSubs], bf[kRuns > kSubs ? kRuns : kSubs];    // exponent - reference = score * af + bf
#pragma unroll
        for (int sub = 0; sub < kSubs; ++sub) af[sub] = kExtra ? 1.f : cs[sub];
#pragma unroll
        for (int run = 0; run < (kExtra ? kRuns : kSubs); ++run) bf[run] = (kExtra ? at[run] : lv[run]) - mu;
        if (__builtin_expect(__any_sync(0xffffffffu, fabsf(mu) >= 1048576.f), 0)) {
#pragma unroll
          for (int k = 0; k < kKpl; k += 2) {
            const float b = kExtra ? at[k / kRun % kRuns] : lv[k / kSubKeys];
            fma2(x.f[k], x.f[k + 1], af[k / kSubKeys], af[k / kSubKeys], b, b);
            add2(x.f[k], x.f[k + 1], -ref, -ref);
          }
#pragma unroll
          for (int sub = 0; sub < kSubs; ++sub) af[sub] = 1.f;
#pragma unroll
          for (int run = 0; run < (kExtra ? kRuns : kSubs); ++run) bf[run] = kHigh;
        }
        uint32_t pk[kKpl / 2];
        bool p_free = n < S::kPBufs;         // the product that last read this P buffer is done
        // Tests ahead of waits, which cost 200 cycles even with nothing to wait for.
        s_ready = ib + 1 < w.n_here && mbar_test(s_full((n + 1) & 1), ((n + 1) >> 1) & 1);
        if (!p_free) p_free = mbar_test(o_done((n - S::kPBufs) & 1), ((n - S::kPBufs) >> 1) & 1);
#pragma unroll
        for (int xs = 0; xs < kSubs; ++xs) {
          float* const y = x.f + xs * kSubKeys;
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int k = 0; k < kSubKeys; k += 2) {
            if constexpr (kExtra) {
              const float b = bf[(xs * kSubKeys + k) / kRun % kRuns];
              add2(y[k], y[k + 1], b, b);
            } else {
              fma2(y[k], y[k + 1], af[xs], af[xs], bf[xs], bf[xs]);
            }
            const float p0 = ex2(y[k]), p1 = ex2(y[k + 1]);
            const uint32_t u = pack2<kE4m3>(p0, p1);
            pk[(xs * kSubKeys + k) / 2] = u;
            // The sum takes bf16 weights as rounded: their error then moves
            // the output by w (v - o) only. The f16 rounding is left out of it.
            if constexpr (kE4m3)
              add2(s0, s1, p0, p1);
            else
              add2(s0, s1, __uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
          }
          l = kE4m3 ? fmaf(s0 + s1, inv_sv[xs], l) : l + (s0 + s1);
        }
        if (__builtin_expect(!__all_sync(0xffffffffu, p_free), 0) &&
            !warp_wait(o_done((n - S::kPBufs) & 1), ((n - S::kPBufs) >> 1) & 1))
          dead = true;
        if (dead) continue;
        tc_fence_after();                    // the product has read what is overwritten now
        tmem_store(tl + S::kColP + (S::kPBufs == 2 ? (n & 1) * (kBlk / 2) : 0) + key0 / 2, pk, Cols<kKpl / 2>{});
        tmem_wait_store();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(n & 1));
      }

      // ---- the tile's output, or this part's share of it ----
      const bool whole = w.blk == 0 && w.n_here == w.nb;
      const size_t slot = (size_t)blockIdx.x * 2 + (w.u == part0 ? 0 : 1);
      float wgt = 1.f, lt = l, M = m_ref;
      if constexpr (S::kCopies > 1) {
        // merge the copies: weights from their references
        sts64(ml_tab + lg * 8, __float_as_uint(m_ref), __float_as_uint(l));
        named_bar_sync(1, 32 * kSoftWarps);
        M = -INFINITY;
        lt = 0.f;
#pragma unroll
        for (int c = 0; c < S::kCopies; ++c)
          M = fmaxf(M, __uint_as_float(lds32(ml_tab + (c * kRP + row) * 8)));
        const float Mu = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int c = 0; c < S::kCopies; ++c)
          lt += __uint_as_float(lds32(ml_tab + (c * kRP + row) * 8 + 4)) *
                ex2(__uint_as_float(lds32(ml_tab + (c * kRP + row) * 8)) - Mu);
        wgt = ex2(m_ref - Mu);
      }
      if (whole) wgt *= lt > 0.f ? 1.f / lt : (lt == 0.f ? 0.f : lt);     // NaN stays
      if (!whole && mine && !dead && copy == 0)
        *reinterpret_cast<float2*>(A.part_ml + (slot * kRP + row) * 2) = make_float2(M, lt);
      if (!dead && !warp_wait(o_done((n - 1) & 1), ((n - 1) >> 1) & 1)) dead = true;
      tc_fence_after();
      const bool has_odd = *odd != 0;
      // 32 columns at a time through shared memory, so that copies add up and
      // rows are written in whole lines: thread (r4, c4) writes 4 columns.
#pragma unroll 1
      for (int c0 = 0; c0 < kD; c0 += 32) {
        if (!dead) {
          uint32_t u[32];
          tmem_load(tl + S::kColO + c0, u);
          if (__builtin_expect(has_odd, 0)) {
            // Infinities and NaN that were held back from the product (rare),
            // for the rows that see them.
            for (int ib = 0; ib < w.n_here; ++ib) {
              if (w.clean(ib)) continue;
              const int jb = w.row(ib) + key0;
              for (int k = 0; k < kKpl && jb + k < w.L; ++k) {
                const bool seen = mine && (sight.mask(jb + k) & 1u);
                const size_t at = (((size_t)w.b * A.Lmax + jb + k) * A.Hkv + w.h) * kD + c0;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  uint32_t bits;
                  bool is_odd;
                  if constexpr (kE4m3) {
                    is_odd = (static_cast<const uint8_t*>(A.v)[at + c] & 0x7fu) == 0x7fu;
                    bits = 0x7fffffffu;
                  } else {
                    bits = (uint32_t)static_cast<const uint16_t*>(A.v)[at + c] << 16;
                    is_odd = (bits & 0x7f800000u) == 0x7f800000u;
                  }
                  if (seen && is_odd) u[c] = __float_as_uint(__uint_as_float(u[c]) + __uint_as_float(bits));
                }
              }
            }
          }
          const uint32_t to = stage + lg * kStagePitch;
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            sts128(to + k * 4, __float_as_uint(__uint_as_float(u[k]) * wgt),
                   __float_as_uint(__uint_as_float(u[k + 1]) * wgt),
                   __float_as_uint(__uint_as_float(u[k + 2]) * wgt),
                   __float_as_uint(__uint_as_float(u[k + 3]) * wgt));
        }
        if constexpr (S::kCopies > 1)
          named_bar_sync(1, 32 * kSoftWarps);
        else
          __syncwarp();
        const int c4 = (lane & 7) * 4;
        constexpr int kRowStep = S::kCopies > 1 ? 16 : 4;        // rows written at a time by who shares them
        const int r0 = (S::kCopies > 1 ? warp * 4 : warp * 32) + (lane >> 3);
        __nv_bfloat16* const out = A.out + (size_t)w.b * A.n_new * A.Hq * kD + c0 + c4;
        float* const part = A.part_o + slot * kRP * kD + c0 + c4;
        constexpr int kWrites = (S::kCopies > 1 ? kRP : 32) / kRowStep;
        float4 v[kWrites];
        uint32_t at[kWrites];
#pragma unroll
        for (int x = 0; x < kWrites; ++x) {
          v[x] = lds128f(stage + (r0 + x * kRowStep) * kStagePitch + c4 * 4);
          at[x] = lds32(place_tab + (r0 + x * kRowStep) * 4);
        }
#pragma unroll
        for (int c = 1; c < S::kCopies; ++c)
#pragma unroll
          for (int x = 0; x < kWrites; ++x) {
            const float4 y = lds128f(stage + (c * kRP + r0 + x * kRowStep) * kStagePitch + c4 * 4);
            add2(v[x].x, v[x].y, y.x, y.y);
            add2(v[x].z, v[x].w, y.z, y.w);
          }
        if (!dead && whole) {
#pragma unroll
          for (int x = 0; x < kWrites; ++x)
            if (r0 + x * kRowStep < rows_here)
              *reinterpret_cast<uint2*>(out + (size_t)at[x] * kD) =
                  make_uint2(pack2<false>(v[x].x, v[x].y), pack2<false>(v[x].z, v[x].w));
        } else if (!dead) {
#pragma unroll
          for (int x = 0; x < kWrites; ++x)
            if (r0 + x * kRowStep < rows_here) *reinterpret_cast<float4*>(part + (r0 + x * kRowStep) * kD) = v[x];
        }
        if constexpr (S::kCopies > 1)
          named_bar_sync(1, 32 * kSoftWarps);
        else
          __syncwarp();
      }
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
  if (warp == kIssuerO) tmem_dealloc(tmem, 512);
  if (*abort && lane == 0)
    // A wait gave up: let every copy already issued land before the CTA exits.
    for (int s = 0; s < kR; ++s) {
      if (issued & (1u << s))
        wait_drain(warp == kProducerV ? v_full(s) : k_full(s), (issued_phase >> s) & 1u);
      if (issued_q & (1u << s)) wait_drain(q_full(s), (issued_q_phase >> s) & 1u);
    }
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
  const long long most = tiles * ((A.Lmax + S::kBlk - 1) / S::kBlk + kTileCost);
  const int parts = cache_attn_parts(A, kCacheAttnCtas, most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts * A.head_lanes);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  CacheAttnLaunch L = A;
  L.note_tiles = note_tiles(A, parts);
  e = cudaLaunchKernelEx(&cfg, cache_attn_kernel<kE4m3, kD, kRP, kExtra>, L, tk, tv, tq);
  if (e != cudaSuccess) return e;
  return launch_combine<kD, kRP>(L, parts, cfg);
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
