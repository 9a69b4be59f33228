// Causal attention over packed prompts: sequences of different lengths end to
// end, grouped heads, with caps, windows and distance biases.
//
// For token i of a sequence and query head hq of KV head h:
//   o_i = sum_j softmax_j(s_ij) v_j over j <= i (and i - j < window),
//   s_ij = scale * q_i . k_j, capped, minus slope * (i - j)
// in one pass over the keys with the running maximum and sum in fp32.
//
// Bound: the tensor cores (4 D operations per visible pair and query head), and,
// as long beside them, the exponentials. Measured (32 query / 8 KV heads of 128,
// graph replays): one prompt of 8192 tokens 350 us, 1570 TFLOP/s, 0.82 of the
// measured bf16 rate; 24 ragged prompts of up to 2500 tokens 143 to 149 us (1080); 64
// dims, 8192 tokens 292 us (942); 256 dims (8 / 4 heads) 190 us (1440), 2 x 4001
// tokens of it with a window of 1024 and a cap 80 us (730). A block of 128 keys
// takes 2740 cycles for the two tiles: each one's products 1180 (16 MMAs of 64
// cycles, and the change between the two kinds), the hand-over of the turn 190,
// each one's softmax 1180 beside the other's products.
//
// Work. A row of the products is a (token, query head) pair of one KV head, so
// a tile of 128 rows is P = 128 / G tokens with their G heads: every head
// count fills the tile, K and V are read once for the group, and short or
// ragged prompts waste less than a tile of 128 tokens would. An item is two
// tiles (one for 256 dims) of a KV head and the blocks of keys they see. A
// first kernel lists a head's items with the longest first; CTAs, one per SM,
// take them off that list one by one, so that unequal prompts end together.
// (Without a list where a CTA has two items at most, and few sequences: each
// finds its own in the offsets.)
//
// CTA (up to 128 dims): warps 0-3 and 4-7 softmax of one tile each, then a
// warp that loads, one for each tile that issues its products, and one that
// looks through value blocks with keys that not every row sees.
//   S = Q K^T, M = 128, N = 128 keys, both operands in shared memory, into
//     the tile's 128 columns of tensor memory;
//   softmax: lane = row. The reference of the exponents moves only when a
//     row's maximum passes it by 2^8, so the output is rarely rescaled;
//   O += P V: P as bf16 over the same columns as S, V the MN-major operand.
// The products of one tile run while the other's softmax does. A tile's next
// scores are issued behind its P V, which the tensor core takes in order, so
// they overwrite P when it has been read, and their barrier also says that the
// output may be rescaled.
// 256 dims: the output takes 256 columns, so there is one tile, with two
// buffers of scores of 64 keys each: the products for one block run while the
// other's softmax does.
#include "cache_attention.cuh"

namespace specdec {
namespace cache_attn {

// 128 columns of this warp's lanes, with the values there.
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&x)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
      "}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63"
      "}, [%129];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
      "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95"
      "}, [%130];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
      "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127"
      "}, [%131];\n\t"
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
        "=r"(x[60]), "=r"(x[61]), "=r"(x[62]), "=r"(x[63]), "=r"(x[64]), "=r"(x[65]),
        "=r"(x[66]), "=r"(x[67]), "=r"(x[68]), "=r"(x[69]), "=r"(x[70]), "=r"(x[71]),
        "=r"(x[72]), "=r"(x[73]), "=r"(x[74]), "=r"(x[75]), "=r"(x[76]), "=r"(x[77]),
        "=r"(x[78]), "=r"(x[79]), "=r"(x[80]), "=r"(x[81]), "=r"(x[82]), "=r"(x[83]),
        "=r"(x[84]), "=r"(x[85]), "=r"(x[86]), "=r"(x[87]), "=r"(x[88]), "=r"(x[89]),
        "=r"(x[90]), "=r"(x[91]), "=r"(x[92]), "=r"(x[93]), "=r"(x[94]), "=r"(x[95]),
        "=r"(x[96]), "=r"(x[97]), "=r"(x[98]), "=r"(x[99]), "=r"(x[100]), "=r"(x[101]),
        "=r"(x[102]), "=r"(x[103]), "=r"(x[104]), "=r"(x[105]), "=r"(x[106]), "=r"(x[107]),
        "=r"(x[108]), "=r"(x[109]), "=r"(x[110]), "=r"(x[111]), "=r"(x[112]), "=r"(x[113]),
        "=r"(x[114]), "=r"(x[115]), "=r"(x[116]), "=r"(x[117]), "=r"(x[118]), "=r"(x[119]),
        "=r"(x[120]), "=r"(x[121]), "=r"(x[122]), "=r"(x[123]), "=r"(x[124]), "=r"(x[125]),
        "=r"(x[126]), "=r"(x[127])
      : "r"(taddr), "r"(taddr + 32), "r"(taddr + 64), "r"(taddr + 96)
      : "memory");
}

constexpr int kPlanThreads = 1024, kPlanBuckets = 1024;
constexpr int kSoftRegs = 208, kRoleRegs = 88;      // registers a thread, of 168 at launch (two tiles: 384 threads)
constexpr int kRoleWarps = 4;                       // behind the softmax warps: loads, issue, values

template <int kD>
struct PromptShape {
  static constexpr int kTiles = prompt_tiles(kD);               // of an item, a softmax warpgroup each
  static constexpr int kBlk = prompt_block(kD);                 // keys per block
  static constexpr int kHalves = kTiles == 2 ? 1 : 2;           // warps that share a row's keys of a block
  static constexpr int kSoft = 4 * kHalves * kTiles;            // softmax warps
  static constexpr int kThreads = 32 * (kSoft + kRoleWarps);
  static constexpr int kPanels = kD / 64;                       // 128-byte runs of a row
  static constexpr int kSlotBytes = kBlk * kD * 2;              // a block of K, or of V
  static constexpr int kQTile = 128 * kD * 2;
  static constexpr int kKeys = kBlk / kHalves;                  // of a block, to a softmax thread
  static constexpr int kStage = 32 * 128;                       // a softmax warp's rows, 64 columns of the output
  static constexpr int kFixed = 1024 + kTiles * kQTile + kSoft * kStage + 1024;
  static constexpr int kRingMax = (kSmemLimit - kFixed) / kSlotBytes;
  static constexpr int kRing = kRingMax < 8 ? kRingMax : 8;     // blocks (K and V alike) in flight
  static constexpr int kSmem = kFixed + kRing * kSlotBytes;
  static_assert(kRing >= 4, "two blocks of each");
  static constexpr int kColS = 0, kColO = 2 * kBlk;             // two buffers of scores, then the outputs
  static_assert(kColO + kTiles * kD <= 512, "tensor memory");
};

__device__ __forceinline__ float min_or_nan(float a, float b) {
  float m;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
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

// capped() of two scores with one reciprocal, which takes as long as two
// exponentials: 1 / a = b / (a b). The bound keeps the product finite; behind it
// the tanh is 1 to 2^-59. A NaN in either is one in both, so both have to be
// scores that the row sees, or numbers.
__device__ __forceinline__ void capped2(float& x, float& y, float cap_exp, float cap_log2e, float plus_x, float plus_y) {
  const float a = 1.f + ex2(min_or_nan(x * cap_exp, 60.f)), b = 1.f + ex2(min_or_nan(y * cap_exp, 60.f));
  const float r = rcp(a * b) * (-2.f * cap_log2e);
  x = fmaf(r, b, plus_x);
  y = fmaf(r, a, plus_y);
}

// An item as its roles see it.
template <int kD>
struct Item {
  using S = PromptShape<kD>;
  static constexpr int kLast = S::kTiles - 1;
  int h, t0, L, row0;                // KV head, first token, the sequence's length and first row
  int lo[S::kTiles], hi[S::kTiles];  // each tile's blocks of keys
  int first, last;                   // all blocks: first .. last - 1
  int clean_lo, clean_hi;            // those that every row sees whole

  __device__ __forceinline__ void set(const PromptLaunch& A, int4 it, int head) {
    constexpr int kBlk = S::kBlk;
    row0 = it.x;
    t0 = it.y;
    L = it.z;
    h = head;
    last = 0;
#pragma unroll
    for (int u = 0; u < S::kTiles; ++u) {
      const int ta = t0 + u * A.tile_tokens, tl = min(ta + A.tile_tokens, L) - 1;
      lo[u] = A.window > 0 ? max(0, ta - A.window + 1) / kBlk : 0;
      hi[u] = ta < L ? tl / kBlk + 1 : lo[u];
      if (ta < L) last = hi[u];
    }
    first = lo[0];
    const int t_end = min(t0 + S::kTiles * A.tile_tokens, L) - 1;
    clean_hi = (t0 + 1) / kBlk;
    clean_lo = A.window > 0 ? (max(0, t_end - A.window + 1) + kBlk - 1) / kBlk : 0;
  }
  // (selected, not indexed: a tile's number may be known at run time only)
  __device__ __forceinline__ int begin(int u) const { return kLast && u ? lo[kLast] : lo[0]; }
  __device__ __forceinline__ int end(int u) const { return kLast && u ? hi[kLast] : hi[0]; }
  __device__ __forceinline__ bool tile(int u) const { return end(u) > begin(u); }
  __device__ __forceinline__ bool on(int u, int i) const { return i >= begin(u) && i < end(u); }
  __device__ __forceinline__ bool clean(int i) const { return i >= clean_lo && i < clean_hi; }
};

// The rows of a sequence, (first, length); a length of -1 where the offsets do
// not fit. Each is read once where it is used: what was looked at is what counts,
// should they change during the call.
__device__ __forceinline__ int2 rows_between(const PromptLaunch& A, int lo, int hi) {
  return lo < 0 || hi < lo || hi > A.T ? make_int2(0, -1) : make_int2(lo, hi - lo);
}
__device__ __forceinline__ int2 rows_of(const PromptLaunch& A, int b) {
  const volatile int32_t* const cu = A.cu_seqlens + b;
  const int lo = cu[0], hi = cu[1];
  return rows_between(A, lo, hi);
}
// The same through L1, for the lister, which comes back to them: 1.5 us less.
__device__ __forceinline__ int2 rows_again(const PromptLaunch& A, int b) {
  int lo, hi;
  asm volatile("ld.global.b32 %0, [%2];\n\tld.global.b32 %1, [%2 + 4];" : "=&r"(lo), "=r"(hi) : "l"(A.cu_seqlens + b));
  return rows_between(A, lo, hi);
}

// The list of a head's items, longest first (equals in any order: no item's
// outcome depends on another's), and the status word.
template <int kD>
__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const __grid_constant__ PromptLaunch A, int ctas) {
  using S = PromptShape<kD>;
  __shared__ int place[kPlanBuckets], warp_sum[32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_launch_dependents();
  place[tid] = 0;
  grid_dependency_wait();
  bool broken = false;
  for (int b = tid; b < A.B; b += kPlanThreads) broken |= rows_again(A, b).y < 0;
  broken = __syncthreads_or(broken);
  const int span = S::kTiles * A.tile_tokens;
  auto each = [&](auto&& take) {
    for (int b = warp; b < A.B; b += kPlanThreads / 32) {
      const int2 rows = rows_again(A, b);
      const int row0 = rows.x, L = rows.y;
      for (int t0 = lane * span; t0 < L; t0 += 32 * span) {
        const int t_end = min(t0 + span, L) - 1;
        const int low = A.window > 0 ? max(0, t0 - A.window + 1) / S::kBlk : 0;
        const int blocks = t_end / S::kBlk + 1 - low;
        take(kPlanBuckets - 1 - min(blocks >> A.cost_shift, kPlanBuckets - 1), make_int4(row0, t0, L, 0));
      }
    }
  };
  if (!broken) each([&](int bucket, int4) { atomicAdd(place + bucket, 1); });
  __syncthreads();
  const int mine = place[tid];
  int run = mine;
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
  run += warp ? warp_sum[warp - 1] : 0;
  place[tid] = run - mine;
  if (tid == kPlanThreads - 1) {
    *A.n_items = (int)(run < A.max_items ? run : A.max_items);
    *A.next = ctas;                  // every CTA begins with the item of its own number
    *A.status = broken ? SPECDEC_ERR_INVALID_ARG : SPECDEC_OK;
  }
  __syncthreads();
  // (within the list, should the offsets have changed since they were counted;
  // entries that are not written then are looked at where they are taken)
  if (!broken)
    each([&](int bucket, int4 it) {
      const int at = atomicAdd(place + bucket, 1);
      if (at < A.max_items) A.items[at] = it;
    });
}

template <int kD, bool kExtra>
__global__ void __launch_bounds__(PromptShape<kD>::kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ PromptLaunch A, const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v) {
  using S = PromptShape<kD>;
  constexpr int kBlk = S::kBlk, kKeys = S::kKeys, kR = S::kRing, kTiles = S::kTiles, kHalves = S::kHalves,
                kSoft = S::kSoft;
  constexpr int kLoad = kSoft, kIssue = kSoft + 1, kCheck = kIssue + kTiles;     // warp indices
  constexpr int kCheckWarps = kRoleWarps - 1 - kTiles;
  constexpr uint32_t kReaders = kSoft + kTiles + kCheckWarps;   // warps that are told of an item
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t qb = (raw + 1023u) & ~1023u;
  const uint32_t ring = qb + kTiles * S::kQTile;
  const uint32_t stage = ring + kR * S::kSlotBytes;
  const uint32_t bars = stage + kSoft * S::kStage;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  auto full = [&](int s) { return bar(s); };
  auto empty = [&](int s) { return bar(kR + s); };
  auto v_clean = [&](int s) { return bar(2 * kR + s); };
  auto q_full = [&](int u) { return bar(3 * kR + u); };
  auto q_empty = [&](int u) { return bar(3 * kR + 2 + u); };
  auto s_full = [&](int u) { return bar(3 * kR + 4 + u); };
  auto p_full = [&](int u) { return bar(3 * kR + 6 + u); };
  auto o_done = [&](int u) { return bar(3 * kR + 8 + u); };
  auto told = [&](int e) { return bar(3 * kR + 10 + e); };
  auto heard = [&](int e) { return bar(3 * kR + 12 + e); };
  const uint32_t drained = bar(3 * kR + 14);
  auto turn = [&](int u) { return bar(3 * kR + 15 + u); };
  const uint32_t board = bar(3 * kR + 18) & ~15u;               // [2] (row0, t0, L, KV head or -1)
  const uint32_t rows_tab = board + 64;                         // [128] what a row's halves tell each other
  uint8_t* const words = smem_raw + (board + 32 - raw);
  volatile int* const abort = reinterpret_cast<volatile int*>(words);
  volatile int* const odd = abort + 1;                          // a value that is no number was held back
  volatile uint32_t* const tmem_slot = reinterpret_cast<volatile uint32_t*>(words) + 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kR; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kTiles + kCheckWarps);
      mbar_init(v_clean(s), kCheckWarps);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(q_full(u), 1);
      mbar_init(q_empty(u), 1);
      mbar_init(s_full(u), 1);
      mbar_init(p_full(u), 4 * kHalves);
      mbar_init(o_done(u), 1);
      mbar_init(turn(u), 1);
      mbar_init(told(u), 1);
      mbar_init(heard(u), kReaders);
    }
    mbar_init(drained, kTiles);
    *abort = 0;
    *odd = 0;
    fence_mbar_init();
  }
  if (warp == kIssue) tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
  grid_dependency_wait();
  grid_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto warp_wait = [&](uint32_t b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait<true>(b, parity, abort, A.status));
  };
  // The next item, as the loading warp put it on the board; false behind the last.
  uint32_t n_told = 0;
  bool ok = true;
  auto hear = [&](Item<kD>& w) {
    const int e = n_told & 1;
    if (!(ok = warp_wait(told(e), (n_told >> 1) & 1))) return false;
    const uint4 it = lds128(board + 16 * e);
    __syncwarp();
    if (lane == 0) mbar_arrive(heard(e));
    ++n_told;
    if ((int)it.w < 0) return false;
    w.set(A, make_int4((int)it.x, (int)it.y, (int)it.z, 0), (int)it.w);
    return true;
  };
  uint32_t issued = 0, issued_phase = 0, issued_q = 0, issued_q_phase = 0;   // copies in flight
  // Ring order: the order in which the issuer takes blocks.
  // Two tiles: K0 V0 K1 V1 ..; one: K0 K1 V0 K2 V1 .. (scores a block ahead).

  if (warp >= kSoft) {
    if constexpr (kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
    if (warp == kLoad) {
      // ----------------------------------------------------------- loads --
      // The items come from the list, or, where there is none, from the
      // offsets themselves, in their order: a warp's running count of items.
      const int span = kTiles * A.tile_tokens;
      auto count_items = [&](int2 rows) { return (max(rows.y, 0) + span - 1) / span; };
      auto find_item = [&](int item) {
        for (int b0 = 0, before = 0; b0 < A.B; b0 += 32) {
          const int2 rows = b0 + lane < A.B ? rows_of(A, b0 + lane) : make_int2(0, 0);
          const int mine = count_items(rows);
          int run = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += x;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, item < before + run);
          if (hit) {
            const int l = __ffs(hit) - 1, t = item - before - __shfl_sync(0xffffffffu, run - mine, l);
            return make_int4(__shfl_sync(0xffffffffu, rows.x, l), t * span, __shfl_sync(0xffffffffu, rows.y, l), 0);
          }
          before += __shfl_sync(0xffffffffu, run, 31);
        }
        return make_int4(0, 0, 0, 0);          // the offsets have changed since they were counted
      };
      // Rows of the batch and a token among them: not so only where the offsets
      // have changed since the items were counted. Such an item is nobody's.
      auto lies = [&](int4 it) {
        return it.x >= 0 && it.x <= A.T && it.z <= A.T - it.x && it.y >= 0 && it.y < it.z;
      };
      int total;                                                 // < 2^31 (host)
      if (A.items) {
        total = *reinterpret_cast<const volatile int*>(A.n_items) * A.Hkv;
      } else {
        bool broken = false;
        int n_items = 0;
        for (int b = lane; b < A.B; b += 32) {
          const int2 rows = rows_of(A, b);
          broken |= rows.y < 0;
          n_items += count_items(rows);
        }
        broken = __any_sync(0xffffffffu, broken);
#pragma unroll
        for (int o = 16; o; o >>= 1) n_items += __shfl_xor_sync(0xffffffffu, n_items, o);
        total = broken ? 0 : (int)(n_items < A.max_items ? n_items : A.max_items) * A.Hkv;
        if (blockIdx.x == 0 && lane == 0) *A.status = broken ? SPECDEC_ERR_INVALID_ARG : SPECDEC_OK;
      }
      int s = 0;
      uint32_t ph = 0, nq[2] = {0, 0};
      int next = blockIdx.x;
      auto load = [&](const Item<kD>& w, bool is_v, int i) {
        if (!(ok = warp_wait(empty(s), ph ^ 1u))) return;
        if (elect_one()) {
          mbar_arrive_expect_tx(full(s), (uint32_t)S::kSlotBytes);
#pragma unroll
          for (int p = 0; p < S::kPanels; ++p)
            tma_load_3d(ring + s * S::kSlotBytes + p * kBlk * 128, is_v ? &tmap_v : &tmap_k, full(s), p * 64, w.h,
                        w.row0 + i * kBlk, policy_evict_normal());
        }
        __syncwarp();
        issued |= 1u << s;
        issued_phase = (issued_phase & ~(1u << s)) | (ph << s);
        if (++s == kR) {
          s = 0;
          ph ^= 1u;
        }
      };
      while (ok) {
        const int e = n_told & 1;
        if (!(ok = warp_wait(heard(e), ((n_told >> 1) & 1) ^ 1u))) break;
        int4 it = make_int4(0, 0, 0, -1);
        while (next < total) {
          it = A.items ? __ldcg(A.items + next / A.Hkv) : find_item(next / A.Hkv);
          it.w = next % A.Hkv;
          if (__builtin_expect(lies(it), 1)) break;
          it.w = -1;
          if (lane == 0) next = A.items ? atomicAdd(A.next, 1) : next + (int)gridDim.x;
          next = __shfl_sync(0xffffffffu, next, 0);
        }
        if (lane == 0) {
          sts128(board + 16 * e, it.x, it.y, it.z, it.w);
          mbar_arrive(told(e));
        }
        __syncwarp();
        ++n_told;
        if (it.w < 0) break;
        if (lane == 0) next = A.items ? atomicAdd(A.next, 1) : next + (int)gridDim.x;      // looked at an item later
        Item<kD> w;
        w.set(A, it, it.w);
        load(w, false, w.first);
#pragma unroll
        for (int u = 0; u < kTiles; ++u) {
          if (!ok || !w.tile(u)) continue;
          if (!(ok = warp_wait(q_empty(u), (nq[u] & 1) ^ 1u))) continue;
          if (elect_one()) {
            mbar_arrive_expect_tx(q_full(u), (uint32_t)(A.tile_tokens * A.G) * 128u * S::kPanels);
#pragma unroll
            for (int p = 0; p < S::kPanels; ++p)
              tma_load_3d(qb + u * S::kQTile + p * 128 * 128, &tmap_q, q_full(u), p * 64, w.h * A.G,
                          w.row0 + w.t0 + u * A.tile_tokens, policy_evict_normal());
          }
          __syncwarp();
          issued_q |= 1u << u;
          issued_q_phase = (issued_q_phase & ~(1u << u)) | ((nq[u] & 1) << u);
          ++nq[u];
        }
        for (int i = w.first; ok && i < w.last; ++i) {
          if (kTiles == 1 && i + 1 < w.last) load(w, false, i + 1);
          if (ok) load(w, true, i);
          if (ok && kTiles == 2 && i + 1 < w.last) load(w, false, i + 1);
        }
        next = __shfl_sync(0xffffffffu, next, 0);
      }
    } else if (warp < kCheck) {
      // ----------------------------------------------------------- issue --
      // A thread to a tile: behind MMAs that wait for their place, even a wait
      // with nothing to wait for takes 200 cycles, which the other's fill. So
      // all that a block's products need is waited for ahead of them. The two
      // take turns, a P V and the next Q K^T each: side by side, both tiles'
      // products would end late, and their softmax leave the tensor core idle.
      constexpr uint32_t id_qk = instr_desc(1, false, kBlk), id_pv = instr_desc(1, true, kD);
      if (elect_one()) {
        const int u = warp - kIssue;
        const uint64_t q_desc = operand_desc<128>(qb + u * S::kQTile, 16), k_desc = operand_desc<128>(ring, 16);
        const uint64_t v_desc = operand_desc<128>(ring, kBlk * 128);
        const uint32_t acc = tmem + S::kColO + u * kD;
        int s = 0;
        uint32_t ph = 0, nq = 0, clean_ph = 0, n = 0, n_turn = 0;
        Item<kD> w;
        auto wait = [&](uint32_t b, uint32_t parity) { return ok = mbar_wait<true>(b, parity, abort, A.status); };
        auto my_turn = [&]() {                   // the second tile's begins with the first one's end
          return wait(turn(u), (n_turn++ & 1) ^ (u == 0 ? 1u : 0u));
        };
        auto pass_turn = [&]() { mbar_arrive(turn(u ^ 1)); };
        auto release = [&](bool used) {          // once what was issued so far is done
          if (used)
            tc_commit(empty(s));
          else
            mbar_arrive(empty(s));
          if (++s == kR) {
            s = 0;
            ph ^= 1u;
          }
        };
        auto scores = [&](int buf, bool last) {  // against the ring's block
          const uint64_t kd = k_desc + (uint64_t)((uint32_t)(s * S::kSlotBytes) >> 4);
#pragma unroll
          for (int p = 0; p < S::kPanels; ++p)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss<false>(tmem + S::kColS + buf * kBlk, q_desc + (uint64_t)((p * 128 * 128 + k * 32) >> 4),
                            kd + (uint64_t)((p * kBlk * 128 + k * 32) >> 4), id_qk, p + k > 0);
          tc_commit(s_full(buf));
          if (last) tc_commit(q_empty(u));
        };
        auto values = [&](int buf, bool more, bool last) {     // more: adds to what is there
          const uint64_t vd = v_desc + (uint64_t)((uint32_t)(s * S::kSlotBytes) >> 4);
#pragma unroll
          for (int k = 0; k < kBlk / 16; ++k)
            mma_ts<false>(acc, tmem + S::kColS + buf * kBlk + k * 8, vd + (uint64_t)(k * 2048 >> 4), id_pv,
                          more || k > 0);
          if (last) tc_commit(o_done(kTiles == 2 ? u : buf));
        };
        // V of block i is in the ring's slot.
        auto arrived_v = [&](int i) {
          if (!wait(full(s), ph)) return false;
          if (!w.clean(i)) {
            if (!wait(v_clean(s), (clean_ph >> s) & 1)) return false;
            clean_ph ^= 1u << s;
          }
          return true;
        };
        while (ok && wait(told(n_told & 1), (n_told >> 1) & 1)) {
          const uint4 it = lds128(board + 16 * (n_told & 1));
          mbar_arrive(heard(n_told++ & 1));
          if ((int)it.w < 0) break;
          w.set(A, make_int4((int)it.x, (int)it.y, (int)it.z, 0), (int)it.w);
          if (w.tile(u) && !wait(q_full(u), nq++ & 1)) break;
          if (!wait(full(s), ph)) break;
          if constexpr (kTiles == 2) {
            if (!my_turn()) break;
            tc_fence_after();
            const bool begins = w.on(u, w.first);
            if (begins) scores(u, w.first + 1 == w.end(u));
            pass_turn();
            release(begins);
            for (int i = w.first; i < w.last; ++i) {
              const bool here = w.on(u, i), then = i + 1 < w.last, more = then && w.on(u, i + 1);
              if (!arrived_v(i)) break;
              if (then && !wait(full(s + 1 == kR ? 0 : s + 1), s + 1 == kR ? ph ^ 1u : ph)) break;
              if (here && !wait(p_full(u), n++ & 1)) break;
              if (!my_turn()) break;
              tc_fence_after();
              if (here) values(u, i > w.begin(u), i + 1 == w.end(u));
              release(here);
              if (more) scores(u, i + 2 == w.end(u));
              pass_turn();
              if (then) release(more);
            }
          } else {
            // scores a block ahead, in buffers taken in turn
            tc_fence_after();
            scores(n & 1, w.first + 1 == w.last);
            release(true);
            for (int i = w.first; i < w.last; ++i, ++n) {
              if (i + 1 < w.last) {
                if (!wait(full(s), ph)) break;
                tc_fence_after();
                // (its buffer's P was read by the product issued last)
                scores((n + 1) & 1, i + 2 == w.last);
                release(true);
              }
              if (!arrived_v(i)) break;
              if (!wait(p_full(n & 1), (n >> 1) & 1)) break;
              tc_fence_after();
              values(n & 1, i > w.first, true);
              release(true);
            }
          }
        }
        // every product has to be done before the tensor memory is given back
        tc_commit(drained);
        wait_drain(drained, 0);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- values --
      // Blocks with keys that not every row sees: an infinity or a NaN there
      // would pass a zero probability, so it stays out of the product, and the
      // epilogue adds it where it is seen. Every block is waited for and
      // released, so that this loop and the ring never part by more than its length.
      const int at = threadIdx.x - 32 * kCheck;
      int s = 0;
      uint32_t ph = 0;
      Item<kD> w;
      auto pass = [&](bool look) {
        if (!(ok = warp_wait(full(s), ph))) return;
        if (look) {
          // 16 bytes of each of kBatch runs at a time: an exponent of ones
          // carries into the sign's place
          constexpr int kBatch = 8, kStep = 32 * kCheckWarps * 16;
          static_assert(S::kSlotBytes % (kStep * kBatch) == 0, "whole batches");
#pragma unroll 1
          for (uint32_t a0 = ring + s * S::kSlotBytes + at * 16, end = a0 + S::kSlotBytes; a0 < end;
               a0 += kStep * kBatch) {
            uint4 v[kBatch];
#pragma unroll
            for (int y = 0; y < kBatch; ++y) v[y] = lds128(a0 + y * kStep);
            uint32_t any = 0;
#pragma unroll
            for (int y = 0; y < kBatch; ++y)
              any |= ((v[y].x & 0x7fff7fffu) + 0x00800080u) | ((v[y].y & 0x7fff7fffu) + 0x00800080u) |
                     ((v[y].z & 0x7fff7fffu) + 0x00800080u) | ((v[y].w & 0x7fff7fffu) + 0x00800080u);
            if (__builtin_expect((any & 0x80008000u) != 0, 0)) {
#pragma unroll 1
              for (int y = 0; y < kBatch; ++y) {
                const uint4 z = lds128(a0 + y * kStep);
                uint32_t x[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if ((x[k] & 0x7f80u) == 0x7f80u) x[k] &= 0xffff0000u;
                  if ((x[k] & 0x7f800000u) == 0x7f800000u) x[k] &= 0x0000ffffu;
                }
                sts128(a0 + y * kStep, x[0], x[1], x[2], x[3]);
              }
              *odd = 1;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(v_clean(s));
        }
        if (lane == 0) mbar_arrive(empty(s));
        if (++s == kR) {
          s = 0;
          ph ^= 1u;
        }
      };
      while (ok && hear(w)) {
        pass(false);
        for (int i = w.first; ok && i < w.last; ++i) {
          if (kTiles == 1 && i + 1 < w.last) pass(false);
          if (ok) pass(!w.clean(i));
          if (ok && kTiles == 2 && i + 1 < w.last) pass(false);
        }
      }
    }
  } else {
    // --------------------------------------------------------------- softmax --
    if constexpr (kTiles == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int u = warp / (4 * kHalves), half = (warp >> 2) % kHalves, row = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);      // this warp's lanes
    const int tok_of_row = row / A.G, gq = row % A.G;
    // Two warps of the same rows meet at a barrier of their own once for every
    // item and block, whatever became of their waits, and so go on, or give up,
    // together.
    const int pair_bar = 1 + (warp & 3);
    auto any_of_row = [&](bool x) {
      return kHalves == 1 ? __any_sync(0xffffffffu, x) != 0 : bar_count(pair_bar, 32 * kHalves, x) > 0;
    };
    // A row's value from both halves.
    auto joined = [&](float x, auto join) {
      if (kHalves == 1) return x;
      const uint32_t at = rows_tab + row * 4;
      if (half == 1) sts32(at, __float_as_uint(x));
      named_bar_sync(pair_bar, 32 * kHalves);
      if (half == 0) {
        x = join(x, __uint_as_float(lds32(at)));
        sts32(at, __float_as_uint(x));
      }
      named_bar_sync(pair_bar, 32 * kHalves);
      return half == 0 ? x : __uint_as_float(lds32(at));
    };
    uint32_t n = 0, n_items = 0;       // this tile's blocks and items
    Item<kD> w;
    for (;;) {
      const bool more = ok && hear(w);
      if (kHalves > 1 && any_of_row(!ok)) ok = false;
      if (!ok || !more) break;
      if (!w.tile(u)) continue;
      const int ta = w.t0 + u * A.tile_tokens, tok = ta + tok_of_row;
      const bool mine = tok_of_row < A.tile_tokens && tok < w.L;
      const float slope = kExtra && A.slopes && tok_of_row < A.tile_tokens ? A.slopes[w.h * A.G + gq] * kLog2e : 0.f;
      float m_ref = -INFINITY, l = 0.f;
      for (int i = w.begin(u); i < w.end(u); ++i, ++n) {
        const int buf = kTiles == 2 ? u : (int)(n & 1);
        const int j0 = i * kBlk + half * kKeys;
        ok = warp_wait(s_full(buf), kTiles == 2 ? n & 1 : (n >> 1) & 1);
        if (kHalves == 1 && !ok) break;
        tc_fence_after();
        union {
          uint32_t u[kKeys];
          float f[kKeys];
        } x;
        tmem_load(tl + S::kColS + buf * kBlk + half * kKeys, x.u);
        // Keys that the thread's row does not see, in a block that has some.
        const bool masked = __builtin_expect(!w.clean(i), 0);
        auto unseen = [&](float score) {
          const int hi = tok - j0, lo = A.window > 0 ? hi - A.window + 1 : 0;     // it sees lo .. hi of its own
#pragma unroll
          for (int k0 = 0; k0 < kKeys; k0 += 32) {
            const int a = lo - k0, b = hi - k0;
            uint32_t m = b < 0 ? 0u : b >= 31 ? 0xffffffffu : (2u << b) - 1u;
            if (a > 0) m &= a >= 32 ? 0u : 0xffffffffu << a;
#pragma unroll
            for (int k = 0; k < 32; ++k) x.f[k0 + k] = (m >> k) & 1u ? x.f[k0 + k] : score;
          }
        };
        float c = A.scale * kLog2e, top = -INFINITY;
        if constexpr (kExtra) {
          // cap and bias: the scores become exponents
          const float b0 = slope * (float)(j0 - tok);
          if (A.cap > 0.f) {
            const float cl = A.cap * kLog2e, ce = A.scale * A.cap_exp;
            if (masked) unseen(0.f);             // a NaN there would reach the key that shares its reciprocal
#pragma unroll
            for (int k = 0; k < kKeys; k += 2)
              capped2(x.f[k], x.f[k + 1], ce, cl, cl + fmaf(slope, (float)k, b0), cl + fmaf(slope, (float)(k + 1), b0));
          } else {
#pragma unroll
            for (int k = 0; k < kKeys; ++k) x.f[k] = fmaf(x.f[k], c, fmaf(slope, (float)k, b0));
          }
          c = 1.f;
        }
        if (masked) unseen(-INFINITY);
#pragma unroll
        for (int k = 0; k < kKeys; k += 32) top = fmaxf(top, largest<32>(x.f + k));
        top *= c;
        // ---- the reference follows the maximum when it has to ----
        // (Behind the barrier both halves have their scores, which P overwrites.)
        if (kHalves > 1) tc_fence_before();
        const bool rare = any_of_row((kHalves > 1 && !ok) || (mine && top > m_ref + kHeadroom));
        if (kHalves > 1) tc_fence_after();
        if (__builtin_expect(rare, 0)) {
          if (kHalves > 1 && any_of_row(!ok)) ok = false;
          if (!ok) break;
          top = joined(top, [](float a, float b) { return fmaxf(a, b); });
          const bool up = mine && top > m_ref + kHeadroom;
          const float alpha = up ? ex2(m_ref - top) : 1.f;
          if (up) m_ref = top;
          l *= alpha;
          if (i > w.begin(u)) {
            // the products so far are done: with two tiles these scores came behind them
            if (kTiles == 1) ok = warp_wait(o_done((n - 1) & 1), ((n - 1) >> 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int c0 = half * (kD / kHalves); c0 < (half + 1) * (kD / kHalves); c0 += 16) {
              uint32_t v[16];
              tmem_load(tl + S::kColO + u * kD + c0, v);
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
              tmem_store(tl + S::kColO + u * kD + c0, v, Cols<16>{});
            }
            tmem_wait_store();
          }
        }
        // ---- probabilities ----
        const float ref = m_ref == -INFINITY ? 0.f : m_ref;
        float sub = -ref;
        if (__builtin_expect(__any_sync(0xffffffffu, fabsf(ref) >= 1048576.f), 0)) {
          // Exponents of 2^20 and more are rounded before the subtraction, as the
          // reference was: a fused one would bring out the reference's rounding.
#pragma unroll
          for (int k = 0; k < kKeys; ++k) x.f[k] = __fadd_rn(__fmul_rn(x.f[k], c), sub);
          c = 1.f;
          sub = 0.f;
        }
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int k0 = 0; k0 < kKeys; k0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float y0 = x.f[k0 + k], y1 = x.f[k0 + k + 1];
            fma2(y0, y1, c, c, sub, sub);
            y0 = ex2(y0);
            y1 = ex2(y1);
            pk[k / 2] = pack2<false>(y0, y1);
            add2(s0, s1, y0, y1);
          }
          tmem_store(tl + S::kColS + buf * kBlk + (half * kKeys + k0) / 2, pk, Cols<16>{});
        }
        l += s0 + s1;
        tmem_wait_store();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(buf));
      }
      // ---- the tile's output ----
      if (ok) {
        const uint32_t done = kTiles == 2 ? o_done(u) : o_done((n - 1) & 1);
        ok = warp_wait(done, kTiles == 2 ? n_items & 1 : ((n - 1) >> 1) & 1);
      }
      if (kHalves > 1 && any_of_row(!ok)) ok = false;
      if (!ok) continue;                         // to the barrier behind which both leave
      ++n_items;
      tc_fence_after();
      l = joined(l, [](float a, float b) { return a + b; });
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);     // NaN stays
      // where a lane's row goes, in 16-byte pieces from the tile's first row (P Hq rows' pieces are below 2^32)
      const uint32_t my_row = (uint32_t)(((long long)tok_of_row * A.Hq + gq) * (kD / 8));
      const uint32_t rows_mine = __ballot_sync(0xffffffffu, mine);
      uint4* const out = reinterpret_cast<uint4*>(A.out) + ((size_t)(w.row0 + ta) * A.Hq + (size_t)w.h * A.G) * (kD / 8);
      const bool has_odd = *odd != 0;
#pragma unroll 1
      for (int c0 = half * (kD / kHalves); c0 < (half + 1) * (kD / kHalves); c0 += 64) {
        uint32_t o[64];
        tmem_load(tl + S::kColO + u * kD + c0, o);
        if (__builtin_expect(has_odd, 0) && mine) {
          // Infinities and NaN that were held back (rare), where they are seen
          const int low = A.window > 0 ? max(0, tok - A.window + 1) : 0;
          for (int i = w.begin(u); i < w.end(u); ++i) {
            if (w.clean(i)) continue;
            for (int j = max(low, i * kBlk); j <= min(tok, i * kBlk + kBlk - 1); ++j) {
              const uint16_t* v = A.v + (size_t)(w.row0 + j) * A.v_stride + (size_t)w.h * kD + c0;
#pragma unroll
              for (int k = 0; k < 64; ++k) {
                const uint32_t bits = (uint32_t)v[k] << 16;
                if ((bits & 0x7f800000u) == 0x7f800000u)
                  o[k] = __float_as_uint(__uint_as_float(o[k]) + __uint_as_float(bits));
              }
            }
          }
        }
        __syncwarp();
        // Through shared memory, so that a store writes 128 bytes of each of four
        // rows: with a row to a lane, each touches 32 lines, and the two tiles'
        // outputs took 5000 cycles.
        const uint32_t mine_at = stage + warp * S::kStage + lane * 128;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t y[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            y[x] = pack2<false>(__uint_as_float(o[8 * k + 2 * x]) * inv, __uint_as_float(o[8 * k + 2 * x + 1]) * inv);
          sts128(mine_at + ((k ^ (lane & 7)) << 4), y[0], y[1], y[2], y[3]);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = k * 4 + (lane >> 3);
          const uint4 y = lds128(stage + warp * S::kStage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
          const uint32_t to = __shfl_sync(0xffffffffu, my_row, r);
          if ((rows_mine >> r) & 1u) out[to + (uint32_t)(c0 / 8 + (lane & 7))] = y;
        }
        __syncwarp();                        // the next load is the whole warp's
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();   // every role has left its loop
  tc_fence_after();
  if (warp == kIssue) tmem_dealloc(tmem, 512);
  if (*abort && warp == kLoad && lane == 0) {
    // A wait gave up: let every copy already issued land before the CTA exits.
    for (int s = 0; s < kR; ++s)
      if (issued & (1u << s)) wait_drain(full(s), (issued_phase >> s) & 1u);
    for (int u = 0; u < kTiles; ++u)
      if (issued_q & (1u << u)) wait_drain(q_full(u), (issued_q_phase >> u) & 1u);
  }
}

template <int kD, bool kExtra>
cudaError_t launch_prompt(const PromptLaunch& A, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          cudaStream_t stream) {
  using S = PromptShape<kD>;
  static std::atomic<int> smem_set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !smem_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(prompt_attn_kernel<kD, kExtra>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    // The softmax warps' larger share comes out of what the block starts with;
    // with less than that the kernel would wait for it without end.
    cudaFuncAttributes attrs;
    e = cudaFuncGetAttributes(&attrs, prompt_attn_kernel<kD, kExtra>);
    if (e != cudaSuccess) return e;
    if (S::kTiles == 2 && attrs.numRegs * S::kThreads < 32 * (S::kSoft * kSoftRegs + kRoleWarps * kRoleRegs))
      return cudaErrorLaunchOutOfResources;
    if (dev >= 0 && dev < 64) smem_set[dev].store(1, std::memory_order_release);
  }
  const long long most = A.max_items * A.Hkv;
  const int ctas = (int)(most < kCacheAttnCtas ? most : kCacheAttnCtas);
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (A.items) {
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    e = cudaLaunchKernelEx(&cfg, prompt_plan_kernel<kD>, A, ctas);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  return cudaLaunchKernelEx(&cfg, prompt_attn_kernel<kD, kExtra>, A, tq, tk, tv);
}

template <int kD>
cudaError_t launch_prompt_dim(const PromptLaunch& A, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, cudaStream_t stream) {
  return A.cap > 0.f || A.slopes ? launch_prompt<kD, true>(A, tq, tk, tv, stream)
                                 : launch_prompt<kD, false>(A, tq, tk, tv, stream);
}

}  // namespace cache_attn

cudaError_t launch_prompt_attention(const PromptLaunch& A, int D, const CUtensorMap& tmap_q, const CUtensorMap& tmap_k,
                                    const CUtensorMap& tmap_v, cudaStream_t stream) {
  switch (D) {
    case 64: return cache_attn::launch_prompt_dim<64>(A, tmap_q, tmap_k, tmap_v, stream);
    case 128: return cache_attn::launch_prompt_dim<128>(A, tmap_q, tmap_k, tmap_v, stream);
    case 256: return cache_attn::launch_prompt_dim<256>(A, tmap_q, tmap_k, tmap_v, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace specdec
