// Host-side launch interface between the C ABI (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace specdec {

// LM-head scoring on the tensor cores (bf16 inputs): logits z = hidden.W^T
// for every token row, with the per-tile softmax / argmax partials and the
// draft-logit partials fused into the epilogue.
struct TcLaunch {
  const CUtensorMap* tmap_w;     // W_lm [V, d], box {64, 128}, 128B swizzle
  const CUtensorMap* tmap_h;     // hidden [M, d], box {64, BT}, 128B swizzle
  const CUtensorMap* tmap_z;     // logits [M, V] fp32, box {32, 32}, 128B swizzle; or null
  int M, V, d, gamma;
  int* status;
  float* fix;                    // stream-K fix-up slots (tc_fix_floats floats)
  unsigned long long* fix_tickets;   // kFixSlots tags, any initial contents
  unsigned long long epoch;      // per-call tag (next_call_epoch)
  const unsigned long long* calls;   // the workspace header's call count
  int max_clusters;              // co-resident clusters of the launch shape (0: unknown)
  int withhold_loads;            // self-test of the bounded waits (normally 0)
  EpiParams ep;
};
cudaError_t launch_lmhead_tc(const TcLaunch& L, int num_sms, cudaStream_t stream);

// The same scoring for fp32 inputs on the CUDA cores.
cudaError_t launch_lmhead_f32(const float* hidden, const float* W, int d, const EpiParams& ep,
                              int* status, cudaStream_t stream);

// A tag that no earlier call in this process used.
unsigned long long next_call_epoch();

// Combine the partials, apply the acceptance rule, write the kept prefix.
struct AcceptLaunch {
  int B, gamma, V, P, Pq, mode, dl_bf16;   // P, Pq: records per p row and per q row
  float c;                       // log2(e) / T
  uint64_t seed;
  const PartialP* pp;
  const PartialQ* pq;
  const float* z;
  const void* dl;
  const int32_t* draft_tokens;
  int32_t* out_tokens;
  int32_t* n_accepted;
  SelectedRow* sel;
  int* counters;
  int* status;
  unsigned long long* calls;     // the workspace header's call count (one added per call)
  float* lse_p;
  float* lse_q;
  float* p_x;
  float* q_x;
  int32_t* argmax_out;
  int tok_offset;                // vocabulary-parallel shard: first token ID it holds (else 0)
};
cudaError_t launch_accept(const AcceptLaunch& L, cudaStream_t stream);

// Residual / bonus draw for every sequence (sampling mode).
struct SampleLaunch {
  int B, gamma, V, nchunks, dl_bf16;
  int vec;          // set by the launcher: 16-byte logit and draft-logit loads are aligned
  int prefetch;     // set by the launcher: small batch, rows prefetched into L2 early
  float c;
  uint64_t seed;
  const float* z;
  const void* dl;
  const SelectedRow* sel;
  float* chunk_sums;
  int* counters;
  int32_t* out_tokens;
};
// Up to kSampleOneKernelItems (sequence, chunk) pairs one kernel sums the
// chunks and draws (the last CTA of each sequence to finish draws); beyond,
// a kernel of chunk sums and a kernel of one drawing CTA per sequence.
constexpr long long kSampleOneKernelItems = 608;
cudaError_t launch_sample(const SampleLaunch& L, cudaStream_t stream);
// Small batches in sampling mode: acceptance and draw in one kernel (every
// drawing CTA folds its sequence's records itself). The sampler tickets
// must be zero when it starts: the LM-head kernel clears them
// (EpiParams::counters). kFusedAcceptItems bounds B * nchunks.
constexpr long long kFusedAcceptItems = 128;
bool fused_accept_sample(int B, int nchunks);
cudaError_t launch_accept_sample(const AcceptLaunch& A, const SampleLaunch& L,
                                 cudaStream_t stream);

// Vocabulary-parallel step (one slice of the vocabulary per GPU). A slice's
// records: target rows [M] (max z, sum exp2, argmax value and global token
// ID), draft rows [B*gamma] (max, sum exp2), guessed tokens [B*gamma] (the
// two logits when this slice holds the token); segments 256-byte aligned.
struct ShardRec {
  float m, s, amax_v;
  int amax_i;
};
struct ShardQRec {
  float m, s;
};
struct ShardXRec {
  float zx, zqx;
  int owned, pad;
};
size_t shard_record_bytes(int B, int gamma);
// Fold the slice's LM-head records into one record per row (A.V = the
// slice's vocabulary, A.tok_offset = its first token ID).
cudaError_t launch_shard_fold(const AcceptLaunch& A, void* records, cudaStream_t stream);
// Fold the gathered records of all slices and decide (A.V = the whole vocabulary).
cudaError_t launch_shard_accept(const AcceptLaunch& A, const void* all_records,
                                size_t record_bytes, int n_shards, cudaStream_t stream);
// The slice's (residual, p) weight sums of each sequence's drawn row.
// Few sequences (B * chunks <= kFusedAcceptItems): accept and the slice sums
// in one kernel; its chunk tickets use counters the LM head zeroed.
bool shard_fused_accept_sums(int B, int nchunks);
cudaError_t launch_shard_accept_sums(const AcceptLaunch& A, const SampleLaunch& L,
                                     const void* all_records, size_t record_bytes, int n_shards,
                                     float* cs_p, float2* shard_sums, cudaStream_t stream);
cudaError_t launch_shard_sums(const SampleLaunch& L, float* cs_p, float2* shard_sums,
                              cudaStream_t stream);
// The draw: the slice holding t = u * S writes its token, the others -1.
cudaError_t launch_shard_draw(const SampleLaunch& L, const float* cs_p, const float2* all_sums,
                              int n_shards, int shard, int tok_offset, cudaStream_t stream);

// Tree verification walk: one cluster of kTreeCluster CTAs per sequence
// (sampling; the CTAs split the vocabulary), kTreeClusterWide when every
// sequence's cluster of that size can be resident at once, or one CTA
// (greedy).
constexpr int kTreeCluster = 8;
constexpr int kTreeClusterWide = 16;
struct TreeLaunch {
  int B, N, V, P, Pq, mode, vec;
  float c;
  uint64_t seed;
  const PartialP* pp;            // [B*N, P] target records
  const PartialQ* pq;            // [B*N, Pq] draft records (sampling)
  const float* z;                // [B*N, V] fp32 logits (sampling)
  const __nv_bfloat16* dl;       // [B*N, V] draft logits (sampling)
  const int32_t* tok;            // [B, N] node tokens (column 0 unused)
  int16_t first_child[SPECDEC_MAX_TREE_NODES];    // -1: none; children in increasing index
  int16_t next_sibling[SPECDEC_MAX_TREE_NODES];
  int16_t parent[SPECDEC_MAX_TREE_NODES];         // parent[0] = -1
  int32_t* out_tokens;           // [B, N]
  int32_t* out_nodes;            // [B, N]
  int32_t* n_accepted;           // [B]
  int* status;
  unsigned long long* calls;     // the workspace header's call count (one added per call)
};
cudaError_t launch_tree_walk(const TreeLaunch& L, cudaStream_t stream);

// Host entry point staging through mapped pinned host memory: segments of
// `bytes` copied from host to the workspace in `unit`-byte pieces (16, 4 or
// 1; both ends aligned to it), the remainder byte by byte.
struct HostSeg {
  const void* src;
  void* dst;
  long long bytes;
  int unit;
};
struct StageInLaunch {
  HostSeg seg[3];
  int nseg;
};
cudaError_t launch_stage_in(const StageInLaunch& S, int num_sms, cudaStream_t stream);

// Verify-step attention (one layer): split-KV partials and their merge.
struct AttnLaunch {
  int B, n_new, Hq, Hkv, Lmax, n_splits, split_len;
  int n_stages;                      // K/V blocks in flight per CTA (attn_n_stages)
  float scale_log2;                  // softmax scale times log2(e)
  const __nv_bfloat16* q;            // [B, n_new, Hq, 128]
  const __nv_bfloat16* k;            // [B, Lmax, Hkv, 128]
  const __nv_bfloat16* v;
  const int32_t* seq_lens;           // [B]
  float* out;                        // [B, n_new, Hq, 128]
  float* part_m;                     // [B, Hkv, n_splits, 64] (n_splits > 1)
  float* part_l;
  float* part_o;                     // [B, Hkv, n_splits, 64, 128]
  int* status;
};
// tmap_k, tmap_v: the caches as 4-D bf16 tensors {128, Hkv, Lmax, B} with a
// {64, 1, 64, 1} box and the 128-byte swizzle.
cudaError_t launch_attention(const AttnLaunch& A, const CUtensorMap& tmap_k,
                             const CUtensorMap& tmap_v, cudaStream_t stream);
int attn_n_stages(int B, int n_new, int Hq, int Hkv);
int attn_smem_bytes(int n_mt, int n_stages);

// Verify-step attention with caps, biases, windows and token trees, over a
// bf16 or an e4m3 cache (cache_attention.cuh).
constexpr int kCacheAttnCtas = 152;       // CTAs at most: one per SM of a 152-SM part,
constexpr int kCacheAttnMaxCtas = 304;    // or two (cache_attention_keys.cuh)
struct CacheAttnLaunch {
  int B, n_new, Hq, Hkv, G, Lmax;    // G = Hq / Hkv
  int n_groups, group_pos;           // the new positions in equal groups of at most 128 rows
  int window;                        // a position sees distances below it (0: all)
  int tree;                          // 1: anc and depth describe the new positions
  int max_depth;                     // of the new positions (n_new - 1 for a chain)
  int n_scale;                       // scales per (sequence, KV head)
  int head_lanes;                    // CTAs beside each other on a part: Hkv, or 1
  int note_tiles;                    // a note per tile (this many), or 0: per CTA
  float scale, cap, cap_exp;         // cap_exp = 2 log2(e) / cap
  long long q_stride;                // elements from one position's queries to the next's
  const __nv_bfloat16* q;            // [B, n_new, Hq, D]
  const void* v;                     // the value cache
  const float* k_scale;              // [B, Hkv, n_scale] (e4m3 cache)
  const float* v_scale;
  const float* slopes;               // [Hq] or null
  const int32_t* seq_lens;           // [B]
  __nv_bfloat16* out;                // [B, n_new, Hq, D]
  float* part_o;                     // [2 CTAs, rows, D]
  float* part_ml;                    // [2 CTAs, rows, 2]
  int4* notes;                       // [tiles or CTAs] who shares a tile (write_note)
  int* status;                       // the status word, and whether a length was bad, for the merge
  uint32_t anc[SPECDEC_MAX_TREE_NODES][4];   // bit a of row i: node i sees node a
  uint8_t depth[SPECDEC_MAX_TREE_NODES];
};
// Lanes that a group of query rows takes: 32, 64 or 128.
constexpr int cache_attn_rows(int rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }
// Keys per block (and TMA box): 128, but 64 at 256 dims (shared memory) and
// for 128 lanes of query rows, where a lane holds a score of every key. 64
// against 128 keys there (when both were built, before scores were released
// early): 38.3 / 40.9 us on a 26-node tree over 8 x 4096 bf16 rows, 127 / 139
// over 32 x 4096 e4m3 rows. With fewer lanes 128 pay: 30.2 /
// 27.6 us for 20 query rows on 16 ragged bf16 sequences with a window.
constexpr int cache_attn_block(int D, int lanes) { return D == 256 || lanes == 128 ? 64 : 128; }
// The form with the cache on the M side (cache_attention_keys.cuh) can take a
// call with up to 24 query rows per KV head, and does from 256 tiles or 4096
// blocks of cache on. Measured, keys against rows form, us a call: 64 x 4096
// rows 105 / 121, 1 x 131072 53.5 / 58.5, 1 x 65536 36.6 / 37.9, 256 x 128 71 /
// 99, 64 x 200 28 / 38, 32 x 256 17.2 / 23.3; below, its longer way to a tile's
// first block shows: 1 x 517 13.5 / 12.0, 8 x 4096 29.7 / 28.3, 16 x 2048 31.2 /
// 30.1, and between 2048 and 4096 blocks the two are within 4 % of each other,
// either way: 1 x 32768 25.4 / 25.9, 10 x 4096 31.4 / 31.3, 12 x 4096 34.0 / 35.3,
// 14 x 4096 38.6 / 38.3 (8 KV heads, 20 query rows each). The lengths are on the
// device, so the cache's capacity stands for them: one sequence of 517 rows in a
// cache of 131072 takes 14.3 us here and would take 13.4 in the other form.
// With a distance bias steep heads leave whole blocks without weights, and each
// costs this form a look at its references: 64 x 384 38.5 / 42.1, but 64 x 512
// 46.4 / 45.5, 64 x 4096 150 / 130.
constexpr int kCacheAttnKeyRows = 24;
constexpr bool cache_attn_can_key(bool e4m3, int D, int rows) { return e4m3 && D == 128 && rows <= kCacheAttnKeyRows; }
inline bool cache_attn_by_keys(const CacheAttnLaunch& A, int D) {
  const long long tiles = (long long)A.B * A.Hkv * A.n_groups;
  return cache_attn_can_key(true, D, A.group_pos * A.G) &&
         (tiles >= 256 || tiles * ((A.Lmax + 127) / 128) >= 4096) && (!A.slopes || A.Lmax < 512);
}
// tmap_q: the queries as a bf16 tensor {D, Hq, n_new, B} with a box of 64
// dims x G heads x group_pos positions, 128-byte swizzle (bf16 cache only).
cudaError_t launch_cache_attention_kv8(const CacheAttnLaunch& A, int D, const CUtensorMap& tmap_k,
                                       const CUtensorMap& tmap_v, const CUtensorMap& tmap_q,
                                       cudaStream_t stream);
cudaError_t launch_cache_attention_bf16(const CacheAttnLaunch& A, int D, const CUtensorMap& tmap_k,
                                        const CUtensorMap& tmap_v, const CUtensorMap& tmap_q,
                                        cudaStream_t stream);

// Quantise new positions' keys and values into an e4m3 cache.
struct Kv8AppendLaunch {
  int B, n, Hkv, D, Lmax, n_scale, max_blocks;
  const __nv_bfloat16* src[2];       // k_new, v_new [B, n, Hkv, D]
  long long stride[2];               // elements from one position to the next
  uint8_t* cache[2];                 // [B, Lmax, Hkv, D] e4m3
  float* scale[2];                   // [B, Hkv, n_scale]
  const int32_t* start;              // [B]
  const int32_t* counts;             // [B] or null (n)
  const int32_t* rows;               // [B, n] or null (0, 1, ...)
  int* status;
};
cudaError_t launch_kv8_append(const Kv8AppendLaunch& A, cudaStream_t stream);

// The driver's tensor-map encoder (null when the driver lacks it).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// The drafter's clustered LM head.
struct ClusterLaunch {
  int M, d, V, n_c, top_k, max_cluster, max_members, sort_n, sample, position;
  float c;                           // log2(e) / T
  uint64_t seed;
  const __nv_bfloat16* h;            // [M, d]
  const __nv_bfloat16* E;            // [n_c, d]
  const __nv_bfloat16* W;            // [V, d] rows grouped by cluster
  const int32_t* starts;             // [n_c + 1]
  const int32_t* token_of_row;       // [V]
  float* y;                          // [M, n_c] cluster logits
  int* offs;                         // [M, top_k + 1] kept members' prefix
  float* z;                          // [M, max_members] kept members' logits
  int* ids;                          // [M, max_members] their token IDs
  int32_t* clusters;                 // [M, top_k]
  int32_t* tokens;                   // [M]
  float* logits_out;                 // [M, V] or null
  int* status;
};
cudaError_t launch_cluster_head(const ClusterLaunch& L, cudaStream_t stream);

cudaError_t launch_philox_uniforms(uint64_t seed, int B, int n_pos, int purpose, float* out,
                                   cudaStream_t stream);

// Tile geometry and schedule of the tensor-core path, shared by the
// workspace planner and the launcher.
constexpr int kMaxGrid = 256;    // persistent CTAs at most (one per SM)
constexpr int kFixSlots = kMaxGrid + 2;   // stream-K boundaries x cluster ranks
struct TcGeometry {
  int BT;                        // token rows per tile: multiple of 16, <= 256
  int n_tt;                      // token tiles
  int kc;                        // 64-wide k slices per shared-memory stage
  int box3d;                     // 3-D boxes {64, rows, kc} (d % 64 == 0)
  int stages, stage_bytes, tmem_cols, smem_bytes;
  int n_vt;                      // vocabulary tiles of 128
  int K;                         // CTAs per cluster sharing hidden slices
  int n_units, nk, grid;
  int stream_k;                  // one token tile: contiguous k-iteration ranges
  int records;                   // partial records per row (grid or vocabulary tiles)
  int rowown;                    // 1: tokens on the MMA's M side (pairs, 256-row token tiles)
  int n_acc;                     // accumulators a tile's k-slices are dealt across (swap-AB)
};
TcGeometry tc_geometry(int M, int V, int d, int num_sms, int max_clusters);
// Co-resident clusters of the kernel for this shape on the current device
// (0 when the shape runs without clusters).
int tc_max_clusters(int M, int V, int d);
// Floats of stream-K fix-up storage for a shape (0 without stream-K).
inline size_t tc_fix_floats(int M, int V, int d) {
  const TcGeometry g = tc_geometry(M, V, d, kMaxGrid, 0);
  return g.stream_k ? (size_t)kFixSlots * 2 * g.BT * kBlockV : 0;
}

}  // namespace specdec
