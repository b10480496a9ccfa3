// stem_kernels.h — kernel launch interfaces used by the host API (stem_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "stem_internal.h"

namespace stem {

// Per-sequence TMA descriptors of one launch (kernel parameters, so the
// kernels need no descriptor copies in global memory).
struct ScoreMaps {
  CUtensorMap q[kMaxSeqPerLaunch];  // token traversal stride s, box 256 tokens
  CUtensorMap k[kMaxSeqPerLaunch];
  // the full s-token groups of a sequence as (dim, head, slot, group), box of
  // 128 (q) or 256 (k) groups of one slot; valid where group_maps[seq] != 0
  CUtensorMap q_groups[kMaxSeqPerLaunch];
  CUtensorMap k_groups[kMaxSeqPerLaunch];
  int group_maps[kMaxSeqPerLaunch];
};

struct BsaMaps {
  CUtensorMap q[kMaxSeqPerLaunch];  // box 128 tokens
  CUtensorMap k[kMaxSeqPerLaunch];  // box 64 tokens (unused when K/V are paged)
  CUtensorMap v[kMaxSeqPerLaunch];
  CUtensorMap k_pool;               // paged K/V: the whole page pool as [pages * page_size] tokens
  CUtensorMap v_pool;
};

struct ScoreArgs {
  int hq, hkv, nbtot, nb_max, stride;
  int block;                // block size (tokens): 128 or 64
  int hk0;                  // first KV head of the launch (its items cover consecutive KV heads)
  int num_sms;              // SMs of the device (the CTA order depends on it, never the results)
  float scale;              // 1 / (sqrt(d) s n)
  const float* q_scale;     // fp8 only
  const float* k_scale;
  const float* vbonus;      // [Hkv][NBtot]
  float* scores;            // [Hq][NBtot][nb_max]
  int* status;
  // fused selection: when set, every CTA also selects the rows it scored
  // (budgets and row_ptr must be complete; nb_max <= kFusedSelectMaxBlocks)
  int fuse_select;
  int sink, window;
  const int32_t* budgets;
  const int32_t* row_ptr;
  int32_t* col_idx;
};
// largest nb_max for which the scoring kernel can select its rows itself (the
// per-warp selection scratch lives in the drained operand stages)
constexpr int kFusedSelectMaxBlocks = 5888;

struct BsaArgs {
  int hq, hkv, nbtot, total_tokens;
  int block;                // block size (tokens): 128, or 64 (one CTA then covers query blocks 2p and 2p + 1)
  int hk0;                  // first KV head of the launch (its items cover consecutive KV heads)
  const int32_t* page_table;  // paged K/V: [num_seqs][max_pages] physical page per logical page, else null
  int page_size;            // tokens per page, a multiple of 64
  int max_pages;            // row length of page_table
  float scale_log2;         // softmax scale * log2(e)
  const float* q_scale;     // fp8 only
  const float* k_scale;
  const float* v_scale;
  const int32_t* row_ptr;
  const int32_t* col_idx;
  const void* q;            // [T, Hq, d] (rows are read straight into TMEM)
  void* out;                // bf16 [T, Hq, d]
  float* lse;               // [Hq][T]
  int* status;
};

// KV heads hk0 .. hk0 + nhk - 1 only.  raw_log: write x = ln max ||v||^2 for a
// later launch_bonus_standardize instead of beta * max(0, x).
cudaError_t launch_vnorm(const SeqBatch& batch, const void* v, const float* v_scale, bool fp8, int hkv, int hk0,
                         int nhk, int nbtot, int block, float beta, bool raw_log, float* vbonus,
                         cudaStream_t stream);
// vbonus[hk][g] = beta * max(0, (x - mean) / std) over the finite x of each
// sequence, for KV heads hk0 .. hk0 + (items per sequence) - 1.
cudaError_t launch_bonus_standardize(const SeqBatch& batch, int hk0, int nbtot, float beta, float* vbonus,
                                     cudaStream_t stream);
cudaError_t launch_score(const ScoreMaps& maps, const SeqBatch& batch, const ScoreArgs& args, bool fp8,
                         cudaStream_t stream);
cudaError_t launch_budget(const SeqBatch& batch, int hq, int nbtot, int64_t nnz_per_head, double rho, double mu,
                          int sink, int window, int mode, int32_t* budgets, int32_t* row_ptr, cudaStream_t stream);
// rows of query heads h0 .. h0 + nh - 1 only; `group` consecutive heads share
// one list selected on the max of their scores (batch items: nh / group * nb
// per sequence)
cudaError_t launch_select(const SeqBatch& batch, int hq, int h0, int nh, int group, int nbtot, int nb_max, int sink,
                          int window,
                          const float* scores, const int32_t* budgets, const int32_t* row_ptr, int32_t* col_idx,
                          cudaStream_t stream);
cudaError_t launch_bsa(const BsaMaps& maps, const SeqBatch& batch, const BsaArgs& args, bool fp8,
                       cudaStream_t stream);
// Rows whose lists are shared by the query heads of a KV group: one CTA per
// (query block, pair of query heads), K and V staged once for the pair
// (batch items: nhk * ceil(G / 2) * nb per sequence).
cudaError_t launch_bsa_pair(const BsaMaps& maps, const SeqBatch& batch, const BsaArgs& args, bool fp8,
                            cudaStream_t stream);
// fp8 V widened to f16 rows [T, Hkv, d] for KV heads hk0 .. hk0 + nhk - 1, read
// packed or (page_table non-null) through the page table.
cudaError_t launch_vwiden(const void* v8, uint16_t* v16, int total_tokens, int hkv, int hk0, int nhk,
                          const int32_t* cu_seqlens, int num_seqs, const int32_t* page_table, int page_size,
                          int num_pages, int max_pages, cudaStream_t stream);

// Raises a kernel's shared-memory limit, once per device (`done`: a bit for each).
inline cudaError_t allow_smem(const void* kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
  if ((done.load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// ---- the paged cache (k_cache_extend.cu, k_rope.cu, k_tree_attn.cu)

// 3-D map of [rows, heads, 128] (a page pool or queries), box: box_heads heads of
// box_rows rows, row-major, 128-byte swizzle, one 128-byte slab wide.
bool encode_rows_map(CUtensorMap* m, const void* base, bool fp8, int heads, int rows, int box_heads, int box_rows);

constexpr int kMaxExtendSeqs = 8192;  // sequences of one stem_cache_extend (16 B of SMEM each)
struct ExtendArgs {
  int seqs, max_tokens, page_size, num_pages, max_pages, num_free, mask_words;
  const int32_t *cache_lens, *new_lens, *held, *free_pages, *cursor, *parents;
  int32_t *page_table, *held_out, *cursor_out, *cu_seqlens, *kv_lens, *slots, *positions;
  uint32_t* mask;
  int* status;
};
cudaError_t launch_cache_extend(const ExtendArgs& args, cudaStream_t stream);

struct RopeArgs {
  uint64_t turn[kHeadDim / 2];  // angular frequency of pair j in 2^-64 turns per position
  float amplitude;
  int rotary_dim;
  int tokens;
  int hq, hkv, hv;              // heads of q, k and v (0: that tensor is not asked for)
  int hkv_rows;                 // KV heads of a token
  const int32_t *positions, *slots;
  const uint8_t *q, *k, *v;     // bf16 rows
  int64_t q_stride, k_stride, v_stride;  // bytes between tokens
  const float *q_scale, *k_scale, *v_scale;
  uint8_t *q_out, *k_out, *v_out, *k_pages, *v_pages;
  int pool_rows;
};
cudaError_t launch_rope(const RopeArgs& args, bool interleaved, bool fp8, cudaStream_t stream);

struct TreeMaps {
  CUtensorMap q;       // box: the group's query heads of tile_tokens tokens
  CUtensorMap k_pool;  // the page pool as [pages * page_size] rows, boxes of 64
  CUtensorMap v_pool;
};
struct TreeArgs {
  int seqs, total_tokens, max_seq_tokens, hq, hkv;
  int group;            // query heads per KV head
  int tile_tokens;      // tokens of a 128-row query tile
  int box_rows;         // rows of the Q box (tile_tokens, or the longest sequence's tokens, times group)
  int tiles;            // query tiles of the longest sequence: CTAs that share a range of keys
  int ranges;           // ranges of keys at most (the grid is ranges * tiles)
  int part_rows;        // rows of a partial result in the workspace
  int unit_keys;        // keys of a unit: 64, or 128 in the narrow kernel
  int item_units;       // units that starting and finishing an item is worth
  int min_range;        // shortest range, in units
  int page_size, num_pages, max_pages, mask_words;
  const int32_t *cu_seqlens, *kv_lens, *page_table;
  const uint32_t* mask;
  float scale_log2;
  const float *q_scale, *k_scale, *v_scale;
  const uint8_t* v_pages;
  void* out;
  float* lse;
  // workspace
  int* status;
  int* cta_status;      // [grid]
  int64_t* unit0;       // [seqs + 1]: length (of all KV heads' items) before each sequence
  float2* part_ml;      // [grid][2][part_rows]: reference max and sum
  float* part_o;        // [grid][2]: [part_rows][128] (narrow kernel) or [128][part_rows]
};
constexpr int kTreeRanges = 296;    // two CTAs on each of 148 SMs
constexpr int kNarrowRanges = 148;  // one CTA per SM (e4m3: twice as many, two per SM)
// Query rows (tokens * group) up to which the narrow kernel is used.  16 rows over
// 16K keys of 16 sequences: 164 us, against 192 us in the 128-row kernel for 64
// rows, which costs the same for fewer; for 32 rows a narrow kernel with 32
// columns took 211 us (e4m3 241), the 128-row kernel 185 (153).  16 e4m3 rows over
// 16K keys of 16 sequences: 109 us, against 126.
constexpr int kNarrowRows = 16;
// Units that an item counts beyond its own.  64 tokens over 1 to 8K keys (narrow):
// none 192 us, one 176, two or three 168; eight 32-token trees over 16-32K: none
// 167 us, two 174 and four or six 172 in an earlier state, five 165.
constexpr int kNarrowItemUnits = 2, kTreeItemUnits = 5;
// Shortest range, in units.  One token over 300 keys: 13.7 us with three, 15.3
// with four, 19.0 with eight; a 32-token tree over 1000: 19.1, 20.2 (six), 23.4
// (twelve); nothing else changes.
constexpr int kNarrowMinRange = 3, kTreeMinRange = 3;
cudaError_t launch_tree_attn(const TreeMaps& maps, const TreeArgs& args, bool fp8, cudaStream_t stream);
cudaError_t launch_tree_narrow(const TreeMaps& maps, const TreeArgs& args, bool fp8, cudaStream_t stream);

size_t score_smem_bytes();
size_t bsa_smem_bytes(bool fp8);

}  // namespace stem
