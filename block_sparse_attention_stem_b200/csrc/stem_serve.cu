// stem_serve.cu — the paged-cache entry points of include/stem.h: argument
// checks, workspace layout, TMA maps and launches of stem_cache_extend,
// stem_rope and stem_tree_attn.  No allocation, no copies, no synchronisation.
#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "stem.h"
#include "stem_internal.h"
#include "stem_kernels.h"

using namespace stem;

namespace {

constexpr size_t kStatusBytes = 256;

struct StageRange {
  explicit StageRange(const char* name) { nvtxRangePushA(name); }
  ~StageRange() { nvtxRangePop(); }
  StageRange(const StageRange&) = delete;
  StageRange& operator=(const StageRange&) = delete;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
stem_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? STEM_OK : STEM_ERR_CUDA; }

stem_status_t check_pool(int32_t page_size, int32_t num_pages) {
  if (page_size < 64 || page_size % 64 != 0 || num_pages < 1) return STEM_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_pages) * page_size > INT32_MAX) return STEM_ERR_INVALID_ARG;
  return STEM_OK;
}

// Angular frequency of every rotated pair in units of 2^-64 turns per position.
void rope_turns(const stem_rope_t& r, RopeArgs* a) {
  constexpr long double kTwoPi = 6.283185307179586476925286766559005768L;
  constexpr long double kTurns = 18446744073709551616.0L / kTwoPi;  // 2^64 to the turn
  const int half = r.rotary_dim / 2;
  long double base = r.base;  // (NTK's may pass the range of a double)
  if (r.scaling == STEM_ROPE_NTK)
    base *= std::pow(static_cast<long double>(r.factor), static_cast<long double>(r.rotary_dim) / (r.rotary_dim - 2));
  double low = 0, high = 1;
  if (r.scaling == STEM_ROPE_YARN) {
    // the (fractional) pair that makes `turns` turns over the trained length
    auto pair_of = [&](double turns) {
      return r.rotary_dim * std::log(r.original_len / (turns * static_cast<double>(kTwoPi))) / (2.0 * std::log(r.base));
    };
    low = std::max(std::floor(pair_of(r.beta_fast)), 0.0);
    high = std::min(std::ceil(pair_of(r.beta_slow)), r.rotary_dim - 1.0);
    if (low == high) high += 0.001;
  }
  // w_j = ratio^j, carried in 64-bit mantissas: off by at most j 2^-63 of itself
  const long double ratio = std::pow(base, -2.0L / r.rotary_dim);
  long double w_j = 1.0L;
  for (int j = 0; j < half; ++j, w_j *= ratio) {
    long double w = w_j;
    if (r.scaling == STEM_ROPE_LINEAR) w /= r.factor;
    if (r.scaling == STEM_ROPE_YARN) {
      // (a ramp whose ends lie on one side of the pairs: all of them are past it, or none)
      const double t = high > low ? std::min(std::max((j - low) / (high - low), 0.0), 1.0) : j < low ? 0.0 : 1.0;
      w = w / r.factor * t + w * (1.0 - t);
    }
    a->turn[j] = static_cast<uint64_t>(w * kTurns);  // w <= 1: below 2^62
  }
  double amp = r.amplitude;
  if (amp == 0.0) amp = r.scaling == STEM_ROPE_YARN ? 0.1 * std::log(r.factor) + 1.0 : 1.0;
  a->amplitude = static_cast<float>(amp);
  a->rotary_dim = r.rotary_dim;
}

stem_status_t check_rope(const stem_rope_t* r) {
  if (!r) return STEM_ERR_INVALID_ARG;
  if (r->layout != STEM_ROPE_HALF && r->layout != STEM_ROPE_INTERLEAVED) return STEM_ERR_INVALID_ARG;
  if (r->rotary_dim < 2 || r->rotary_dim > kHeadDim || r->rotary_dim % 2 != 0) return STEM_ERR_INVALID_ARG;
  if (r->rotary_dim % 16 != 0) return STEM_ERR_UNSUPPORTED;
  if (r->scaling < STEM_ROPE_PLAIN || r->scaling > STEM_ROPE_YARN) return STEM_ERR_INVALID_ARG;
  if (!(r->base > 1.0) || !std::isfinite(r->base)) return STEM_ERR_INVALID_ARG;
  if (r->scaling != STEM_ROPE_PLAIN && (!(r->factor >= 1.0) || !std::isfinite(r->factor))) return STEM_ERR_INVALID_ARG;
  if (r->scaling == STEM_ROPE_YARN &&
      (r->original_len < 1 || !(r->beta_slow > 0.0) || !(r->beta_fast > r->beta_slow) || !std::isfinite(r->beta_fast)))
    return STEM_ERR_INVALID_ARG;
  if (!(r->amplitude >= 0.0) || !std::isfinite(r->amplitude)) return STEM_ERR_INVALID_ARG;
  return STEM_OK;
}

// One input of stem_rope: present when an output wants it.
stem_status_t check_rows(const void* in, int64_t stride, int heads, const void* packed, const void* pool,
                         const float* scale, bool fp8, bool in_place_ok) {
  if (!packed && !pool) return STEM_OK;
  if (!in || heads < 1 || stride < static_cast<int64_t>(heads) * kHeadDim || stride % 8 != 0)
    return STEM_ERR_INVALID_ARG;
  if (stride > INT64_MAX / 4 / INT32_MAX) return STEM_ERR_INVALID_ARG;  // byte offsets of every token fit 64 bits
  if (!aligned(in, 16) || (packed && !aligned(packed, 16)) || (pool && !aligned(pool, 16))) return STEM_ERR_MISALIGNED;
  if (fp8 && !scale) return STEM_ERR_INVALID_ARG;
  if (packed == in && (!in_place_ok || fp8 || stride != static_cast<int64_t>(heads) * kHeadDim))
    return STEM_ERR_INVALID_ARG;
  return STEM_OK;
}

constexpr double kMaxScale = 0x1p127;  // times log2(e) it is still an fp32 number

struct TreeLayout {
  int group, tile_tokens, box_tokens, tiles, ranges, part_rows, unit_keys;
  size_t off_cta, off_unit0, off_ml, off_o, bytes;
};

stem_status_t tree_layout(const stem_tree_t* t, TreeLayout* out) {
  if (!t) return STEM_ERR_INVALID_ARG;
  if (t->dtype != STEM_BF16 && t->dtype != STEM_FP8_E4M3) return STEM_ERR_INVALID_ARG;
  if (t->num_seqs < 1 || t->total_tokens < 0 || t->max_seq_tokens < 0) return STEM_ERR_INVALID_ARG;
  if (t->num_q_heads < 1 || t->num_kv_heads < 1 || t->num_q_heads % t->num_kv_heads != 0) return STEM_ERR_INVALID_ARG;
  if (t->head_dim != kHeadDim) return t->head_dim < 1 ? STEM_ERR_INVALID_ARG : STEM_ERR_UNSUPPORTED;
  if (t->mask ? t->mask_words < 1 : t->mask_words < 0) return STEM_ERR_INVALID_ARG;
  if (!(t->softmax_scale >= 0.0) || t->softmax_scale > kMaxScale) return STEM_ERR_INVALID_ARG;
  if (t->total_tokens > (1 << 30) || static_cast<int64_t>(t->num_seqs) * t->num_kv_heads > (1 << 30))
    return STEM_ERR_UNSUPPORTED;
  TreeLayout l{};
  l.group = t->num_q_heads / t->num_kv_heads;
  if (l.group > 128) return STEM_ERR_UNSUPPORTED;
  l.tile_tokens = 128 / l.group;
  const int most = t->max_seq_tokens > 0 && t->max_seq_tokens < t->total_tokens ? t->max_seq_tokens
                                                                                : std::max(t->total_tokens, 1);
  l.box_tokens = std::min(l.tile_tokens, most);
  l.tiles = (most + l.tile_tokens - 1) / l.tile_tokens;
  const bool narrow = most <= kNarrowRows / l.group;
  l.unit_keys = narrow ? 128 : 64;
  l.ranges = narrow ? kNarrowRanges * (t->dtype == STEM_FP8_E4M3 ? 2 : 1) : std::max(kTreeRanges / l.tiles, 1);
  const int rows32 = (l.box_tokens * l.group + 31) / 32 * 32;
  l.part_rows = narrow ? l.box_tokens * l.group : rows32;
  const size_t grid = std::max<size_t>(static_cast<size_t>(l.ranges) * l.tiles, kTreeRanges);
  l.off_cta = kStatusBytes;
  l.off_unit0 = l.off_cta + align256(grid * sizeof(int));
  l.off_ml = l.off_unit0 + align256((static_cast<size_t>(t->num_seqs) + 1) * sizeof(int64_t));
  // sized for the largest grid and tile of these heads, so that the size never shrinks with the lengths
  const size_t parts = static_cast<size_t>(kTreeRanges) * 2 * rows32;
  l.off_o = l.off_ml + align256(parts * sizeof(float2));
  l.bytes = l.off_o + align256(parts * kHeadDim * sizeof(float));
  *out = l;
  return STEM_OK;
}

}  // namespace

extern "C" {

stem_status_t stem_cache_extend(const stem_cache_step_t* step, int32_t* page_table, int32_t* held_out,
                                int32_t* cursor_out, int32_t* cu_seqlens, int32_t* kv_lens, int32_t* slots,
                                int32_t* positions, uint32_t* mask, void* ws, size_t ws_bytes, stem_stream_t stream) {
  if (!step || step->num_seqs < 1 || step->max_tokens < 0 || step->num_free < 0 || step->max_pages_per_seq < 1)
    return STEM_ERR_INVALID_ARG;
  stem_status_t st = check_pool(step->page_size, step->num_pages);
  if (st != STEM_OK) return st;
  // counters of tokens and table entries step past their ends in 32 bits
  if (step->max_tokens > (1 << 30) || static_cast<int64_t>(step->num_seqs) * step->max_pages_per_seq > (1 << 30))
    return STEM_ERR_INVALID_ARG;
  if (!step->cache_lens || !step->new_lens || !step->held_pages || !step->cursor ||
      (!step->free_pages && step->num_free > 0))
    return STEM_ERR_INVALID_ARG;
  if (!page_table || !held_out || !cursor_out || !cu_seqlens || !kv_lens || !ws) return STEM_ERR_INVALID_ARG;
  if (step->max_tokens > 0 && (!slots || !positions)) return STEM_ERR_INVALID_ARG;
  if ((step->parents != nullptr) != (mask != nullptr) || (mask && step->mask_words < 1)) return STEM_ERR_INVALID_ARG;
  if (!aligned(ws, 4)) return STEM_ERR_MISALIGNED;
  if (ws_bytes < kStatusBytes) return STEM_ERR_WORKSPACE_TOO_SMALL;
  if (step->num_seqs > kMaxExtendSeqs) return STEM_ERR_UNSUPPORTED;
  StageRange nvtx_range("stem: cache extend");
  ExtendArgs a{};
  a.seqs = step->num_seqs;
  a.max_tokens = step->max_tokens;
  a.page_size = step->page_size;
  a.num_pages = step->num_pages;
  a.max_pages = step->max_pages_per_seq;
  a.num_free = step->num_free;
  a.mask_words = step->mask_words;
  a.cache_lens = step->cache_lens;
  a.new_lens = step->new_lens;
  a.held = step->held_pages;
  a.free_pages = step->free_pages;
  a.cursor = step->cursor;
  a.parents = step->parents;
  a.page_table = page_table;
  a.held_out = held_out;
  a.cursor_out = cursor_out;
  a.cu_seqlens = cu_seqlens;
  a.kv_lens = kv_lens;
  a.slots = slots;
  a.positions = positions;
  a.mask = mask;
  a.status = static_cast<int*>(ws);
  return cuda_status(launch_cache_extend(a, reinterpret_cast<cudaStream_t>(stream)));
}

stem_status_t stem_rope(const stem_rope_t* rope, const stem_rope_io_t* io, const stem_paged_kv_t* cache,
                        stem_stream_t stream) {
  stem_status_t st = check_rope(rope);
  if (st != STEM_OK) return st;
  if (!io || io->num_tokens < 0 || io->num_q_heads < 0 || io->num_kv_heads < 0) return STEM_ERR_INVALID_ARG;
  if (io->out_dtype != STEM_BF16 && io->out_dtype != STEM_FP8_E4M3) return STEM_ERR_INVALID_ARG;
  if (io->head_dim != kHeadDim) return io->head_dim < 1 ? STEM_ERR_INVALID_ARG : STEM_ERR_UNSUPPORTED;
  if (io->num_q_heads > 4096 || io->num_kv_heads > 2048) return STEM_ERR_UNSUPPORTED;
  if (cache) {
    if ((st = check_pool(cache->page_size, cache->num_pages)) != STEM_OK) return st;
    if (!cache->k_pages || !cache->v_pages) return STEM_ERR_INVALID_ARG;
  }
  if (io->num_tokens == 0) return STEM_OK;
  if (!io->q_out && !io->k_out && !io->v_out && !cache) return STEM_ERR_INVALID_ARG;
  if (!io->positions || (cache && !io->slots)) return STEM_ERR_INVALID_ARG;
  const bool fp8 = io->out_dtype == STEM_FP8_E4M3;
  void* kp = cache ? const_cast<void*>(cache->k_pages) : nullptr;
  void* vp = cache ? const_cast<void*>(cache->v_pages) : nullptr;
  if ((st = check_rows(io->q, io->q_stride, io->num_q_heads, io->q_out, nullptr, io->q_scale, fp8, true)) != STEM_OK ||
      (st = check_rows(io->k, io->k_stride, io->num_kv_heads, io->k_out, kp, io->k_scale, fp8, true)) != STEM_OK ||
      (st = check_rows(io->v, io->v_stride, io->num_kv_heads, io->v_out, vp, io->v_scale, fp8, false)) != STEM_OK)
    return st;
  StageRange nvtx_range("stem: rope");
  RopeArgs a{};
  rope_turns(*rope, &a);
  a.tokens = io->num_tokens;
  a.hq = io->q_out ? io->num_q_heads : 0;
  a.hkv = io->k_out || cache ? io->num_kv_heads : 0;
  a.hkv_rows = io->num_kv_heads;
  a.hv = io->v_out || cache ? io->num_kv_heads : 0;
  a.positions = io->positions;
  a.slots = io->slots;
  a.q = static_cast<const uint8_t*>(io->q);
  a.k = static_cast<const uint8_t*>(io->k);
  a.v = static_cast<const uint8_t*>(io->v);
  a.q_stride = io->q_stride * 2;
  a.k_stride = io->k_stride * 2;
  a.v_stride = io->v_stride * 2;
  a.q_scale = io->q_scale;
  a.k_scale = io->k_scale;
  a.v_scale = io->v_scale;
  a.q_out = static_cast<uint8_t*>(io->q_out);
  a.k_out = static_cast<uint8_t*>(io->k_out);
  a.v_out = static_cast<uint8_t*>(io->v_out);
  a.k_pages = static_cast<uint8_t*>(kp);
  a.v_pages = static_cast<uint8_t*>(vp);
  a.pool_rows = cache ? cache->num_pages * cache->page_size : 0;
  return cuda_status(
      launch_rope(a, rope->layout == STEM_ROPE_INTERLEAVED, fp8, reinterpret_cast<cudaStream_t>(stream)));
}

stem_status_t stem_tree_plan(const stem_tree_t* tree, size_t* ws_bytes) {
  if (!ws_bytes) return STEM_ERR_INVALID_ARG;
  TreeLayout l;
  const stem_status_t st = tree_layout(tree, &l);
  if (st == STEM_OK) *ws_bytes = l.bytes;
  return st;
}

stem_status_t stem_tree_attn(const stem_tree_t* tree, const stem_paged_kv_t* kv, void* out, float* lse, void* ws,
                             size_t ws_bytes, stem_stream_t stream) {
  TreeLayout l;
  stem_status_t st = tree_layout(tree, &l);
  if (st != STEM_OK) return st;
  if (!kv || !ws) return STEM_ERR_INVALID_ARG;
  if ((st = check_pool(kv->page_size, kv->num_pages)) != STEM_OK) return st;
  if (kv->max_pages_per_seq < 1) return STEM_ERR_INVALID_ARG;
  const bool fp8 = tree->dtype == STEM_FP8_E4M3;
  if (tree->total_tokens > 0) {
    if (!tree->q || !out || !lse) return STEM_ERR_INVALID_ARG;
    if (!aligned(tree->q, 16) || !aligned(out, 16)) return STEM_ERR_MISALIGNED;
  }
  if (!tree->cu_seqlens || !tree->kv_lens || !kv->page_table || !kv->k_pages || !kv->v_pages)
    return STEM_ERR_INVALID_ARG;
  if (!aligned(kv->k_pages, 16) || !aligned(kv->v_pages, 16)) return STEM_ERR_MISALIGNED;
  if (!aligned(ws, 16)) return STEM_ERR_MISALIGNED;
  if (fp8 && (!tree->q_scale || !tree->k_scale || !tree->v_scale)) return STEM_ERR_INVALID_ARG;
  if (ws_bytes < l.bytes) return STEM_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (tree->total_tokens == 0) return cuda_status(cudaMemsetAsync(ws, 0, sizeof(int), s));
  StageRange nvtx_range("stem: tree attention");
  TreeMaps maps;
  const int rows = kv->num_pages * kv->page_size;
  if (!encode_rows_map(&maps.q, tree->q, fp8, tree->num_q_heads, tree->total_tokens, l.group, l.box_tokens) ||
      !encode_rows_map(&maps.k_pool, kv->k_pages, fp8, tree->num_kv_heads, rows, 1, 64) ||
      !encode_rows_map(&maps.v_pool, kv->v_pages, fp8, tree->num_kv_heads, rows, 1, 64))
    return STEM_ERR_CUDA;
  uint8_t* w = static_cast<uint8_t*>(ws);
  TreeArgs a{};
  a.seqs = tree->num_seqs;
  a.total_tokens = tree->total_tokens;
  a.max_seq_tokens = tree->max_seq_tokens > 0 ? tree->max_seq_tokens : tree->total_tokens;
  a.hq = tree->num_q_heads;
  a.hkv = tree->num_kv_heads;
  a.group = l.group;
  a.tile_tokens = l.tile_tokens;
  a.box_rows = l.box_tokens * l.group;
  a.tiles = l.tiles;
  a.ranges = l.ranges;
  a.part_rows = l.part_rows;
  a.unit_keys = l.unit_keys;
  a.item_units = l.unit_keys == 128 ? kNarrowItemUnits : kTreeItemUnits;
  a.min_range = l.unit_keys == 128 ? kNarrowMinRange : kTreeMinRange;
  a.page_size = kv->page_size;
  a.num_pages = kv->num_pages;
  a.max_pages = kv->max_pages_per_seq;
  a.mask_words = tree->mask_words;
  a.cu_seqlens = tree->cu_seqlens;
  a.kv_lens = tree->kv_lens;
  a.page_table = kv->page_table;
  a.mask = tree->mask;
  const double scale = tree->softmax_scale > 0.0 ? tree->softmax_scale : 1.0 / std::sqrt(static_cast<double>(kHeadDim));
  a.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  a.q_scale = tree->q_scale;
  a.k_scale = tree->k_scale;
  a.v_scale = tree->v_scale;
  a.v_pages = static_cast<const uint8_t*>(kv->v_pages);
  a.out = out;
  a.lse = lse;
  a.status = reinterpret_cast<int*>(w);
  a.cta_status = reinterpret_cast<int*>(w + l.off_cta);
  a.unit0 = reinterpret_cast<int64_t*>(w + l.off_unit0);
  a.part_ml = reinterpret_cast<float2*>(w + l.off_ml);
  a.part_o = reinterpret_cast<float*>(w + l.off_o);
  return cuda_status(launch_tree_attn(maps, a, fp8, s));
}

}  // extern "C"
