// stem_tree_common.cuh — pieces shared by the kernels of attention over the
// paged cache: the shape of a sequence, the equal cuts of the keys, the walk
// over a range's items, masks and page lookups.
#pragma once

#include "stem_device.cuh"
#include "stem_kernels.h"

namespace stem {
namespace {

// Keys and queries of one sequence, as the call sees them.
struct SeqShape {
  int tok0, n, rows;  // first packed token, new tokens, tokens that are computed
  int ctx, kv;        // keys before the new tokens (negative when some are not cached), end of the keys; ctx <= kv
  int units;          // 0: nothing to do
  bool bad;
};

__device__ __forceinline__ SeqShape seq_shape(const TreeArgs& a, int s) {
  SeqShape r;
  const int t0 = __ldg(a.cu_seqlens + s), t1 = __ldg(a.cu_seqlens + s + 1);
  const int kv = max(__ldg(a.kv_lens + s), 0);
  const int64_t cap = i64min(static_cast<int64_t>(a.max_pages) * a.page_size, 0x7fffff80);
  r.bad = t0 < 0 || t1 < t0 || t1 > a.total_tokens;
  r.tok0 = t0;
  r.n = r.bad ? 0 : t1 - t0;
  r.rows = min(r.n, a.max_seq_tokens);
  r.kv = kv < cap ? kv : static_cast<int>(cap);
  // (where the table's row ends before the new tokens, no key is one of them: the last unit is then an edge, too)
  r.ctx = min(kv - r.n, r.kv);
  r.units = r.n == 0 ? 0 : max((r.kv + a.unit_keys - 1) / a.unit_keys, 1);
  if (r.n > 0) r.bad |= r.rows < r.n || kv > cap || __ldg(a.kv_lens + s) < 0;
  return r;
}

// All items are laid end to end and cut into equal ranges.  An item's length is
// its units and a.item_units more, in front of them, for what starting and
// finishing an item costs; those are walked over.
__device__ __forceinline__ int64_t seq_length(const TreeArgs& a, const SeqShape& q) {
  return q.units == 0 ? 0 : static_cast<int64_t>(q.units + a.item_units) * a.hkv;
}
// Floor of x / y (0 <= x, 0 < y): most operands fit 32 bits, whose division is far shorter.
__device__ __forceinline__ int64_t div_floor(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}
__device__ __forceinline__ int64_t range_begin(int64_t total, int ranges, int k) { return div_floor(total * k, ranges); }
// ranges in use: none is shorter than a.min_range
__device__ __forceinline__ int ranges_used(const TreeArgs& a, int64_t total) {
  return static_cast<int>(i64max(i64min(a.ranges, div_floor(total, a.min_range)), 1));
}

// Walks the items (sequence, KV head) of a range; every role walks alike.
struct Walk {
  int s, hk, at;  // next item and the place in it
  int64_t left;   // length of the range from there on
  int index;      // items with a unit in the range so far
  SeqShape q;
  // current item
  int hk_cur, ub, ue;
  bool whole;
  __device__ __forceinline__ void start(const TreeArgs& a, int first_seq, int64_t skip, int64_t count) {
    s = first_seq;
    left = count;
    index = 0;
    q.units = 0;
    if (count > 0) {
      q = seq_shape(a, s);
      const int len = q.units + a.item_units;
      hk = static_cast<int>(div_floor(skip, len));
      at = static_cast<int>(skip - static_cast<int64_t>(hk) * len);
    }
  }
  // the next item whose sequence has this tile; false at the end of the range
  __device__ __forceinline__ bool next(const TreeArgs& a, int tile) {
    while (left > 0) {
      if (hk >= a.hkv) {
        hk = 0;
        do {
          if (++s >= a.seqs) {  // the lengths changed under the call
            left = 0;
            return false;
          }
          q = seq_shape(a, s);
        } while (q.units == 0);
      }
      hk_cur = hk;
      const int len = q.units + a.item_units;
      const int to = static_cast<int>(i64min(len, at + left));
      ub = max(at - a.item_units, 0);
      ue = to - a.item_units;
      whole = ub == 0 && ue == q.units;
      left -= to - at;
      at = to;
      if (to == len) {
        at = 0;
        ++hk;
      }
      if (ue <= ub) continue;  // the range ends before the item's first unit
      ++index;
      if (tile * a.tile_tokens < q.rows) return true;
    }
    return false;
  }
};

// Steps of P V over unit u: those that hold a key before `kv` (one if none does).
template <int kUnit, int kStepKeys>
__device__ __forceinline__ int key_steps(int kv, int u) {
  return max((min(kv - u * kUnit, kUnit) + kStepKeys - 1) / kStepKeys, 1);
}

// Bits of the 64 keys from `key0` on that query i of the sequence sees.  `known`
// holds the first `words` (at most two) words of the query's mask row.
__device__ __forceinline__ uint64_t visible(const TreeArgs& a, const SeqShape& q, int i, int key0, uint64_t known,
                                            int words) {
  const int d0 = key0 - q.ctx;  // index, among the new tokens, of the first key
  uint64_t bits;
  if (a.mask == nullptr) {
    const int seen = i + 1 - d0;  // new tokens up to i, from the first key on
    bits = seen <= 0 ? 0ull : seen >= 64 ? ~0ull : (1ull << seen) - 1;
  } else {
    const uint32_t* row = a.mask + static_cast<size_t>(q.tok0 + i) * a.mask_words;
    const int from = max(d0, 0);
    const int w = from >> 5, sh = from & 31;
    auto word = [&](int x) -> uint64_t {
      if (x < words) return x == 0 ? static_cast<uint32_t>(known) : static_cast<uint32_t>(known >> 32);
      return x < a.mask_words ? __ldg(row + x) : 0u;
    };
    const uint64_t lo = word(w) | word(w + 1) << 32;
    bits = sh == 0 ? lo : lo >> sh | word(w + 2) << (64 - sh);
    if (q.n - from < 64) bits &= (1ull << (q.n - from > 0 ? q.n - from : 0)) - 1;
    if (d0 < 0) bits = (d0 > -64 ? bits << -d0 | ((1ull << -d0) - 1) : ~0ull);
  }
  const int keys = q.kv - key0;
  if (keys < 64) bits &= keys <= 0 ? 0ull : (1ull << keys) - 1;
  return bits;
}

// A logit's factor, at least 2^-126: hidden scores are -inf, which times zero would be NaN,
// and with a factor this small all logits vanish anyway.
__device__ __forceinline__ float logit_scale(float c) { return c < 1.17549435e-38f ? 1.17549435e-38f : c; }

// Pool row of key u of sequence s, or the first row past the pool (reads zeros).
__device__ __forceinline__ int pool_row(const TreeArgs& a, int s, int u) {
  const int pg = u / a.page_size;
  const int page = pg < a.max_pages ? __ldg(a.page_table + static_cast<size_t>(s) * a.max_pages + pg) : -1;
  if (page < 0 || page >= a.num_pages) return a.num_pages * a.page_size;
  return page * a.page_size + (u - pg * a.page_size);
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// L2 cache policy for data that is read once, and the tile load that carries it.
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Non-finite bf16 elements (exponent 0xff) of a pair are zeroed.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w, bool& odd) {
  if ((w & 0x7f80u) == 0x7f80u) {
    w &= 0xffff0000u;
    odd = true;
  }
  if ((w & 0x7f800000u) == 0x7f800000u) {
    w &= 0x0000ffffu;
    odd = true;
  }
  return w;
}

// Where a range starts, found by all threads of the CTA (kThreads of them):
// prefix sums of the sequences' lengths.
struct RangeScratch {
  int64_t scan[16];
  int64_t skip;  // length of first_seq before the range
  int first_seq;
  int bad;  // bad lengths (the caller clears it first)
};
// One __syncthreads inside; the caller's next one publishes skip, first_seq and
// bad (count is known to every thread).  CTA 0 also writes unit0 for the joining
// kernel and notices bad lengths.
template <int kThreads>
__device__ __forceinline__ int64_t find_range(const TreeArgs& a, int range, RangeScratch& sm) {
  // the first read of memory that earlier kernels may still be writing
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = warp_id(), lane = lane_id();
  const int per = (a.seqs + kThreads - 1) / kThreads;
  const int s_beg = min(static_cast<int>(threadIdx.x) * per, a.seqs), s_end = min(s_beg + per, a.seqs);
  int64_t mine = 0;
  bool bad = false;
  for (int s = s_beg; s < s_end; ++s) {
    const SeqShape q = seq_shape(a, s);
    mine += seq_length(a, q);
    bad |= q.bad;
  }
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) sm.scan[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sm.scan[w];
    total += sm.scan[w];
  }
  const int used = ranges_used(a, total);
  const int64_t u0 = range < used ? range_begin(total, used, range) : total;
  const int64_t count = range < used ? range_begin(total, used, range + 1) - u0 : 0;
  if (blockIdx.x == 0) {
    if (bad) sm.bad = 1;
    int64_t at = before;
    for (int s = s_beg; s < s_end; ++s) {
      a.unit0[s] = at;
      at += seq_length(a, seq_shape(a, s));
    }
    if (threadIdx.x == 0) a.unit0[a.seqs] = total;
  }
  if (count > 0 && before <= u0 && u0 < before + mine) {
    int64_t at = before;
    int s = s_beg;
    for (; s + 1 < s_end; ++s) {
      const int64_t more = seq_length(a, seq_shape(a, s));
      if (u0 < at + more) break;
      at += more;
    }
    sm.first_seq = s;
    sm.skip = u0 - at;
  }
  return count;
}

// A CTA's word: a wait that ran out, whose outputs are invalid, stands over bad lengths.
__device__ __forceinline__ int cta_word(int status, const RangeScratch& sm) {
  return status != 0 ? status : sm.bad ? STEM_ERR_BAD_INPUT_CODE : 0;
}

// Launches a kernel whose start may overlap the end of the one before it in the
// stream (it waits for that one in griddepcontrol.wait).  One token over 1000 keys:
// 14.2 against 14.5 us, four 32-token trees over 4K 32.4 against 33.1; letting the
// joining kernel start while the main one runs took 14.3 and 33.8.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace stem
