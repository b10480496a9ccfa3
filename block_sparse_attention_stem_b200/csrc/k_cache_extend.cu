// k_cache_extend.cu — page tables, slot maps, positions and tree masks of one
// step, from lengths that are on the GPU.
//
// Everything follows from two exclusive prefix sums over the sequences: of the
// new tokens (cu) and of the pages to take (tp).  Token t belongs to the last
// sequence with cu <= t, new page e to the last one with tp <= e, so both maps
// are a binary search in shared memory, and a long prompt costs no more than
// the same tokens spread over many sequences.
//
// Measured on the GPU: four requests with a token each 3.9 us, 256 trees of 17 to
// 64 tokens 9.4 us (with eight CTAs at most 13.4), 213K prompt tokens 13.3 us.
//
// One cluster: every CTA reads all lengths and repeats the (short) scans, the
// cluster's barrier separates those reads from the writes, so the outputs may
// be the inputs (a captured step advances its own lengths), and then the CTAs
// share the tokens and pages.  A step moves a few hundred bytes to a few MB, so
// launches bound it: one launch, no clearing pass.
#include <cooperative_groups.h>

#include "stem_device.cuh"
#include "stem_kernels.h"

namespace stem {

namespace {

constexpr int kExtendThreads = 1024;

// Exclusive prefix sum of one value per thread over the block; *total gets the
// sum.  `scratch`: 33 words, free for reuse after the call's last barrier.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* scratch, int64_t* total) {
  const int lane = lane_id(), warp = warp_id();
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t w = scratch[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += y;
    }
    scratch[lane] = w;
  }
  __syncthreads();
  const int64_t before = warp > 0 ? scratch[warp - 1] : 0;
  *total = scratch[31];
  __syncthreads();
  return before + x - v;
}

// Last index s with a[s] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int find_last(const int32_t* a, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace

__global__ void __launch_bounds__(kExtendThreads, 1) cache_extend_kernel(const ExtendArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ int32_t sm_seq[];  // cu, tp, cache length, held: S words each
  __shared__ int64_t scratch[33];
  const int S = a.seqs, ps = a.page_size;
  int32_t* cu = sm_seq;
  int32_t* tp = cu + S;
  int32_t* clen = tp + S;
  int32_t* held = clen + S;
  const int tid = threadIdx.x;
  bool bad = false, out_of_pages = false;

  const int cur_in = *a.cursor;  // (may be written below, after every CTA has read it)
  const int cursor = min(max(cur_in, 0), a.num_free);
  bad |= cursor != cur_in;
  const int avail = a.num_free - cursor;

  int64_t tokens = 0, pages = 0;  // running totals over the chunks of 1024 sequences
  for (int s0 = 0; s0 < S; s0 += kExtendThreads) {
    const int s = s0 + tid;
    int c = 0, n = 0, h = 0;
    if (s < S) {
      c = a.cache_lens[s];
      n = a.new_lens[s];
      h = a.held[s];
      bad |= c < 0 || n < 0 || h < 0 || h > a.max_pages;
      c = max(c, 0);
      n = max(n, 0);
      h = min(max(h, 0), a.max_pages);
    }
    int64_t sum;
    const int64_t at = tokens + block_scan(n, scratch, &sum);
    tokens += sum;
    // tokens that do not fit the outputs are dropped
    const int64_t room = at < a.max_tokens ? a.max_tokens - at : 0;
    const int64_t kept = n < room ? n : room;
    bad |= kept != n;
    const uint32_t end = static_cast<uint32_t>(c) + static_cast<uint32_t>(kept);  // < 2^32
    const int64_t want = end == 0 ? 0 : (end - 1) / static_cast<uint32_t>(ps) + 1;
    out_of_pages |= want > a.max_pages;
    const int64_t need = want < a.max_pages ? want : a.max_pages;
    const int64_t first = pages + block_scan(need > h ? need - h : 0, scratch, &sum);
    pages += sum;
    if (s < S) {
      cu[s] = static_cast<int32_t>(at < a.max_tokens ? at : a.max_tokens);
      tp[s] = static_cast<int32_t>(first);  // < S * max_pages < 2^31
      clen[s] = c;
      held[s] = h;
    }
  }
  const int T = static_cast<int>(tokens < a.max_tokens ? tokens : a.max_tokens);
  const int P = static_cast<int>(pages);
  out_of_pages |= P > avail;
  const int rank = static_cast<int>(cluster.block_rank()), size = static_cast<int>(cluster.num_blocks());
  if (rank == 0 && tid == 0) *a.status = 0;
  cluster.sync();  // every length is read (and staged): from here on the outputs are written

  for (int s = rank * kExtendThreads + tid; s < S; s += size * kExtendThreads) {
    const int t1 = s + 1 < S ? cu[s + 1] : T, p1 = s + 1 < S ? tp[s + 1] : P;
    const int got = max(min(p1, avail) - tp[s], 0);
    a.cu_seqlens[s] = cu[s];
    a.kv_lens[s] = static_cast<int32_t>(i64min(static_cast<int64_t>(clen[s]) + (t1 - cu[s]), 0x7fffffff));
    a.held_out[s] = held[s] + got;
  }
  if (rank == 0 && tid == 0) {
    a.cu_seqlens[S] = T;
    *a.cursor_out = cursor + min(P, avail);
  }
  // new pages, in the order of the list
  for (int e = rank * kExtendThreads + tid; e < P; e += size * kExtendThreads) {
    const int s = find_last(tp, S, e);
    int page = -1;
    if (e < avail) {
      page = __ldg(a.free_pages + cursor + e);
      if (page < 0 || page >= a.num_pages) {
        page = -1;
        bad = true;
      }
    }
    a.page_table[static_cast<size_t>(s) * a.max_pages + held[s] + (e - tp[s])] = page;
  }
  // tokens: slot, position and the bits of the ancestors
  for (int t = rank * kExtendThreads + tid; t < a.max_tokens; t += size * kExtendThreads) {
    int slot = -1, pos = 0, cur = -1;
    const int32_t* par = a.parents;
    if (t < T) {
      const int s = find_last(cu, S, t);
      const int i = t - cu[s];
      const uint32_t p = static_cast<uint32_t>(clen[s]) + static_cast<uint32_t>(i);  // < 2^32
      pos = static_cast<int>(min(p, 0x7fffffffu));
      const uint32_t pg = p / static_cast<uint32_t>(ps);
      if (pg < static_cast<uint32_t>(a.max_pages)) {
        const int e = static_cast<int>(pg) - held[s];
        int page = -1;
        if (e < 0) page = a.page_table[static_cast<size_t>(s) * a.max_pages + pg];  // entries < held are not written
        else if (tp[s] + e < avail) page = __ldg(a.free_pages + cursor + tp[s] + e);
        if (page >= 0 && page < a.num_pages) slot = page * ps + static_cast<int>(p - pg * static_cast<uint32_t>(ps));
        else bad |= e < 0 || tp[s] + e < avail;
      }
      if (par != nullptr) {
        par += cu[s];
        cur = i;
        pos = clen[s];
      }
    }
    a.slots[t] = slot;
    if (a.mask != nullptr) {
      // ancestors come in descending order, so the words are finished one by one from the last
      uint32_t* row = a.mask + static_cast<size_t>(t) * a.mask_words;
      int w = a.mask_words - 1, depth = -1;
      uint32_t bits = 0;
      while (cur >= 0) {
        ++depth;
        const int cw = cur >> 5;
        if (cw >= a.mask_words) {
          bad = true;
        } else {
          for (; w > cw; --w) {
            row[w] = bits;
            bits = 0;
          }
          bits |= 1u << (cur & 31);
        }
        const int up = __ldg(par + cur);
        if (up >= cur || up < -1) {
          bad = true;
          break;
        }
        cur = up;
      }
      for (; w >= 0; --w) {
        row[w] = bits;
        bits = 0;
      }
      if (depth > 0) pos = static_cast<int>(i64min(static_cast<int64_t>(pos) + depth, 0x7fffffff));
    }
    a.positions[t] = pos;
  }
  // the larger code stands, whichever thread comes first
  static_assert(STEM_ERR_OUT_OF_PAGES_CODE > STEM_ERR_BAD_INPUT_CODE, "a step without pages says so");
  if (out_of_pages) atomicMax(a.status, STEM_ERR_OUT_OF_PAGES_CODE);
  else if (bad) atomicMax(a.status, STEM_ERR_BAD_INPUT_CODE);
}

cudaError_t launch_cache_extend(const ExtendArgs& args, cudaStream_t stream) {
  // a CTA for every 1024 outputs (tokens, or sequences), up to the largest cluster
  const int work = args.max_tokens > args.seqs ? args.max_tokens : args.seqs;
  unsigned ctas = 1;
  while (ctas < 16 && work > static_cast<int>(ctas) * kExtendThreads) ctas *= 2;
  const size_t smem = static_cast<size_t>(args.seqs) * 4 * sizeof(int32_t);
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) {
    // the largest step's, once: a smaller one must not lower it under another thread's launch
    static std::atomic<uint64_t> allowed{0};
    constexpr size_t kMostSmem = static_cast<size_t>(kMaxExtendSeqs) * 4 * sizeof(int32_t);
    e = allow_smem(reinterpret_cast<const void*>(cache_extend_kernel), kMostSmem, allowed);
    if (e != cudaSuccess) return e;
  }
  if (ctas > 8) {  // more than the portable cluster
    e = cudaFuncSetAttribute(cache_extend_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  if (ctas == 1) {
    cache_extend_kernel<<<1, kExtendThreads, smem, stream>>>(args);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kExtendThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, cache_extend_kernel, args);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace stem
