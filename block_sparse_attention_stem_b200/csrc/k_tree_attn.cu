// k_tree_attn.cu — attention of drafted trees, single tokens or causal chunks
// over the paged cache (more than 16 query rows per sequence and KV head; fewer:
// k_tree_narrow.cu), and the kernels that join the pieces of both.
//
//   O = sum_u exp2(c q.k_u - m) v_u / l,  m the running reference max, l the sum
//
// over the keys u of the sequence: all cached ones, and of the step's own
// tokens those whose bit is set in the query's mask row.  The query heads of a
// KV group and the tokens of a sequence share the keys, so they are the rows of
// one 128-row tile (row = token * group + head), and the keys, 64 at a time
// ("unit"), stream through tcgen05 as in the block-sparse kernel:
//   S = Q K^T     tcgen05.mma M 128, N 64 into S buffer h % 2 (TMEM)
//   P = exp2(..)  the softmax warps (thread = row = TMEM lane), over S
//   O += P V      tcgen05.mma, P from TMEM, V from SMEM; O stays in TMEM
//
// Work split: all SMs have to stream all the time, whatever the lengths.  The
// items (sequence, KV head) are laid end to end and cut into equal ranges, one
// per CTA (two CTAs per SM); an item counts a few units more than it has, for
// its start and its epilogue.  A range may hold the end of one item, several
// whole ones and the start of another; whole ones are written at once, the at
// most two pieces go to the workspace (fp32 O, m, l; dim by dim, so that a
// warp's 32 rows are one line) and a second kernel joins them in range order.
// The cuts depend on the lengths alone, so results repeat bit for bit.  Sequences
// with more than 128 rows have several tiles: the CTAs of one range (blockIdx =
// range * tiles + tile) read the same keys at the same time, from L2.
//
// bf16: P is kept as a sum of two bf16 (15 significant bits; they fill the 64
// columns of S exactly), so its rounding does not add to the output's: with a
// single bf16 P the error of a long average is as large as the output rounding
// itself.  e4m3: Q K^T on the e4m3 operands, P in f16, V widened to f16 (exact)
// by warps of their own.  The largest weight of a row is kept at 2^13 to 2^15.9 of
// f16's 2^16, since a small weight has to keep its bits where an attention sink
// takes most of the sum: it is off by 2^-11 of itself down to 2^-27 of the row's
// largest (19 nats), by 2^-38 of the largest below.  (The reference then moves at
// 2^2.9 over it instead of 2^8, and with it that of every row of the warp that grew:
// sixteen 33-63-token trees 197 against 192 us; without the others' 199; at 2^12 and
// 2^3.9 194.5.)
//
// Masked keys: S is replaced by -inf, so nothing in K matters.  A product 0 * v
// would still carry a NaN or infinity of V into rows that do not see the key,
// so in units that hold new tokens or the end of the sequence, rows of V behind
// the end are zeroed in SMEM and non-finite elements of new tokens too; rows
// that do see such an element get it added in the epilogue.
//
// What bounds it.  bf16, one full tile: HBM (eight 32-token trees over 16-32K,
// 811 MB: the kernel reads 5.67 TB/s, 143 us; 163 us with the join, about 200
// when the power cap lowers the clock; tensor pipe 57%).  e4m3: no unit is full
// (sixteen 33-63-token trees, two tiles, 346 MB: 197 to 206 us; issue slots 47%, tensor
// pipe 32%, HBM 26%), what takes the time is each unit's chain of waits through
// four roles, with the work done for each of the two tiles: scores read from TMEM
// twice, V fetched and widened twice.  The roles share one instruction cache.
// Steps on the way, before the f16 weights were raised: rolling the exponentials
// and the widening loop took 279 to 222 us, four widening warps at 96 registers
// 213, fixed addresses without bank conflicts 206 to 192.  Widening by moving
// bits instead of cvt measured 316 us, keeping the scores in registers with two
// widening warps 195.
//
// 192 threads (320 for e4m3):
//   warps 0-3  softmax, epilogue (TMEM lane quarter = warp)
//   warp  4    TMA producer of Q, K and V
//   warp  5    TMEM owner and MMA issuer    warps 6-9 (e4m3)  V -> f16
// Every wait is bounded; on expiry all roles leave and the call reports it.
#include "stem_bsa_common.cuh"
#include "stem_tree_common.cuh"

namespace stem {

namespace {

constexpr int kUnit = 64;  // keys per S buffer
constexpr int kProducer = 4, kMmaIssuer = 5, kWidenWarp = 6;
constexpr uint32_t kTmemCols = 256;  // S buffers at 0 and 64, O at 128

template <bool kFp8>
struct TreeCfg {
  static constexpr int kWidenWarps = 4;
  static constexpr bool kKeep = !kFp8;  // scores stay in registers between the maximum and the exponentials
  static constexpr int kThreads = 192 + (kFp8 ? kWidenWarps * 32 : 0);
  static constexpr int kQBytes = kFp8 ? 16384 : 32768;
  static constexpr int kSlabs = kFp8 ? 1 : 2;  // 128-byte slabs of a head row
  static constexpr int kUnitBytes = kFp8 ? 8192 : 16384;
  static constexpr int kKSlots = kFp8 ? 4 : 3;
  static constexpr int kVSlots = kFp8 ? 4 : 2;
  // A row's reference puts its largest weight at 2^kBias; it moves when one passes that by more
  // than 2^kSlack.  e4m3: f16 ends at 65504 and loses bits below 2^-14.
  static constexpr float kBias = kFp8 ? 13.f : 0.f;
  static constexpr float kSlack = kFp8 ? 2.9f : BsaCfg<false>::kRescaleLog2;
};

template <bool kFp8>
struct TreeSmem {
  using C = TreeCfg<kFp8>;
  uint8_t q[C::kQBytes];  // 1024-aligned
  uint8_t k[C::kKSlots][C::kUnitBytes];
  uint8_t v[C::kVSlots][C::kUnitBytes];
  uint8_t wide[kFp8 ? 2 : 1][kFp8 ? 16384 : 16];  // V as f16, e4m3 only
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[C::kKSlots], k_empty[C::kKSlots];
  uint64_t v_full[C::kVSlots], v_empty[C::kVSlots];
  uint64_t wide_full[2];
  uint64_t s_full[2];   // S_h complete
  uint64_t p_full[2];   // the softmax warps stored P_h (and rescaled O)
  uint64_t pv_done[2];  // P_h V_h complete
  uint64_t drain;
  RangeScratch range;
  uint32_t tmem_base;
  int status, abort;
  int odd_v[4];  // [item % 4]: item + 1 when a non-finite element of V was zeroed in it
};

// Four e4m3 bytes as two f16 pairs (exact).
__device__ __forceinline__ void widen_e4m3x4(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

// Scores of keys that are not seen become -inf.
__device__ __forceinline__ void hide(uint32_t (&rr)[32], uint32_t see) {
#pragma unroll
  for (int x = 0; x < 32; ++x)
    if (!((see >> x) & 1u)) rr[x] = 0xff800000u;
}

}  // namespace

template <bool kFp8>
__global__ void __launch_bounds__(TreeCfg<kFp8>::kThreads, 2)
    tree_attn_kernel(const __grid_constant__ TreeMaps maps, const __grid_constant__ TreeArgs a) {
  using Cfg = TreeCfg<kFp8>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  TreeSmem<kFp8>& sm = *reinterpret_cast<TreeSmem<kFp8>*>(smem_raw);
  const int warp = warp_id(), lane = lane_id();
  const int range = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;

  // ---- where this range starts: prefix sum of the sequences' units
  if (threadIdx.x == 0) {
    sm.status = 0;
    sm.range.bad = 0;
    sm.abort = (smem_u32(smem_raw) & 1023u) != 0;  // the swizzled tiles need this alignment
    if (sm.abort) sm.status = STEM_ERR_TIMEOUT_CODE;
    for (int x = 0; x < 4; ++x) sm.odd_v[x] = 0;
  }
  // the barriers, a lane each, and the tensor maps' fetch, before earlier kernels are waited for
  constexpr int kBars = 13 + 2 * Cfg::kKSlots + 2 * Cfg::kVSlots;
  static_assert(offsetof(TreeSmem<kFp8>, drain) == offsetof(TreeSmem<kFp8>, q_full) + (kBars - 1) * 8, "barriers in a row");
  if (warp == kMmaIssuer && lane < kBars) {
    uint64_t* bar = &sm.q_full[0] + lane;
    uint32_t count = 1;
    if (bar >= &sm.p_full[0] && bar < &sm.p_full[2]) count = 4;
    if (kFp8 && bar >= &sm.wide_full[0] && bar < &sm.wide_full[2]) count = Cfg::kWidenWarps;
    if (kFp8 && bar >= &sm.v_empty[0] && bar < &sm.v_empty[Cfg::kVSlots]) count = Cfg::kWidenWarps;
    mbar_init(bar, count);
    fence_mbar_init();
  }
  if (warp == kProducer && lane < 3) tma_prefetch_desc(lane == 0 ? &maps.k_pool : lane == 1 ? &maps.q : &maps.v_pool);
  const int64_t count = find_range<Cfg::kThreads>(a, range, sm.range);
  if (count == 0) {
    __syncthreads();
    if (threadIdx.x == 0) a.cta_status[blockIdx.x] = cta_word(sm.status, sm.range);
    return;
  }
  if (warp == kMmaIssuer) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;
  int* status = &sm.status;
  Walk wk;
  wk.start(a, sm.range.first_seq, sm.range.skip, count);
  // Q tiles of at most 64 rows have two buffers, so that the next item's
  // products need not wait for the last one's
  const int qbufs = a.box_rows <= 64 ? 2 : 1;
  const int qslab = 16384 / qbufs;  // bytes of a slab

  if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    // Lane 0 issues; the warp looks up 32 units' pages at a time.  K runs ahead
    // of V by `ahead` units.  While V_h is the next V, the products up to
    // S_{h+1} can complete, and the Q tile of K_{h+ahead-1} may have to wait for
    // S_{h+ahead-1-qbufs} (items of one unit): hence ahead <= 2 + qbufs.
    struct Stream {
      Walk w;
      int u, rows, h, slot, round;
      bool more;
    };
    Stream ks{wk, 0, 0, 0, 0, 0, false}, vs{wk, 0, 0, 0, 0, 0, false};
    int item = 0;  // Q tiles issued
    bool ok = !*abort;
    auto enter = [&](Stream& st) {
      st.more = st.w.next(a, tile);
      if (st.more) st.u = st.w.ub;
    };
    // issues the stream's next unit; false when a wait ran out
    auto load = [&](Stream& st, const CUtensorMap* m, uint8_t* base, uint64_t* full, uint64_t* empty, int slots) -> bool {
      const int x = (st.u - st.w.ub) & 31;
      if (x == 0) st.rows = pool_row(a, st.w.s, min(st.u + lane, st.w.ue - 1) * kUnit);
      const int row = __shfl_sync(0xffffffffu, st.rows, x);
      bool good = true;
      if (lane == 0) {
        if (st.round > 0) good = mbar_wait(&empty[st.slot], (st.round - 1) & 1, abort, status);
        if (good) {
          mbar_arrive_expect_tx(&full[st.slot], Cfg::kUnitBytes);
          for (int y = 0; y < Cfg::kSlabs; ++y)
            tma_load_3d(base + st.slot * Cfg::kUnitBytes + y * (kUnit * 128), m, &full[st.slot], y * 64, st.w.hk_cur, row);
        }
      }
      if (!__shfl_sync(0xffffffffu, good, 0)) return false;
      ++st.h;
      if (++st.slot == slots) {
        st.slot = 0;
        ++st.round;
      }
      ++st.u;
      return true;
    };
    auto load_k = [&]() -> bool {
      if (ks.u == ks.w.ub) {
        bool good = true;
        if (lane == 0) {
          const int b = item % qbufs;
          if (item >= qbufs) good = mbar_wait(&sm.q_empty[b], (item / qbufs - 1) & 1, abort, status);
          if (good) {
            mbar_arrive_expect_tx(&sm.q_full[b], a.box_rows * 128 * Cfg::kSlabs);
            for (int x = 0; x < Cfg::kSlabs; ++x)
              tma_load_3d(sm.q + (b * Cfg::kSlabs + x) * qslab, &maps.q, &sm.q_full[b], x * 64, ks.w.hk_cur * a.group,
                          ks.w.q.tok0 + tile * a.tile_tokens);
          }
        }
        if (!__shfl_sync(0xffffffffu, good, 0)) return false;
        ++item;
      }
      if (!load(ks, &maps.k_pool, sm.k[0], sm.k_full, sm.k_empty, Cfg::kKSlots)) return false;
      if (ks.u == ks.w.ue) enter(ks);
      return true;
    };
    if (ok) {
      enter(ks);
      enter(vs);
    }
    const int ahead = min(Cfg::kKSlots, 2 + qbufs);
    for (int x = 0; x < ahead && ok && ks.more; ++x) ok = load_k();
    while (ok && vs.more) {
      ok = load(vs, &maps.v_pool, sm.v[0], sm.v_full, sm.v_empty, Cfg::kVSlots);
      if (ok && vs.u == vs.w.ue) enter(vs);
      if (ok && ks.more) ok = load_k();
    }
    // every copy has landed before the CTA can exit (a slot or Q buffer has at
    // most one copy in flight)
    if (lane == 0) {
      auto quiesce = [&](uint64_t* full, int slots, int n) {
        for (int x = 0; x < slots && x < n; ++x) {
          const int last = n - 1 - (n - 1 - x) % slots;
          mbar_wait_quiesce(&full[x], (last / slots) & 1, status);
        }
      };
      quiesce(sm.k_full, Cfg::kKSlots, ks.h);
      quiesce(sm.v_full, Cfg::kVSlots, vs.h);
      quiesce(sm.q_full, qbufs, item);
    }
    __syncwarp();
  } else if (warp == kMmaIssuer) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      const uint32_t idesc_s = make_idesc(kFp8 ? 0u : 1u, 0u, 128u, static_cast<uint32_t>(kUnit));
      const uint32_t idesc_o = make_idesc(kFp8 ? 0u : 1u, 1u, 128u, 128u);
      const uint32_t o_tmem = tmem + 128;
      // two walks: S runs two units ahead of P V
      Walk ws = wk;
      int hs = 0, us = 0, qitem = -1;
      bool more_s = ws.next(a, tile);
      if (more_s) us = ws.ub;
      auto issue_s = [&]() -> bool {
        if (us == ws.ub) {
          ++qitem;
          if (!mbar_wait(&sm.q_full[qitem % qbufs], (qitem / qbufs) & 1, abort, status)) return false;
        }
        const int slot = hs % Cfg::kKSlots;
        if (!mbar_wait(&sm.k_full[slot], (hs / Cfg::kKSlots) & 1, abort, status)) return false;
        tc_fence_after();
        const uint64_t dq = make_sdesc_sw128(smem_u32(sm.q) + (qitem % qbufs) * Cfg::kSlabs * qslab, 16, 1024);
        const uint64_t dk = make_sdesc_sw128(smem_u32(sm.k[slot]), 16, 1024);
        const uint32_t d = tmem + kUnit * (hs & 1);
        // descriptors count 16-byte units
        if constexpr (kFp8) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8_ss(d, dq + kk * 2, dk + kk * 2, idesc_s, kk != 0);
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ss(d, dq + (kk >> 2) * (qslab >> 4) + (kk & 3) * 2, dk + (kk >> 2) * (kUnit * 8) + (kk & 3) * 2, idesc_s,
                        kk != 0);
        }
        mma_commit(&sm.k_empty[slot]);
        mma_commit(&sm.s_full[hs & 1]);
        ++hs;
        if (++us == ws.ue) {
          mma_commit(&sm.q_empty[qitem % qbufs]);
          more_s = ws.next(a, tile);
          if (more_s) us = ws.ub;
        }
        return true;
      };
      bool ok = !*abort;
      for (int x = 0; x < 2 && ok && more_s; ++x) ok = issue_s();
      int h = 0;
      while (ok && wk.next(a, tile)) {
        for (int u = wk.ub; u < wk.ue && ok; ++u, ++h) {
          const int slot = h % Cfg::kVSlots;
          uint64_t* vbar = kFp8 ? &sm.wide_full[h & 1] : &sm.v_full[slot];
          ok = mbar_wait(&sm.p_full[h & 1], (h >> 1) & 1, abort, status) &&
               mbar_wait(vbar, (kFp8 ? h >> 1 : h / Cfg::kVSlots) & 1, abort, status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv = make_sdesc_sw128(smem_u32(kFp8 ? sm.wide[h & 1] : sm.v[slot]), kUnit * 128, 1024);
          const uint32_t p = tmem + kUnit * (h & 1);
          const int steps = key_steps<kUnit, 16>(wk.q.kv, u);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 16 keys per step
            if (kk < steps) mma_bf16_ts(o_tmem, p + (kFp8 ? kk * 8 : (kk >> 1) * 32 + (kk & 1) * 8), dv + kk * 128, idesc_o,
                        u != wk.ub || kk != 0);
          if constexpr (!kFp8) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // the low parts of P
              if (kk < steps) mma_bf16_ts(o_tmem, p + (kk >> 1) * 32 + (kk & 1) * 8 + 16, dv + kk * 128, idesc_o, 1u);
            mma_commit(&sm.v_empty[slot]);
          }
          mma_commit(&sm.pv_done[h & 1]);
          if (more_s) ok = issue_s();
        }
      }
      mma_commit(&sm.drain);
      mbar_wait_quiesce(&sm.drain, 0, status);
    }
    __syncwarp();
  } else if (kFp8 && warp >= kWidenWarp) {
    // ------------------------------------------------------------ V -> f16
    if constexpr (kFp8) {
      // Thread: 16-byte chunk c of rows r, r + 16, r + 32, r + 48, whose 16 elements are
      // chunks 2 (c % 4) and + 1 of slab c / 4 of the wide tile.  The lanes of one slab
      // take even rows while those of the other take odd ones, so that the eight
      // lanes of a shared-memory phase write eight different chunk positions.
      const int t = (warp - kWidenWarp) * 32 + lane;
      const int c = t & 7, r = (t >> 3) ^ (c >> 2);
      const int from = r * 128 + ((c ^ (r & 7)) << 4);
      const int to = (c >> 2) * (kUnit * 128) + r * 128;
      const int to0 = to + (((2 * (c & 3)) ^ (r & 7)) << 4), to1 = to + (((2 * (c & 3) + 1) ^ (r & 7)) << 4);
      int h = 0;
      bool ok = !*abort;
      for (int item = 0; ok && wk.next(a, tile); ++item) {
        for (int u = wk.ub; u < wk.ue; ++u, ++h) {
          const int slot = h % Cfg::kVSlots;
          ok = mbar_wait(&sm.v_full[slot], (h / Cfg::kVSlots) & 1, abort, status) &&
               (h < 2 || mbar_wait(&sm.pv_done[h & 1], ((h - 2) >> 1) & 1, abort, status));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint8_t* src = sm.v[slot] + from;
          uint8_t* dst = sm.wide[h & 1];
          const bool check = (u + 1) * kUnit > wk.q.ctx;
          const int fresh = wk.q.ctx - u * kUnit;  // rows from here on are new tokens, or
          const int end = wk.q.kv - u * kUnit;     // from here on behind the keys
          bool odd = false;
#pragma unroll 1
          for (int step = 0; step < kUnit * 128; step += Cfg::kWidenWarps * 4 * 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + step);
            const uint32_t in[4] = {x.x, x.y, x.z, x.w};
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) widen_e4m3x4(in[e], w[2 * e], w[2 * e + 1]);
            if (check && r + step / 128 >= fresh) {  // a cached key's NaN is everyone's
              const bool behind = r + step / 128 >= end;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                if (behind) w[e] = 0u;
                if ((w[e] & 0x7c00u) == 0x7c00u) {
                  w[e] &= 0xffff0000u;
                  odd = true;
                }
                if ((w[e] & 0x7c000000u) == 0x7c000000u) {
                  w[e] &= 0x0000ffffu;
                  odd = true;
                }
              }
            }
            *reinterpret_cast<uint4*>(dst + to0 + step) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(dst + to1 + step) = make_uint4(w[4], w[5], w[6], w[7]);
          }
          if (odd) sm.odd_v[item & 3] = item + 1;  // at most two items ahead of the epilogue
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.wide_full[h & 1]);
            mbar_arrive(&sm.v_empty[slot]);
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int row = warp * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t o_tmem = tmem + 128 + lane_off;
    const float ninf = -__int_as_float(0x7f800000);
    const int g = row % a.group, ti = row / a.group;  // head of the group, token of the tile
    int h = 0;
    bool ok = !*abort;
    for (int item = 0; ok && wk.next(a, tile); ++item) {
      const int i = tile * a.tile_tokens + ti;  // token of the sequence
      const bool valid = ti < a.tile_tokens && i < wk.q.rows;
      const bool active = __any_sync(0xffffffffu, valid);
      const int hq = wk.hk_cur * a.group + g;
      float c = a.scale_log2;
      if constexpr (kFp8) c *= __ldg(a.q_scale + hq) * __ldg(a.k_scale + wk.hk_cur);
      c = logit_scale(c);
      float m_ref = ninf, l = 0.f;
      // the row's first mask words now, so that the item's last units do not wait for them
      uint64_t known = 0ull;
      const int words = a.mask == nullptr || !valid ? 0 : min(a.mask_words, 2);
      if (words > 0) {
        const uint32_t* row_words = a.mask + (static_cast<size_t>(wk.q.tok0) + i) * a.mask_words;
        known = __ldg(row_words);
        if (words > 1) known |= static_cast<uint64_t>(__ldg(row_words + 1)) << 32;
      }
#pragma unroll 1
      for (int u = wk.ub; u < wk.ue; ++u, ++h) {
        const int b = h & 1;
        const uint32_t s_tmem = tmem + kUnit * b + lane_off;
        const bool edge = (u + 1) * kUnit > wk.q.ctx;  // new tokens or the end of the keys
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.s_full[b], (h >> 1) & 1, abort, status))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (!kFp8 && edge) {
          // no NaN or infinity of V may meet a weight of zero
          const int slot = h % Cfg::kVSlots;
          if (!__all_sync(0xffffffffu, mbar_wait(&sm.v_full[slot], (h / Cfg::kVSlots) & 1, abort, status))) {
            ok = false;
            break;
          }
          const int r0 = max(wk.q.ctx - u * kUnit, 0), r1 = 16 * key_steps<kUnit, 16>(wk.q.kv, u);
          bool odd = false;
#pragma unroll 1
          for (int x = r0 * 16 + row; x < r1 * 16; x += 128) {  // 16-byte chunk x % 16 of row x / 16
            const int r = x >> 4;
            uint4* at = reinterpret_cast<uint4*>(sm.v[slot] + ((x >> 3) & 1) * (kUnit * 128) + r * 128 + (x & 7) * 16);
            uint4 w = *at;
            if (u * kUnit + r >= wk.q.kv) w = make_uint4(0u, 0u, 0u, 0u);
            w.x = finite_bf16x2(w.x, odd);
            w.y = finite_bf16x2(w.y, odd);
            w.z = finite_bf16x2(w.z, odd);
            w.w = finite_bf16x2(w.w, odd);
            *at = w;
          }
          if (odd) sm.odd_v[item & 3] = item + 1;
          fence_async_smem();
        }
        if (active) {
          const uint64_t see = !edge ? ~0ull : valid ? visible(a, wk.q, i, u * kUnit, known, words) : 0ull;
          // 32 keys at a time.  bf16: the scores stay in registers.  e4m3: they are
          // read again from TMEM, which keeps the code short enough for the
          // instruction cache that all roles share, and the threads at 96 registers.
          uint32_t rr[Cfg::kKeep ? 2 : 1][32];
          float top = ninf;
          if constexpr (Cfg::kKeep) {
            tmem_ld32(s_tmem, rr[0]);
            tmem_ld32(s_tmem + 32, rr[1]);
            tmem_ld_wait();
          }
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t(&x32)[32] = rr[Cfg::kKeep ? ch : 0];
            if constexpr (!Cfg::kKeep) {
              tmem_ld32(s_tmem + 32 * ch, x32);
              tmem_ld_wait();
            }
            if (edge) hide(x32, static_cast<uint32_t>(see >> (32 * ch)));
            float m4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              m4[e] = fmax3(__uint_as_float(x32[e * 8]), __uint_as_float(x32[e * 8 + 1]), __uint_as_float(x32[e * 8 + 2]));
#pragma unroll
            for (int x = 3; x < 7; x += 2)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                m4[e] = fmax3(m4[e], __uint_as_float(x32[e * 8 + x]), __uint_as_float(x32[e * 8 + x + 1]));
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], __uint_as_float(x32[e * 8 + 7]));
            top = fmaxf(top, fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3])));
          }
          const float m_cand = top == ninf ? ninf : fmaf(top, c, -Cfg::kBias);
          const bool need =
              valid && ((m_ref == ninf) ? (m_cand != ninf) : (m_cand > m_ref + Cfg::kSlack));
          if (__any_sync(0xffffffffu, need)) {
            const float m_new = valid && m_cand > m_ref ? m_cand : m_ref;  // O is read anyway: every row that grew
            const float alpha = (m_ref == ninf) ? 0.f : fast_exp2(m_ref - m_new);
            l *= alpha;
            if (u > wk.ub) {
              // O holds P V up to the unit before: let that product finish first
              if (!__all_sync(0xffffffffu,
                              mbar_wait(&sm.pv_done[b ^ 1], ((h - 1) >> 1) & 1, abort, status))) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll 1
              for (int ch = 0; ch < 4; ++ch) {
                uint32_t oo[32];
                tmem_ld32(o_tmem + ch * 32, oo);
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 32; ++x) oo[x] = __float_as_uint(__uint_as_float(oo[x]) * alpha);
                tmem_st32(o_tmem + ch * 32, oo);
              }
            }
            m_ref = m_new;
          }
          const float m_use = (m_ref == ninf) ? 0.f : m_ref;
          const float2 c2 = make_float2(c, c), nm2 = make_float2(-m_use, -m_use);
          float2 ps0 = make_float2(0.f, 0.f), ps1 = make_float2(0.f, 0.f);
#pragma unroll (Cfg::kKeep ? 2 : 1)
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t hi[16], lo[16];
            uint32_t(&x32)[32] = rr[Cfg::kKeep ? ch : 0];
            if constexpr (!Cfg::kKeep) {
              tmem_ld32(s_tmem + 32 * ch, x32);
              tmem_ld_wait();
              if (edge) hide(x32, static_cast<uint32_t>(see >> (32 * ch)));
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float2 e =
                  ffma2(make_float2(__uint_as_float(x32[2 * x]), __uint_as_float(x32[2 * x + 1])), c2, nm2);
              const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));
              if (x & 1) ps1 = fadd2(ps1, p);
              else ps0 = fadd2(ps0, p);
              if constexpr (kFp8) {
                hi[x] = f32x2_to_f16x2(p.x, p.y);
              } else {
                // hi: the largest bf16 below p (p (1 - 2^-24) rounds to the float before p),
                // so that both parts of a weight above zero are above zero and an
                // infinity of V stays one
                const float2 e = fmul2(p, make_float2(0.99999994f, 0.99999994f));
                const uint32_t e0 = __float_as_uint(e.x) & 0xffff0000u, e1 = __float_as_uint(e.y) & 0xffff0000u;
                hi[x] = __byte_perm(e0, e1, 0x7632);
                const float2 r = fsub2(p, make_float2(__uint_as_float(e0), __uint_as_float(e1)));
                lo[x] = pack_bf16x2(r.x, r.y);
              }
            }
            // P over the scores just read: bf16 in 32 columns (high, low parts), f16 in 16
            tmem_st16(s_tmem + (kFp8 ? 16 : 32) * ch, hi);
            if constexpr (!kFp8) tmem_st16(s_tmem + 32 * ch + 16, lo);
          }
          l += (ps0.x + ps0.y) + (ps1.x + ps1.y);
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[b]);
      }
      if (!ok) break;

      // ---- epilogue of the item: h - 1 is its last unit
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.pv_done[(h - 1) & 1], ((h - 1) >> 1) & 1, abort, status))) {
        ok = false;
        break;
      }
      tc_fence_after();
      // every sanitised V of the item is behind a wait of this thread, so the flag is seen
      const bool odd_v = *reinterpret_cast<volatile int*>(&sm.odd_v[item & 3]) == item + 1;
      if (active) {
        const size_t tok = static_cast<size_t>(wk.q.tok0) + i;
        const size_t part = static_cast<size_t>(blockIdx.x) * 2 + (wk.index > 1 ? 1 : 0);
        float inv = (l != 0.f) ? 1.f / l : 0.f;
        if constexpr (kFp8) inv *= __ldg(a.v_scale + wk.hk_cur);
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t rr[32];
          __syncwarp();
          tmem_ld32(o_tmem + ch * 32, rr);
          tmem_ld_wait();
          if (odd_v && valid) {
            // add the non-finite elements of V that this row does see
            for (int u = max(wk.ub, wk.q.ctx / kUnit); u < wk.ue; ++u) {
              uint64_t see = visible(a, wk.q, i, u * kUnit, known, words);
              for (; see != 0ull; see &= see - 1) {
                const int key = u * kUnit + __ffsll(static_cast<long long>(see)) - 1;
                if (key < wk.q.ctx) continue;
                const int pr = pool_row(a, wk.s, key);
                if (pr >= a.num_pages * a.page_size) continue;
                const uint8_t* v = a.v_pages + ((static_cast<size_t>(pr) * a.hkv + wk.hk_cur) * kHeadDim + ch * 32) *
                                                   (kFp8 ? 1 : 2);
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                  float e;
                  if constexpr (kFp8) e = (v[x] & 0x7f) == 0x7f ? __int_as_float(0x7fffffff) : 0.f;
                  else e = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(v)[x]) << 16);
                  if ((__float_as_uint(e) & 0x7f800000u) == 0x7f800000u)
                    rr[x] = __float_as_uint(__uint_as_float(rr[x]) + e);
                }
              }
            }
          }
          if (valid && wk.whole) {
            uint8_t* dst = static_cast<uint8_t*>(a.out) + ((tok * a.hq + hq) * static_cast<size_t>(kHeadDim) + ch * 32) * 2;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16x2(__uint_as_float(rr[q * 8 + 2 * e]) * inv,
                                   __uint_as_float(rr[q * 8 + 2 * e + 1]) * inv);
              reinterpret_cast<uint4*>(dst)[q] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (valid) {
            // dim by dim, so that a warp's 32 rows are one line
            float* dst = a.part_o + (part * kHeadDim + ch * 32) * a.part_rows + row;
#pragma unroll
            for (int x = 0; x < 32; ++x) dst[static_cast<size_t>(x) * a.part_rows] = __uint_as_float(rr[x]);
          }
        }
        if (valid) {
          if (wk.whole)
            a.lse[static_cast<size_t>(hq) * a.total_tokens + tok] =
                (l != 0.f) ? (m_ref + log2f(l)) * 0.69314718055994530942f : ninf;
          else
            a.part_ml[part * a.part_rows + row] = make_float2(m_ref, l);
        }
      }
      // the next item's first product into O waits for this warp's next P,
      // which comes after these reads
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) a.cta_status[blockIdx.x] = cta_word(sm.status, sm.range);
  if (warp == kMmaIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- joining the pieces of the items that were cut (blockIdx.y: item, that is
// sequence x KV head), in the order of the ranges

// The CTAs' status words become the call's, the smaller code if there are two.  One block.
__device__ __forceinline__ void reduce_status(const TreeArgs& a, int ctas) {
  __shared__ int sm_status;
  static_assert(STEM_ERR_TIMEOUT_CODE < STEM_ERR_BAD_INPUT_CODE, "a wait that ran out stands");
  constexpr int kNone = 0x7fffffff;
  if (threadIdx.x == 0) sm_status = kNone;
  __syncthreads();
  for (int i = threadIdx.x; i < ctas; i += blockDim.x) {
    const int st = a.cta_status[i];
    if (st != 0) atomicMin(&sm_status, st);
  }
  __syncthreads();
  if (threadIdx.x == 0) *a.status = sm_status == kNone ? 0 : sm_status;
}

struct Pieces {
  int s, hk;    // item
  int k0, k1;   // ranges that hold a unit of it
  int slot0;    // its slot in range k0: 0 when it is the first item there
};
// False when the item was not cut.
__device__ __forceinline__ bool find_pieces(const TreeArgs& a, int item, Pieces* p) {
  const int64_t total = a.unit0[a.seqs];
  const int used = ranges_used(a, total);
  p->s = item / a.hkv;
  p->hk = item % a.hkv;
  const int64_t at = a.unit0[p->s];
  const int64_t len = div_floor(a.unit0[p->s + 1] - at, a.hkv);  // of an item
  if (len == 0) return false;
  const int64_t begin = at + p->hk * len, first = begin + a.item_units, last = begin + len - 1;
  // the range that holds unit x: the largest k with range_begin(k) <= x
  p->k0 = static_cast<int>(div_floor((first + 1) * used - 1, total));
  p->k1 = static_cast<int>(div_floor((last + 1) * used - 1, total));
  p->slot0 = range_begin(total, used, p->k0) >= begin ? 0 : 1;
  return p->k0 != p->k1;
}

// Row-major pieces [rows][128] (narrow kernel).  A warp takes a row; rows of
// many pieces are taken by all warps of the block, every kJoinWarps-th piece each.
constexpr int kJoinWarps = 8;
constexpr int kJoinAlone = 8;  // pieces up to which a warp takes a row alone

__global__ void __launch_bounds__(kJoinWarps * 32)
    tree_join_rows_kernel(const __grid_constant__ TreeArgs a, int ctas, int rows_per_block) {
  __shared__ float sm_o[kJoinWarps][kHeadDim];
  __shared__ float sm_l[kJoinWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = warp_id(), lane = lane_id();
  if (blockIdx.x == 0 && blockIdx.y == 0) reduce_status(a, ctas);
  const float ninf = -__int_as_float(0x7f800000);
  for (int item = blockIdx.y; item < a.seqs * a.hkv; item += gridDim.y) {
    Pieces pc;
    if (!find_pieces(a, item, &pc)) continue;
    const int k0 = pc.k0, k1 = pc.k1, hk = pc.hk;
    const SeqShape q = seq_shape(a, pc.s);
    const bool together = k1 - k0 >= kJoinAlone;  // more pieces than that
    const int rows = min((static_cast<int>(blockIdx.x) + 1) * rows_per_block, q.rows * a.group);
    const float vscale = a.v_scale != nullptr ? __ldg(a.v_scale + hk) : 1.f;
    for (int r = blockIdx.x * rows_per_block + (together ? 0 : warp); r < rows; r += together ? 1 : kJoinWarps) {
      const int i = r / a.group;
      auto part = [&](int k) -> size_t { return (static_cast<size_t>(k) * 2 + (k == k0 ? pc.slot0 : 0)) * a.part_rows + r; };
      float m = ninf, m_use, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](float2 ml, float4 x) {
        if (ml.x == ninf) return;  // the row sees no key of the piece
        const float w = exp2f(ml.x - m_use);
        l += w * ml.y;
        o.x += w * x.x;
        o.y += w * x.y;
        o.z += w * x.z;
        o.w += w * x.w;
      };
      if (!together) {
        // every load of the row in flight at once
        float2 ml[kJoinAlone];
        float4 x[kJoinAlone];
#pragma unroll
        for (int j = 0; j < kJoinAlone; ++j) {
          ml[j] = make_float2(ninf, 0.f);
          if (k0 + j <= k1) {
            const size_t p = part(k0 + j);
            ml[j] = a.part_ml[p];
            x[j] = *reinterpret_cast<const float4*>(a.part_o + p * kHeadDim + lane * 4);
          }
        }
#pragma unroll
        for (int j = 0; j < kJoinAlone; ++j) m = fmaxf(m, ml[j].x);
        m_use = m == ninf ? 0.f : m;
#pragma unroll
        for (int j = 0; j < kJoinAlone; ++j) add(ml[j], x[j]);
      } else {
        for (int k = k0 + lane; k <= k1; k += 32) m = fmaxf(m, a.part_ml[part(k)].x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        m_use = m == ninf ? 0.f : m;
#pragma unroll 4
        for (int k = k0 + warp; k <= k1; k += kJoinWarps) {
          const size_t p = part(k);
          add(a.part_ml[p], *reinterpret_cast<const float4*>(a.part_o + p * kHeadDim + lane * 4));
        }
      }
      if (together) {
        *reinterpret_cast<float4*>(&sm_o[warp][lane * 4]) = o;
        if (lane == 0) sm_l[warp] = l;
        __syncthreads();
        if (warp == 0) {
          for (int w = 1; w < kJoinWarps; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(&sm_o[w][lane * 4]);
            l += sm_l[w];
            o.x += x.x;
            o.y += x.y;
            o.z += x.z;
            o.w += x.w;
          }
        }
        __syncthreads();
        if (warp != 0) continue;
      }
      const float inv = l != 0.f ? vscale / l : 0.f;
      const int h = hk * a.group + r % a.group;
      const size_t tok = static_cast<size_t>(q.tok0) + i;
      reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + (tok * a.hq + h) * static_cast<size_t>(kHeadDim) * 2)[lane] =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (lane == 0)
        a.lse[static_cast<size_t>(h) * a.total_tokens + tok] = l != 0.f ? (m_use + log2f(l)) * 0.69314718055994530942f : ninf;
    }
  }
}

// Dim-major pieces [128][rows] (wide kernel): a lane takes a row, a warp kCols
// dims of 32 rows.  blockIdx.x: tile, 32-row group of it and dims of the block.
template <int kCols>
__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_dims_kernel(const __grid_constant__ TreeArgs a, int ctas) {
  __shared__ float sm_w[kTreeRanges][32], sm_m[kJoinWarps][32], sm_l[kJoinWarps][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = warp_id(), lane = lane_id();
  if (blockIdx.x == 0 && blockIdx.y == 0) reduce_status(a, ctas);
  const float ninf = -__int_as_float(0x7f800000);
  constexpr int kParts = kHeadDim / (kCols * kJoinWarps);  // blocks that share the dims
  const int d0 = (static_cast<int>(blockIdx.x) % kParts * kJoinWarps + warp) * kCols;
  const int groups = a.part_rows / 32;
  const int row = static_cast<int>(blockIdx.x) / kParts % groups * 32 + lane;
  const int tile = static_cast<int>(blockIdx.x) / (kParts * groups);
  const int ti = row / a.group, i = tile * a.tile_tokens + ti;
  for (int item = blockIdx.y; item < a.seqs * a.hkv; item += gridDim.y) {
    Pieces pc;
    if (!find_pieces(a, item, &pc)) continue;
    const SeqShape q = seq_shape(a, pc.s);
    const bool valid = ti < a.tile_tokens && i < q.rows;
    if (!__any_sync(0xffffffffu, valid)) continue;
    auto part = [&](int k) -> size_t {
      return (static_cast<size_t>(k) * a.tiles + tile) * 2 + (k == pc.k0 ? pc.slot0 : 0);
    };
    // each warp takes every kJoinWarps-th piece's reference and sum; the weights go to SMEM
    const int n = pc.k1 - pc.k0 + 1;
    float m = ninf;
#pragma unroll 4
    for (int k = warp; k < n; k += kJoinWarps)
      if (valid) m = fmaxf(m, a.part_ml[part(pc.k0 + k) * a.part_rows + row].x);
    sm_m[warp][lane] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, sm_m[w][lane]);
    const float m_use = m == ninf ? 0.f : m;
    float l = 0.f;
#pragma unroll 4
    for (int k = warp; k < n; k += kJoinWarps) {
      if (valid) {
        const float2 ml = a.part_ml[part(pc.k0 + k) * a.part_rows + row];
        const float w = exp2f(ml.x - m_use);
        sm_w[k][lane] = ml.x == ninf ? -1.f : w;  // below 0: the row sees no key of the piece
        l += w * ml.y;
      }
    }
    sm_l[warp][lane] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) l += sm_l[w][lane];
    float o[kCols];
#pragma unroll
    for (int e = 0; e < kCols; ++e) o[e] = 0.f;
#pragma unroll (32 / kCols)
    for (int k = 0; k < n; ++k) {
      if (valid) {
        const float* src = a.part_o + (part(pc.k0 + k) * kHeadDim + d0) * a.part_rows + row;
        const float w = sm_w[k][lane];
#pragma unroll
        for (int e = 0; e < kCols; ++e) {
          const float x = src[static_cast<size_t>(e) * a.part_rows];
          if (!(w < 0.f)) o[e] += w * x;
        }
      }
    }
    __syncthreads();  // the next item writes the tables again
    if (!valid) continue;
    float inv = l != 0.f ? 1.f / l : 0.f;
    if (a.v_scale != nullptr) inv *= __ldg(a.v_scale + pc.hk);
    const int h = pc.hk * a.group + row % a.group;
    const size_t tok = static_cast<size_t>(q.tok0) + i;
    uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) +
                                          ((tok * a.hq + h) * static_cast<size_t>(kHeadDim) + d0) * 2);
#pragma unroll
    for (int e = 0; e < kCols; e += 4)
      dst[e / 4] = make_uint2(pack_bf16x2(o[e] * inv, o[e + 1] * inv), pack_bf16x2(o[e + 2] * inv, o[e + 3] * inv));
    if (d0 == 0)
      a.lse[static_cast<size_t>(h) * a.total_tokens + tok] = l != 0.f ? (m_use + log2f(l)) * 0.69314718055994530942f : ninf;
  }
}

template <bool kFp8>
static cudaError_t launch_tree_t(const TreeMaps& maps, const TreeArgs& args, cudaStream_t stream) {
  const size_t smem = sizeof(TreeSmem<kFp8>);
  static_assert(sizeof(TreeSmem<kFp8>) <= 115712, "two CTAs per SM");
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(tree_attn_kernel<kFp8>), smem, allowed);
  if (e != cudaSuccess) return e;
  const int grid = args.ranges * args.tiles;
  if (args.unit_keys == kUnit) {
    e = launch_after(tree_attn_kernel<kFp8>, dim3(grid), TreeCfg<kFp8>::kThreads, smem, stream, maps, args);
  } else {
    e = launch_tree_narrow(maps, args, kFp8, stream);
  }
  if (e != cudaSuccess) return e;
  TreeArgs j = args;
  if (!kFp8) j.v_scale = nullptr;
  const int most = args.max_seq_tokens < args.total_tokens ? args.max_seq_tokens : args.total_tokens;
  const int64_t items = static_cast<int64_t>(args.seqs) * args.hkv;
  const unsigned gy = static_cast<unsigned>(i64min(items, 65535));
  if (args.ranges == 1)  // one range holds everything: nothing is cut, only the status is left
    return launch_after(tree_join_rows_kernel, dim3(1), kJoinWarps * 32, 0, stream, j, grid, 0);
  if (args.unit_keys == kUnit) {
    // few items: more blocks, with fewer dims each (four 32-token trees over 4K: 34 us, with
    // 16 dims a warp 41)
    const int groups = args.tiles * (args.part_rows / 32);
    if (groups * items >= 4 * 148)
      return launch_after(tree_join_dims_kernel<16>, dim3(groups, gy), kJoinWarps * 32, 0, stream, j, grid);
    return launch_after(tree_join_dims_kernel<4>, dim3(groups * 4, gy), kJoinWarps * 32, 0, stream, j, grid);
  }
  // few rows in all: a block for each; else a row a warp
  const int rows = most * args.group;  // <= 32
  const int rows_per_block = rows * items <= 1024 ? 1 : kJoinWarps;
  return launch_after(tree_join_rows_kernel, dim3((rows + rows_per_block - 1) / rows_per_block, gy), kJoinWarps * 32, 0,
                      stream, j, grid, rows_per_block);
}

cudaError_t launch_tree_attn(const TreeMaps& maps, const TreeArgs& args, bool fp8, cudaStream_t stream) {
  return fp8 ? launch_tree_t<true>(maps, args, stream) : launch_tree_t<false>(maps, args, stream);
}

}  // namespace stem
