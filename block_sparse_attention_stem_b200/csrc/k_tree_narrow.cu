// k_tree_narrow.cu — attention over the paged cache for few query rows: single
// tokens and the smallest trees, at most 16 rows (tokens * query heads of a KV
// group) per sequence and KV head.
//
// The 128-row tile of the other kernel would be almost empty, and the tensor
// cores would spend the same time and power on it.  Here the products are
// turned round, so that the keys fill the 128 rows and the queries are the N
// columns:
//   S^T = K Q^T       128 keys x 16 rows, 8 steps (4 in e4m3)
//   P^T = exp2(..)    thread = key, one value per row, to SMEM as the B operand
//   O^T += V^T P^T    128 dims x (16 * terms), V^T read MN-major from the V tile
// The tensor cores are 4% busy where the 128-row tile kept them at 50%, which
// held the clock at 1.55 GHz under the power cap.
//
// Columns are cheap, so P is kept to more bits as several terms in columns of
// their own, added in the epilogue.  bf16: two (cut off below p, and the rest).
// e4m3: three, each the e4m3 of what is left, times 16 and 256, so V is used as
// it is and never widened.  With the largest weight at 2^5 that is 2^-12 p from
// 2^-6 on and 2^-18 below, too little for the many small weights beside an
// attention sink, so weights below 2^-8 go to three columns of their own, times
// 2^16: a weight is off by 2^-10 of itself at most down to 2^-29 of the row's
// largest (20 nats), and by 2^-39 of the largest below.  The second bank costs
// zeros (six byte stores per weight instead of three): none of it shows with 8
// rows (64 tokens over 1 to 8K keys 107.6 us with one bank or two), up to 9% with
// 16, where P takes the place of one K buffer: three tokens over 64K 38.2 against
// 35.0 us, sixteen 4-token trees over 16K 109 against 112 (in the 128-row kernel
// 60.9 and 125.9).
//
// No reduction across the keys while the reference holds: a thread keeps its
// key's share of every row's sum, and a value that passes the reference by more
// than 2^kSlack is noticed by one barrier with a vote, which the four softmax
// warps need anyway to agree on leaving.  Only then (always at an item's first
// unit) are the rows' maxima reduced and O scaled.  That code and the epilogue
// are rolled loops: unrolled, an item switch in mid-stream waited 30 us for
// instructions that the stream of keys had pushed out of L2 (which the keys'
// evict-first policy prevents too).
//
// Bound by HBM in bf16.  Measured: 16 tokens over 16K keys each (1.07 GB) 163 us,
// 6.59 TB/s (reads alone pass what a copy reaches); 64 over 1 to 8K 168 us; one over
// 128K (537 MB) 90 us.  e4m3: 64 over 1 to 8K (538 MB) 108 us, 5.0 TB/s, a unit's
// chain of waits.  Against 32 rows the 128-row kernel is faster (eight tokens of
// four heads over 16K: 185 against 211 us), since a thread's work grows with the
// rows.
//
// 192 threads; bf16: one CTA per SM (216 KB of SMEM, most of it K and V in
// flight); e4m3: two, because a unit's chain of waits (about 1300 cycles) is as
// long as HBM takes for its bytes:
//   warps 0-3 softmax and epilogue, warp 4 TMA producer, warp 5 MMA issuer.
#include "stem_tree_common.cuh"

namespace stem {

namespace {

constexpr int kUnit = 128;  // keys per tile
constexpr int kThreads = 192;
constexpr int kProducer = 4, kMmaIssuer = 5;
constexpr int kN = 16;  // query rows at most
constexpr int kQBufs = 2;
// e4m3 weights below kSmall go to a bank of terms of their own, times kUp
constexpr float kSmall = 0.00390625f, kUp = 65536.f;

// kRows: query rows at most
template <bool kFp8, int kRows>
struct NarrowCfg {
  static constexpr int kElt = kFp8 ? 1 : 2;
  static constexpr int kSlabs = kFp8 ? 1 : 2;          // 128-byte slabs of a head row
  static constexpr int kUnitBytes = kUnit * kHeadDim * kElt;
  static constexpr int kTerms = kFp8 ? 6 : 2;          // columns per row of P^T
  static constexpr int kPCols = kTerms * kRows;
  static constexpr int kStepKeys = kFp8 ? 32 : 16;     // keys per MMA of O^T
  static constexpr int kVSlots = 3;
  static constexpr int kKSlots = kFp8 && kRows > 8 ? 2 : 3;  // (P takes the third one's place)
  static constexpr int kCtas = kFp8 ? 2 : 1;           // per SM
  static constexpr int kQBytes = kN * kHeadDim * kElt;
  static constexpr int kPBytes = kPCols * kUnit * kElt;
  static constexpr uint32_t kOCol = 2 * kN;            // S buffers at 0 and kN
  static constexpr uint32_t kTmemCols = 128;
  // P may reach 2^(kBias + kSlack): e4m3 ends at 448
  static constexpr float kBias = kFp8 ? 5.f : 0.f;
  static constexpr float kSlack = kFp8 ? 3.75f : 8.f;
  static_assert(kPCols % 16 == 0 && kOCol + kPCols <= kTmemCols && kPBytes % 1024 == 0 && kPBytes >= kRows * kUnit * 4);
};

template <bool kFp8, int kRows>
struct NarrowSmem {
  using C = NarrowCfg<kFp8, kRows>;
  uint8_t k[C::kKSlots][C::kUnitBytes];  // 1024-aligned
  uint8_t v[C::kVSlots][C::kUnitBytes];
  uint8_t q[kQBufs][C::kQBytes];
  uint8_t p[2][C::kPBytes];
  uint64_t q_full[kQBufs], q_empty[kQBufs];
  uint64_t k_full[C::kKSlots], k_empty[C::kKSlots];
  uint64_t v_full[C::kVSlots], v_empty[C::kVSlots];
  uint64_t s_full[2];   // S^T_h complete
  uint64_t p_full[2];   // P^T_h stored (and O scaled)
  uint64_t pv_done[2];  // O += V^T_h P^T_h complete
  uint64_t drain;
  RangeScratch range;
  float red[4][kN];     // per softmax warp: row maxima, row sums
  uint32_t tmem_base;
  int status, abort;
  int odd_v[4];  // [item % 4]: item + 1 when a non-finite element of V was zeroed in it
};

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// True on all 128 threads of the softmax warps when it is on one of them.
__device__ __forceinline__ bool vote_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

// Maximum over the warp; NaN counts as nothing.
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint16_t v) {
  const uint32_t h = e4m3x2_to_f16x2(v);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace

template <bool kFp8, int kRows>
__global__ void __launch_bounds__(kThreads, NarrowCfg<kFp8, kRows>::kCtas)
    tree_narrow_kernel(const __grid_constant__ TreeMaps maps, const __grid_constant__ TreeArgs a) {
  using Cfg = NarrowCfg<kFp8, kRows>;
  using Smem = NarrowSmem<kFp8, kRows>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    sm.status = 0;
    sm.range.bad = 0;
    sm.abort = (smem_u32(smem_raw) & 1023u) != 0;  // the swizzled tiles need this alignment
    if (sm.abort) sm.status = STEM_ERR_TIMEOUT_CODE;
    for (int x = 0; x < 4; ++x) sm.odd_v[x] = 0;
  }
  // the barriers, a lane each, and the tensor maps' fetch, before earlier kernels are waited for
  constexpr int kBars = 2 * kQBufs + 2 * Cfg::kKSlots + 2 * Cfg::kVSlots + 7;
  static_assert(offsetof(Smem, drain) == offsetof(Smem, q_full) + (kBars - 1) * 8, "barriers in a row");
  if (warp == kMmaIssuer && lane < kBars) {
    uint64_t* bar = &sm.q_full[0] + lane;
    mbar_init(bar, bar == &sm.p_full[0] || bar == &sm.p_full[1] ? 4 : 1);
    fence_mbar_init();
  }
  if (warp == kProducer && lane < 3) tma_prefetch_desc(lane == 0 ? &maps.k_pool : lane == 1 ? &maps.q : &maps.v_pool);
  const int64_t count = find_range<kThreads>(a, blockIdx.x, sm.range);
  if (count == 0) {
    __syncthreads();
    if (threadIdx.x == 0) a.cta_status[blockIdx.x] = cta_word(sm.status, sm.range);
    return;
  }
  if (warp == kMmaIssuer) {
    tmem_alloc(&sm.tmem_base, Cfg::kTmemCols);
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

  if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    // Lane 0 issues; the warp looks up the pages of 16 units (32 half units of
    // 64 keys, which never straddle a page) at a time.  K runs up to `ahead`
    // units before V: while V_h is the next V, the products up to S_{h+1} can
    // complete, and the Q tile of K_{h+ahead-1} may have to wait for
    // S_{h+ahead-1-kQBufs} (items of one unit): ahead <= 2 + kQBufs.
    constexpr int kAhead = Cfg::kKSlots < 2 + kQBufs ? Cfg::kKSlots : 2 + kQBufs;
    struct Stream {
      Walk w;
      int u, rows, h, slot, round;
      bool more;
    };
    Stream ks{wk, 0, 0, 0, 0, 0, false}, vs{wk, 0, 0, 0, 0, 0, false};
    const uint64_t policy = evict_first_policy();  // a key is read once: leave L2 to code, pages and pieces
    int item = 0;  // Q tiles issued
    bool ok = !*abort;
    auto enter = [&](Stream& st) {
      st.more = st.w.next(a, 0);
      if (st.more) st.u = st.w.ub;
    };
    // issues the stream's next unit; false when a wait ran out
    auto load = [&](Stream& st, const CUtensorMap* m, uint8_t* base, uint64_t* full, uint64_t* empty, int slots) -> bool {
      const int x = ((st.u - st.w.ub) & 15) * 2;
      if (x == 0) {
        // halves behind the last key read zeros, not memory
        const int key0 = st.u * kUnit;  // (a key behind the last one may not fit 32 bits)
        st.rows = lane * 64 < st.w.q.kv - key0 ? pool_row(a, st.w.s, key0 + lane * 64) : a.num_pages * a.page_size;
      }
      const int row0 = __shfl_sync(0xffffffffu, st.rows, x), row1 = __shfl_sync(0xffffffffu, st.rows, x + 1);
      bool good = true;
      if (lane == 0) {
        if (st.round > 0) good = mbar_wait(&empty[st.slot], (st.round - 1) & 1, abort, status);
        if (good) {
          mbar_arrive_expect_tx(&full[st.slot], Cfg::kUnitBytes);
          for (int y = 0; y < Cfg::kSlabs; ++y) {
            uint8_t* dst = base + st.slot * Cfg::kUnitBytes + y * (kUnit * 128);
            tma_load_3d_hint(dst, m, &full[st.slot], y * 64, st.w.hk_cur, row0, policy);
            tma_load_3d_hint(dst + 64 * 128, m, &full[st.slot], y * 64, st.w.hk_cur, row1, policy);
          }
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
          const int b = item % kQBufs;
          if (item >= kQBufs) good = mbar_wait(&sm.q_empty[b], (item / kQBufs - 1) & 1, abort, status);
          if (good) {
            mbar_arrive_expect_tx(&sm.q_full[b], a.box_rows * 128 * Cfg::kSlabs);
            for (int x = 0; x < Cfg::kSlabs; ++x)
              tma_load_3d(sm.q[b] + x * (kN * 128), &maps.q, &sm.q_full[b], x * 64, ks.w.hk_cur * a.group, ks.w.q.tok0);
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
    for (int x = 0; x < kAhead && ok && ks.more; ++x) ok = load_k();
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
      quiesce(sm.q_full, kQBufs, item);
    }
    __syncwarp();
  } else if (warp == kMmaIssuer) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      const uint32_t fmt = kFp8 ? 0u : 1u;  // e4m3 (kind::f8f6f4) or bf16 (kind::f16)
      const uint32_t idesc_s = make_idesc(fmt, 0u, 128u, static_cast<uint32_t>(kN));
      const uint32_t idesc_o = make_idesc(fmt, 0u, 128u, static_cast<uint32_t>(Cfg::kPCols)) | (1u << 15);  // A MN-major
      const uint32_t o_tmem = tmem + Cfg::kOCol;
      // two walks: S runs two units ahead of O
      Walk ws = wk;
      int hs = 0, us = 0, qitem = -1;
      bool more_s = ws.next(a, 0);
      if (more_s) us = ws.ub;
      auto issue_s = [&]() -> bool {
        if (us == ws.ub) {
          ++qitem;
          if (!mbar_wait(&sm.q_full[qitem % kQBufs], (qitem / kQBufs) & 1, abort, status)) return false;
        }
        const int slot = hs % Cfg::kKSlots;
        if (!mbar_wait(&sm.k_full[slot], (hs / Cfg::kKSlots) & 1, abort, status)) return false;
        tc_fence_after();
        // descriptors count 16-byte units
        const uint64_t dq = make_sdesc_sw128(smem_u32(sm.q[qitem % kQBufs]), 16, 1024);
        const uint64_t dk = make_sdesc_sw128(smem_u32(sm.k[slot]), 16, 1024);
        const uint32_t d = tmem + kN * (hs & 1);
        if constexpr (kFp8) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 32 dims per step
            mma_f8_ss(d, dk + kk * 2, dq + kk * 2, idesc_s, kk != 0);
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // 16 dims per step
            mma_bf16_ss(d, dk + (kk >> 2) * (kUnit * 8) + (kk & 3) * 2, dq + (kk >> 2) * (kN * 8) + (kk & 3) * 2, idesc_s,
                        kk != 0);
        }
        mma_commit(&sm.k_empty[slot]);
        mma_commit(&sm.s_full[hs & 1]);
        ++hs;
        if (++us == ws.ue) {
          mma_commit(&sm.q_empty[qitem % kQBufs]);
          more_s = ws.next(a, 0);
          if (more_s) us = ws.ub;
        }
        return true;
      };
      bool ok = !*abort;
      for (int x = 0; x < 2 && ok && more_s; ++x) ok = issue_s();
      int h = 0;
      while (ok && wk.next(a, 0)) {
        for (int u = wk.ub; u < wk.ue && ok; ++u, ++h) {
          const int slot = h % Cfg::kVSlots;
          ok = mbar_wait(&sm.p_full[h & 1], (h >> 1) & 1, abort, status) &&
               mbar_wait(&sm.v_full[slot], (h / Cfg::kVSlots) & 1, abort, status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv = make_sdesc_sw128(smem_u32(sm.v[slot]), kUnit * 128, 1024);
          const uint64_t dp = make_sdesc_sw128(smem_u32(sm.p[h & 1]), 16, 1024);
          const int steps = key_steps<kUnit, Cfg::kStepKeys>(wk.q.kv, u);
          if constexpr (kFp8) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 32 keys per step
              if (kk < steps) mma_f8_ss(o_tmem, dv + kk * 256, dp + kk * 2, idesc_o, u != wk.ub || kk != 0);
          } else {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)  // 16 keys per step
              if (kk < steps)
                mma_bf16_ss(o_tmem, dv + kk * 128, dp + (kk >> 2) * (Cfg::kPCols * 8) + (kk & 3) * 2, idesc_o,
                            u != wk.ub || kk != 0);
          }
          mma_commit(&sm.v_empty[slot]);
          mma_commit(&sm.pv_done[h & 1]);
          if (more_s) ok = issue_s();
        }
      }
      mma_commit(&sm.drain);
      mbar_wait_quiesce(&sm.drain, 0, status);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int kx = warp * 32 + lane;  // key of the unit; dim of the head in the epilogue
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t o_tmem = tmem + Cfg::kOCol + lane_off;
    const float ninf = -__int_as_float(0x7f800000);
    // where this key's values go in a row of P^T (row r: 128 r bytes further, chunk ^ r % 8)
    const uint32_t pchunk = kFp8 ? static_cast<uint32_t>(kx >> 4) << 4 : static_cast<uint32_t>((kx & 63) >> 3) << 4;
    const uint32_t pbyte = kFp8 ? static_cast<uint32_t>(kx & 15)
                                : static_cast<uint32_t>(kx >> 6) * (Cfg::kPCols * 128) + (kx & 7) * 2;
    int h = 0;
    bool ok = !*abort;
    ok = !vote_any(!ok);
    for (int item = 0; ok && wk.next(a, 0); ++item) {
      const int rows = wk.q.rows * a.group;
      // per row: scale (e4m3: with the head's), reference less kBias, this key lane's share of the sum
      float c[kFp8 ? kRows : 1], m[kRows], l[kRows];
      float c_lane = a.scale_log2;  // row `lane`'s scale
      if constexpr (!kFp8) {
        c_lane = logit_scale(c_lane);
        c[0] = c_lane;
      } else {
        if (lane < rows)
          c_lane *= __ldg(a.q_scale + wk.hk_cur * a.group + lane % a.group) * __ldg(a.k_scale + wk.hk_cur);
        c_lane = logit_scale(c_lane);
#pragma unroll
        for (int r = 0; r < kRows; ++r) c[r] = __shfl_sync(0xffffffffu, c_lane, r);
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) m[r] = l[r] = 0.f;
      float ref = 0.f;   // row `lane`: the same as m[lane]
      bool set = false;  // row `lane` has a reference
#pragma unroll 1
      for (int u = wk.ub; u < wk.ue; ++u, ++h) {
        const int b = h & 1;
        const bool edge = (u + 1) * kUnit > wk.q.ctx;  // new tokens or the end of the keys
        bool good = mbar_wait(&sm.s_full[b], (h >> 1) & 1, abort, status);
        const int key = u * kUnit + kx;
        if (edge) {
          // no NaN or infinity of V may meet a weight of zero
          const int slot = h % Cfg::kVSlots;
          good = good && mbar_wait(&sm.v_full[slot], (h / Cfg::kVSlots) & 1, abort, status);
          if (good) {
            const int r0 = max(wk.q.ctx - u * kUnit, 0), r1 = Cfg::kStepKeys * key_steps<kUnit, Cfg::kStepKeys>(wk.q.kv, u);
            bool odd = false;
#pragma unroll 1
            for (int x = r0 * 8 * Cfg::kSlabs + kx; x < r1 * 8 * Cfg::kSlabs; x += 128) {
              // 16-byte chunk x of rows r0 .. r1 - 1, slab by slab of a row
              const int row = x / (8 * Cfg::kSlabs), chunk = x % (8 * Cfg::kSlabs);
              const int at_key = u * kUnit + row;
              uint4* at = reinterpret_cast<uint4*>(sm.v[slot] + (chunk >> 3) * (kUnit * 128) + row * 128 + (chunk & 7) * 16);
              uint4 w = *at;
              if (at_key >= wk.q.kv) w = make_uint4(0u, 0u, 0u, 0u);
              if constexpr (kFp8) {
                uint32_t* e = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  // bytes 0x7f and 0xff are the NaNs
                  const uint32_t nan = __vcmpeq4(e[y] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                  odd |= nan != 0;
                  e[y] &= ~nan;
                }
              } else {
                w.x = finite_bf16x2(w.x, odd);
                w.y = finite_bf16x2(w.y, odd);
                w.z = finite_bf16x2(w.z, odd);
                w.w = finite_bf16x2(w.w, odd);
              }
              *at = w;
            }
            if (odd) sm.odd_v[item & 3] = item + 1;
          }
        }
        __syncwarp();
        tc_fence_after();
        uint32_t s[kRows];
        if constexpr (kRows == 8) tmem_ld8(tmem + kN * b + lane_off, s);
        else tmem_ld16(tmem + kN * b + lane_off, s);
        tmem_ld_wait();
        uint32_t see = 0xffffffffu;  // rows that see this key
        if (edge) {
          if (key >= wk.q.ctx) {
            const int d = key - wk.q.ctx;  // index among the new tokens
            const uint32_t head_bits = 0xffffffffu >> (32 - a.group);
            see = 0u;
            if (key < wk.q.kv && (a.mask == nullptr || (d >> 5) < a.mask_words)) {
              const uint32_t* word = a.mask + static_cast<size_t>(wk.q.tok0) * a.mask_words + (d >> 5);
#pragma unroll 1
              for (int i = 0; i < wk.q.rows; ++i, word += a.mask_words)
                if (a.mask == nullptr ? d <= i : (__ldg(word) >> (d & 31)) & 1u) see |= head_bits << (i * a.group);
            }
          }
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            if (!((see >> r) & 1u)) s[r] = 0xff800000u;  // -inf
        }
        // t = s c - m; does a row pass its reference by more than the slack?
        float t[kRows], top = ninf;
#pragma unroll
        for (int r = 0; r < kRows; r += 4) {
          if (r < rows) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              t[r + e] = fmaf(__uint_as_float(s[r + e]), c[kFp8 ? r + e : 0], -m[r + e]);
              if (r + e < rows) top = fmaxf(top, t[r + e]);
            }
          }
        }
        const bool unset = lane < rows && !set;
        const bool move = !good || top > Cfg::kSlack + Cfg::kBias || ((edge || u == wk.ub) && unset);
        if (vote_any(move)) {
          // ---- new references: the rows' maxima over the unit's keys.  Lane r of
          // every warp decides for row r.  (Rare code that may have left every
          // cache by the time it is needed: kept short.)
          if (vote_any(!good)) {
            ok = false;
            break;
          }
          float peak = ninf;
#pragma unroll 1
          for (int r = 0; r < rows; ++r) {
            uint32_t x;  // again from TMEM: registers cannot be indexed
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(tmem + kN * b + lane_off + r));
            tmem_ld_wait();
            const float cr = kFp8 ? __shfl_sync(0xffffffffu, c_lane, r) : c_lane;
            const float y = warp_max((see >> r) & 1u ? __uint_as_float(x) * cr : ninf);
            if (lane == r) peak = y;
          }
          if (lane < rows) sm.red[warp][lane] = peak;
          vote_any(false);
          float alpha = 1.f;
          bool scale = false;
          if (lane < rows) {
            const float x = fmaxf(fmaxf(sm.red[0][lane], sm.red[1][lane]), fmaxf(sm.red[2][lane], sm.red[3][lane]));
            if (set ? x > ref + Cfg::kSlack + Cfg::kBias : x != ninf) {
              scale = set;
              if (set) alpha = fast_exp2(ref - (x - Cfg::kBias));
              ref = x - Cfg::kBias;
              set = true;
            }
            set |= !edge;  // keys that are all seen but have no finite logit: reference 0
          }
          bool fine = true;
          if (u > wk.ub && __any_sync(0xffffffffu, scale)) {
            // O holds the products up to the unit before: let them finish first
            fine = __all_sync(0xffffffffu, mbar_wait(&sm.pv_done[b ^ 1], ((h - 1) >> 1) & 1, abort, status));
            tc_fence_after();
            if (fine) {
#pragma unroll 1
              for (int n = 0; n < Cfg::kPCols; ++n) {
                const float f = __shfl_sync(0xffffffffu, alpha, n % kRows);
                uint32_t o;
                asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(o) : "r"(o_tmem + n));
                tmem_ld_wait();
                o = __float_as_uint(__uint_as_float(o) * f);
                asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(o_tmem + n), "r"(o) : "memory");
              }
              tmem_st_wait();
            }
          }
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            if (r < rows) {
              m[r] = __shfl_sync(0xffffffffu, ref, r);
              l[r] *= __shfl_sync(0xffffffffu, alpha, r);
              t[r] = fmaf(__uint_as_float(s[r]), c[kFp8 ? r : 0], -m[r]);
            }
          }
          if (vote_any(!fine)) {  // also: every thread has read red
            ok = false;
            break;
          }
        }
        // ---- weights, their share of the sums, and their terms to SMEM
        uint8_t* prow = sm.p[b] + pbyte;
#pragma unroll
        for (int r = 0; r < kRows; r += 2) {
          if (r < rows) {
            const float2 p = make_float2(fast_exp2(t[r]), r + 1 < rows ? fast_exp2(t[r + 1]) : 0.f);
            l[r] += p.x;
            l[r + 1] += p.y;
            auto at = [&](int n) -> uint8_t* { return prow + n * 128 + (pchunk ^ ((n & 7) << 4)); };
            if constexpr (kFp8) {
              // three terms in one of two banks of columns, zeros in the other
              constexpr int kTerm = kRows * 128, kBank = 3 * kTerm;  // bytes
              const bool s0 = p.x < kSmall, s1 = p.y < kSmall;
              uint8_t *in0 = at(r) + (s0 ? kBank : 0), *no0 = at(r) + (s0 ? 0 : kBank);
              uint8_t *in1 = at(r + 1) + (s1 ? kBank : 0), *no1 = at(r + 1) + (s1 ? 0 : kBank);
              float2 left = fmul2(p, make_float2(s0 ? kUp : 1.f, s1 ? kUp : 1.f));
#pragma unroll
              for (int e = 0; e < 3; ++e) {
                const uint16_t w = to_e4m3x2(left.x, left.y);
                in0[e * kTerm] = static_cast<uint8_t>(w);
                in1[e * kTerm] = static_cast<uint8_t>(w >> 8);
                no0[e * kTerm] = 0;
                no1[e * kTerm] = 0;
                if (e < 2) left = fmul2(fsub2(left, from_e4m3x2(w)), make_float2(16.f, 16.f));
              }
            } else {
              // the largest bf16 below p (p (1 - 2^-24) rounds to the float before p), so
              // that both terms of a weight above zero are above zero and an infinity of
              // V stays one
              const float2 e = fmul2(p, make_float2(0.99999994f, 0.99999994f));
              const uint32_t e0 = __float_as_uint(e.x) & 0xffff0000u, e1 = __float_as_uint(e.y) & 0xffff0000u;
              const uint32_t lo = pack_bf16x2(p.x - __uint_as_float(e0), p.y - __uint_as_float(e1));
              *reinterpret_cast<uint16_t*>(at(r)) = static_cast<uint16_t>(e0 >> 16);
              *reinterpret_cast<uint16_t*>(at(r + 1)) = static_cast<uint16_t>(e1 >> 16);
              *reinterpret_cast<uint16_t*>(at(kRows + r)) = static_cast<uint16_t>(lo);
              *reinterpret_cast<uint16_t*>(at(kRows + r + 1)) = static_cast<uint16_t>(lo >> 16);
            }
          }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[b]);
      }
      if (!ok) break;

      // ---- epilogue of the item: h - 1 is its last unit
      const bool good = mbar_wait(&sm.pv_done[(h - 1) & 1], ((h - 1) >> 1) & 1, abort, status);
      if (vote_any(!good)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // the sums: every thread's shares to SMEM (P is free: its products are
      // done), then one warp adds the 128 of a row
      float* share = reinterpret_cast<float*>(sm.p[0]);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (r < rows) share[r * 128 + kx] = l[r];
      vote_any(false);
#pragma unroll 1
      for (int r = warp; r < rows; r += 4) {
        float x = (share[r * 128 + lane] + share[r * 128 + 32 + lane]) +
                  (share[r * 128 + 64 + lane] + share[r * 128 + 96 + lane]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (lane == 0) sm.red[0][r] = x;
      }
      vote_any(false);
      const bool odd_v = *reinterpret_cast<volatile int*>(&sm.odd_v[item & 3]) == item + 1;
      const size_t part = (static_cast<size_t>(blockIdx.x) * 2 + (wk.index > 1 ? 1 : 0)) * a.part_rows;
      const float vscale = kFp8 ? __ldg(a.v_scale + wk.hk_cur) : 1.f;
      int i = 0, g = 0;  // token of the sequence and head of the group of row r
#pragma unroll 1
      for (int r = 0; r < rows; ++r) {
        uint32_t o[Cfg::kTerms];
#pragma unroll
        for (int e = 0; e < Cfg::kTerms; ++e)
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(o[e]) : "r"(o_tmem + e * kRows + r));
        tmem_ld_wait();
        float acc = __uint_as_float(o[0]);
        if constexpr (kFp8)
          acc += __uint_as_float(o[1]) * 0.0625f + __uint_as_float(o[2]) * 0.00390625f +
                 (__uint_as_float(o[3]) + __uint_as_float(o[4]) * 0.0625f + __uint_as_float(o[5]) * 0.00390625f) * (1.f / kUp);
        else
          acc += __uint_as_float(o[1]);
        if (odd_v) {
          // add the non-finite elements of V that this row does see
#pragma unroll 1
          for (int key = max(wk.ub * kUnit, wk.q.ctx); key < min(wk.ue * kUnit, wk.q.kv); ++key) {
            if (!(visible(a, wk.q, i, key, 0ull, 0) & 1ull)) continue;
            const int pr = pool_row(a, wk.s, key);
            if (pr >= a.num_pages * a.page_size) continue;
            const size_t at = (static_cast<size_t>(pr) * a.hkv + wk.hk_cur) * kHeadDim + kx;
            float e;
            if constexpr (kFp8) e = (a.v_pages[at] & 0x7f) == 0x7f ? __int_as_float(0x7fffffff) : 0.f;
            else e = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(a.v_pages)[at]) << 16);
            if ((__float_as_uint(e) & 0x7f800000u) == 0x7f800000u) acc += e;
          }
        }
        const float sum = sm.red[0][r];
        float mr = __shfl_sync(0xffffffffu, ref, r);
        if (sum == 0.f) mr = ninf;
        if (wk.whole) {
          const size_t tok = static_cast<size_t>(wk.q.tok0) + i;
          const int hq = wk.hk_cur * a.group + g;
          const float inv = sum != 0.f ? vscale / sum : 0.f;
          reinterpret_cast<uint16_t*>(a.out)[(tok * a.hq + hq) * kHeadDim + kx] =
              static_cast<uint16_t>(pack_bf16x2(acc * inv, 0.f));
          if (kx == 0)
            a.lse[static_cast<size_t>(hq) * a.total_tokens + tok] =
                sum != 0.f ? (mr + log2f(sum)) * 0.69314718055994530942f : ninf;
        } else {
          a.part_o[(part + r) * kHeadDim + kx] = acc;
          if (kx == 0) a.part_ml[part + r] = make_float2(mr, sum);
        }
        if (++g == a.group) {
          g = 0;
          ++i;
        }
      }
      // the next item's first product into O waits for this warp's next P, which
      // comes after these reads; red is free again after the next vote
      tc_fence_before();
      vote_any(false);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) a.cta_status[blockIdx.x] = cta_word(sm.status, sm.range);
  if (warp == kMmaIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

template <bool kFp8, int kRows>
static cudaError_t launch_narrow_t(const TreeMaps& maps, const TreeArgs& args, cudaStream_t stream) {
  const size_t smem = sizeof(NarrowSmem<kFp8, kRows>);
  static_assert(sizeof(NarrowSmem<kFp8, kRows>) <= (kFp8 ? 115712 : 232448), "CTAs per SM");
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(tree_narrow_kernel<kFp8, kRows>), smem, allowed);
  if (e != cudaSuccess) return e;
  return launch_after(tree_narrow_kernel<kFp8, kRows>, dim3(args.ranges), kThreads, smem, stream, maps, args);
}

cudaError_t launch_tree_narrow(const TreeMaps& maps, const TreeArgs& args, bool fp8, cudaStream_t stream) {
  if (!fp8) return launch_narrow_t<false, 16>(maps, args, stream);
  return args.box_rows <= 8 ? launch_narrow_t<true, 8>(maps, args, stream) : launch_narrow_t<true, 16>(maps, args, stream);
}

}  // namespace stem
