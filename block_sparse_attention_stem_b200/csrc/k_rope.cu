// k_rope.cu — rotary positions for q and k, and a step's K and V into the
// paged cache, in one pass over the projection's rows.
//
// Angle: pair j turns by p w_j at position p.  Only the fraction of a turn
// matters, so w_j is kept as a 64-bit integer in units of 2^-64 turns and the
// product p w_j is taken modulo 2^64: the reduction is exact for every int32
// position, where p w_j in fp32 would be off by 2^-24 of up to 10^6 radians.
// The top 32 bits, as a signed number of 2^-31 half turns, go to sincospif;
// what is left out is below 2^-25 half turns.  No table, nothing to keep.
//
// Eight lanes own one head row, lane u the 16 elements of "unit" u as two
// 16-byte vectors: unit u < r/16 holds eight whole pairs (HALF: vectors u and
// u + r/16; INTERLEAVED: 2u and 2u + 1), the other units are copied.  A warp
// works on one token, four heads at a time; a lane's eight sines and cosines
// serve every head of the token.  The kernel moves each byte once and is bound
// by HBM as long as its instructions keep up, so q, k and v are loops of their
// own with pointers that step, pairs are rotated two at a time in packed fp32,
// and the reciprocal scales come from SMEM.  The loads in flight are those of
// many warps: four blocks of 256 threads per SM at 64 registers and one row at a
// time per lane measured 134 us (32K tokens, bf16) and 323 us (96K, e4m3), two or
// four rows at a time with fewer warps 144 to 157 and 392 to 530 us.
#include <algorithm>

#include "stem_device.cuh"
#include "stem_kernels.h"

namespace stem {

namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Elements 2i and 2i + 1 of eight bf16.
__device__ __forceinline__ void unpack8(const uint4& v, float2 (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

// Eight values to their place: 16 bytes of bf16, or 8 of e4m3 after scaling.
template <bool kFp8>
__device__ __forceinline__ void store8(uint8_t* dst, const float2 (&x)[4], float2 inv_scale) {
  if constexpr (kFp8) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = fmul2(x[2 * i], inv_scale), b = fmul2(x[2 * i + 1], inv_scale);
      w[i] = static_cast<uint32_t>(e4m3x2(a.x, a.y)) | static_cast<uint32_t>(e4m3x2(b.x, b.y)) << 16;
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                                                pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
  }
}

// What a lane needs of its unit.
struct Unit {
  int va, vb;            // its two vectors (of 8 elements) inside a head row
  bool rot;              // it holds pairs
  float2 cs[4], sn[4];   // HALF: pairs 2i, 2i + 1; INTERLEAVED: one pair each, see rotate
};

// HALF: a[i], b[i] are the first and second elements of pairs 2i and 2i + 1.
// INTERLEAVED: a[i] is pair i and b[i] pair 4 + i, as (first, second).
template <bool kInterleaved>
__device__ __forceinline__ void rotate(float2 (&a)[4], float2 (&b)[4], const Unit& un) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kInterleaved) {
      const float ca = un.cs[i].x, sa = un.sn[i].x, cb = un.cs[i].y, sb = un.sn[i].y;
      a[i] = ffma2(make_float2(a[i].y, a[i].x), make_float2(-sa, sa), fmul2(a[i], make_float2(ca, ca)));
      b[i] = ffma2(make_float2(b[i].y, b[i].x), make_float2(-sb, sb), fmul2(b[i], make_float2(cb, cb)));
    } else {
      const float2 x = a[i], y = b[i];
      a[i] = ffma2(y, make_float2(-un.sn[i].x, -un.sn[i].y), fmul2(x, un.cs[i]));
      b[i] = ffma2(x, un.sn[i], fmul2(y, un.cs[i]));
    }
  }
}

// The heads first, first + step, .. of one tensor of a token: rotated (kRotate)
// and stored to a packed row and a row of the pool, either may be null.  src,
// packed and pool point at head 0.
template <bool kRotate, bool kInterleaved, bool kFp8>
__device__ __forceinline__ void rope_heads(const Unit& un, const uint8_t* src, int heads, int first, int step,
                                           uint8_t* packed, uint8_t* pool, const float* inv_scale) {
  constexpr int kElt = kFp8 ? 1 : 2;
  constexpr int kRow = kHeadDim * kElt;  // bytes of an output head row
  const bool rot = kRotate && un.rot;
  for (int h = first; h < heads; h += step) {
    const uint8_t* row = src + static_cast<size_t>(h) * (kHeadDim * 2);
    const uint4 va = *reinterpret_cast<const uint4*>(row + un.va * 16);
    const uint4 vb = *reinterpret_cast<const uint4*>(row + un.vb * 16);
    const size_t at = static_cast<size_t>(h) * kRow;
    if (!kFp8 && !rot) {
      // bf16 rows that are not rotated keep their bits (a NaN's payload too)
      if (packed) {
        *reinterpret_cast<uint4*>(packed + at + un.va * 16) = va;
        *reinterpret_cast<uint4*>(packed + at + un.vb * 16) = vb;
      }
      if (pool) {
        *reinterpret_cast<uint4*>(pool + at + un.va * 16) = va;
        *reinterpret_cast<uint4*>(pool + at + un.vb * 16) = vb;
      }
    } else {
      float2 a[4], b[4], inv = make_float2(1.f, 1.f);
      unpack8(va, a);
      unpack8(vb, b);
      if (rot) rotate<kInterleaved>(a, b, un);
      if constexpr (kFp8) inv.x = inv.y = inv_scale[h];
      if (packed) {
        store8<kFp8>(packed + at + un.va * 8 * kElt, a, inv);
        store8<kFp8>(packed + at + un.vb * 8 * kElt, b, inv);
      }
      if (pool) {
        store8<kFp8>(pool + at + un.va * 8 * kElt, a, inv);
        store8<kFp8>(pool + at + un.vb * 8 * kElt, b, inv);
      }
    }
  }
}

}  // namespace

// grid: x = groups of 8 tokens (a warp each), y = splits of a token's heads
template <bool kInterleaved, bool kFp8>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float inv_scale[];  // e4m3: reciprocals, q then k then v heads
  const int lane = lane_id();
  if constexpr (kFp8) {
    for (int i = threadIdx.x; i < a.hq + a.hkv + a.hv; i += kRopeThreads) {
      const float* s = i < a.hq ? a.q_scale + i : i < a.hq + a.hkv ? a.k_scale + (i - a.hq) : a.v_scale + (i - a.hq - a.hkv);
      inv_scale[i] = 1.f / __ldg(s);
    }
    __syncthreads();
  }
  const int u = lane & 7;
  const int units = a.rotary_dim >> 4;  // units that rotate
  Unit un;
  un.rot = u < units;
  un.va = kInterleaved || !un.rot ? 2 * u : u;
  un.vb = kInterleaved || !un.rot ? 2 * u + 1 : u + units;
  const int first = blockIdx.y * 4 + (lane >> 3), step = gridDim.y * 4;
  const size_t row = kHeadDim * (kFp8 ? 1 : 2);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + warp_id(); t < a.tokens;
       t += static_cast<int64_t>(gridDim.x) * (kRopeThreads / 32)) {
    if (un.rot) {
      const int64_t p = __ldg(a.positions + t);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t phase = static_cast<uint64_t>(p) * a.turn[8 * u + i];
        float s, c;
        sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);
        s *= a.amplitude;
        c *= a.amplitude;
        // HALF: pairs 2j and 2j + 1 together; INTERLEAVED: pairs j and 4 + j
        const int j = kInterleaved ? i & 3 : i >> 1;
        if (kInterleaved ? i < 4 : (i & 1) == 0) {
          un.cs[j].x = c;
          un.sn[j].x = s;
        } else {
          un.cs[j].y = c;
          un.sn[j].y = s;
        }
      }
    }
    if (a.hq > 0)
      rope_heads<true, kInterleaved, kFp8>(un, a.q + t * a.q_stride, a.hq, first, step, a.q_out + t * a.hq * row, nullptr,
                                           inv_scale);
    int64_t slot = -1;
    if (a.k_pages != nullptr) {
      const int sl = __ldg(a.slots + t);
      if (sl >= 0 && sl < a.pool_rows) slot = sl;
    }
    const size_t at = static_cast<size_t>(t) * a.hkv_rows * row, to = static_cast<size_t>(slot < 0 ? 0 : slot) * a.hkv_rows * row;
    if (a.hkv > 0)
      rope_heads<true, kInterleaved, kFp8>(un, a.k + t * a.k_stride, a.hkv, first, step, a.k_out ? a.k_out + at : nullptr,
                                           slot < 0 ? nullptr : a.k_pages + to, inv_scale + a.hq);
    if (a.hv > 0)
      rope_heads<false, kInterleaved, kFp8>(un, a.v + t * a.v_stride, a.hv, first, step, a.v_out ? a.v_out + at : nullptr,
                                            slot < 0 ? nullptr : a.v_pages + to, inv_scale + a.hq + a.hkv);
  }
}

template <bool kInterleaved, bool kFp8>
static cudaError_t launch_rope_t(const RopeArgs& args, cudaStream_t stream) {
  const int most = std::max(args.hq, std::max(args.hkv, args.hv));
  if (args.tokens == 0 || most == 0) return cudaSuccess;
  const unsigned bx = static_cast<unsigned>((args.tokens + kRopeThreads / 32 - 1) / (kRopeThreads / 32));
  // few tokens: spread a token's heads over more warps
  const unsigned splits = static_cast<unsigned>((most + 3) / 4);
  unsigned by = 1;
  while (by < splits && bx * by < 2 * 148) by *= 2;
  if (by > splits) by = splits;
  const size_t smem = kFp8 ? (static_cast<size_t>(args.hq) + args.hkv + args.hv) * sizeof(float) : 0;
  rope_kernel<kInterleaved, kFp8><<<dim3(bx, by), kRopeThreads, smem, stream>>>(args);
  return cudaGetLastError();
}

cudaError_t launch_rope(const RopeArgs& args, bool interleaved, bool fp8, cudaStream_t stream) {
  if (interleaved) return fp8 ? launch_rope_t<true, true>(args, stream) : launch_rope_t<true, false>(args, stream);
  return fp8 ? launch_rope_t<false, true>(args, stream) : launch_rope_t<false, false>(args, stream);
}

}  // namespace stem
