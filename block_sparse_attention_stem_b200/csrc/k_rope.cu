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
// by HBM; loads of kUnroll head rows are issued before the first is used.
#include <cuda_fp8.h>

#include "stem_device.cuh"
#include "stem_kernels.h"

namespace stem {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kUnroll = 4;

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Eight values to their place: 16 bytes of bf16, or 8 of e4m3 after scaling.
template <bool kFp8>
__device__ __forceinline__ void store8(uint8_t* dst, const float (&x)[8], float inv_scale) {
  if constexpr (kFp8) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = static_cast<uint32_t>(e4m3x2(x[4 * i] * inv_scale, x[4 * i + 1] * inv_scale)) |
             static_cast<uint32_t>(e4m3x2(x[4 * i + 2] * inv_scale, x[4 * i + 3] * inv_scale)) << 16;
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
}

}  // namespace

// grid: x = groups of 8 tokens' warps, y = splits of the head rows of a token
template <bool kInterleaved, bool kFp8>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kElt = kFp8 ? 1 : 2;
  constexpr int kRow = kHeadDim * kElt;  // bytes of an output head row
  const int lane = lane_id();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + warp_id();
  if (t >= a.tokens) return;
  const int u = lane & 7, sub = lane >> 3;
  const int units = a.rotary_dim >> 4;  // units that rotate
  const bool rot = u < units;
  // the unit's two vectors (of 8 elements) inside a head row
  int va, vb;
  if (kInterleaved || !rot) {
    va = 2 * u;
    vb = 2 * u + 1;
  } else {
    va = u;
    vb = u + units;
  }

  float cs[8], sn[8];
  if (rot) {
    const int64_t p = __ldg(a.positions + t);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t phase = static_cast<uint64_t>(p) * a.turn[8 * u + i];
      sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &sn[i], &cs[i]);
      cs[i] *= a.amplitude;
      sn[i] *= a.amplitude;
    }
  }
  int64_t slot = -1;
  if (a.k_pages != nullptr) {
    const int sl = __ldg(a.slots + t);
    if (sl >= 0 && sl < a.pool_rows) slot = sl;
  }

  // head rows of the token: q, then k, then v
  const int rows = a.hq + a.hkv + (a.has_v ? a.hkv_rows : 0);
  const int step = gridDim.y * 4;
  for (int r0 = blockIdx.y * 4 + sub; r0 < rows; r0 += step * kUnroll) {
    uint4 in[kUnroll][2];
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int r = r0 + x * step;
      if (r >= rows) break;
      const uint8_t* src;
      if (r < a.hq) src = a.q + t * a.q_stride + static_cast<int64_t>(r) * (kHeadDim * 2);
      else if (r < a.hq + a.hkv) src = a.k + t * a.k_stride + static_cast<int64_t>(r - a.hq) * (kHeadDim * 2);
      else src = a.v + t * a.v_stride + static_cast<int64_t>(r - a.hq - a.hkv) * (kHeadDim * 2);
      in[x][0] = *reinterpret_cast<const uint4*>(src + va * 16);
      in[x][1] = *reinterpret_cast<const uint4*>(src + vb * 16);
    }
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int r = r0 + x * step;
      if (r >= rows) break;
      const bool is_q = r < a.hq, is_v = r >= a.hq + a.hkv;
      const int head = is_q ? r : is_v ? r - a.hq - a.hkv : r - a.hq;
      const int heads = is_q ? a.hq : a.hkv_rows;
      float xa[8], xb[8];
      unpack8(in[x][0], xa);
      unpack8(in[x][1], xb);
      if (rot && !is_v) {
        if constexpr (kInterleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a0 = xa[2 * i], a1 = xa[2 * i + 1], b0 = xb[2 * i], b1 = xb[2 * i + 1];
            xa[2 * i] = a0 * cs[i] - a1 * sn[i];
            xa[2 * i + 1] = a1 * cs[i] + a0 * sn[i];
            xb[2 * i] = b0 * cs[4 + i] - b1 * sn[4 + i];
            xb[2 * i + 1] = b1 * cs[4 + i] + b0 * sn[4 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a0 = xa[i], b0 = xb[i];
            xa[i] = a0 * cs[i] - b0 * sn[i];
            xb[i] = b0 * cs[i] + a0 * sn[i];
          }
        }
      }
      float inv = 1.f;
      if constexpr (kFp8) inv = 1.f / __ldg((is_q ? a.q_scale : is_v ? a.v_scale : a.k_scale) + head);
      uint8_t* packed = is_q ? a.q_out : is_v ? a.v_out : a.k_out;
      uint8_t* pool = is_q || slot < 0 ? nullptr : is_v ? a.v_pages : a.k_pages;
      // bf16 rows that are not rotated keep their bits (a NaN's payload too)
      const bool keep = !kFp8 && (is_v || !rot);
#pragma unroll
      for (int to = 0; to < 2; ++to) {
        uint8_t* base = to == 0 ? packed : pool;
        if (base == nullptr) continue;
        base += ((to == 0 ? t : slot) * heads + head) * kRow;
        if (keep) {
          *reinterpret_cast<uint4*>(base + va * 16) = in[x][0];
          *reinterpret_cast<uint4*>(base + vb * 16) = in[x][1];
        } else {
          store8<kFp8>(base + va * 8 * kElt, xa, inv);
          store8<kFp8>(base + vb * 8 * kElt, xb, inv);
        }
      }
    }
  }
}

cudaError_t launch_rope(const RopeArgs& args, bool interleaved, bool fp8, cudaStream_t stream) {
  const int rows = args.hq + args.hkv + (args.has_v ? args.hkv_rows : 0);
  if (args.tokens == 0 || rows == 0) return cudaSuccess;
  const unsigned bx = static_cast<unsigned>((args.tokens + kRopeThreads / 32 - 1) / (kRopeThreads / 32));
  // few tokens: spread a token's head rows over more warps
  unsigned by = 1;
  const unsigned most = static_cast<unsigned>((rows + 3) / 4);
  while (by < most && bx * by < 2 * 148) by *= 2;
  if (by > most) by = most;
  const dim3 grid(bx, by);
  if (interleaved) {
    if (fp8) rope_kernel<true, true><<<grid, kRopeThreads, 0, stream>>>(args);
    else rope_kernel<true, false><<<grid, kRopeThreads, 0, stream>>>(args);
  } else {
    if (fp8) rope_kernel<false, true><<<grid, kRopeThreads, 0, stream>>>(args);
    else rope_kernel<false, false><<<grid, kRopeThreads, 0, stream>>>(args);
  }
  return cudaGetLastError();
}

}  // namespace stem
