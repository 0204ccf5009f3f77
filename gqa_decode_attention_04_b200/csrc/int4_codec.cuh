// The 4-bit cache's format (include/gqa_int4.h): quantising a group, and where a token's
// bytes lie inside a tile of 16 tokens.
//
// A group of 64 channels is held by 8 consecutive lanes, 8 channels each, so its minimum and
// maximum are three shuffles and every lane ends up with exactly one 32-bit word of codes.
#pragma once

#include "ptx.cuh"

namespace gqa {
namespace int4 {

constexpr int kTile = 16;    // tokens per tile
constexpr int kGroup = 64;   // channels that share a step and a minimum

template <int D>
struct Layout {
  static constexpr int kGroups = D / kGroup;
  static constexpr int kVCodes = 8 * D;       // byte offsets of a tile's sections
  static constexpr int kParams = 16 * D;
  static constexpr int kTileBytes = 18 * D;
  static constexpr int kLanes = D / 8;        // lanes that hold one row

  // Byte offset, in the tile, of the word of codes of lane j's channels 8 j .. 8 j + 7.
  __device__ static __forceinline__ int k_word(int tau, int j) {
    return tau * (D / 2) + ((j & 7) >> 1) * (D / 8) + (j >> 3) * 8 + (j & 1) * 4;
  }
  __device__ static __forceinline__ int v_row(int tau) {
    return (tau & 8) + ((tau & 1) << 2) + ((tau & 7) >> 1);
  }
  __device__ static __forceinline__ int v_word(int tau, int j) {
    const int g = j & 7, u = j >> 3;
    return kVCodes + (g / (8 / kGroups)) * 512 + v_row(tau) * 32 + (g % (8 / kGroups)) * (4 * kGroups) + u * 4;
  }
  // The (step, low) pair of group r of K (kv = 0) or V (kv = 1).
  __device__ static __forceinline__ int param(int tau, int kv, int r) {
    return kParams + tau * (8 * kGroups) + kv * (4 * kGroups) + 4 * r;
  }
};

// Minimum / maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float bf16_round(float x) {
  return __bfloat162float(__float2bfloat16_rn(x));
}

// Codes of this lane's 8 channels (nibble n = channel n) of a group held by 8 aligned lanes;
// pair = step (low half) | low (high half), the same in the 8 lanes.  Every lane of the warp
// takes part.  The quotient (x - low) / step is the correctly rounded one: with
// r = RN(1 / step), y = RN(t r) and the exact residual e = t - y step (one fma), RN(y + e r)
// is RN(t / step) (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990) where nothing over- or underflows; a step outside
// [2^-60, 2^60] takes the plain division.  A tie of code + 1/2 is therefore decided as in
// exact arithmetic, to the even code.
__device__ __forceinline__ uint32_t quantize8(const float (&x)[8], uint32_t& pair) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, d));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, d));
  }
  const float low = bf16_round(lo);
  const float step = bf16_round(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
  if (!(fabsf(low) < INFINITY) || !(step < INFINITY)) {  // a NaN, an infinity, or an infinite range
    pair = 0x7fff7fffu;
    return 0;
  }
  pair = __float_as_uint(low) | (__float_as_uint(step) >> 16);
  if (step == 0.0f) return 0;
  const float r = __frcp_rn(step);
  const bool plain = step < 0x1p-60f || step > 0x1p60f;
  uint32_t word = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float t = __fsub_rn(x[i], low);
    float y = __fmul_rn(t, r);
    y = __fmaf_rn(__fmaf_rn(-y, step, t), r, y);
    if (plain) y = __fdiv_rn(t, step);
    y = fminf(fmaxf(y, 0.0f), 15.0f);
    // adding 1.5 * 2^23 leaves rint(y), ties to even, in the low mantissa bits
    word = (word << 4) | (__float_as_uint(__fadd_rn(y, 12582912.0f)) & 15u);
  }
  return word;
}

// bf16 pairs (element 0 in the low half) of 16 bytes as 8 floats.
__device__ __forceinline__ void unpack8(const uint4 w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v[i] << 16);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint4 w;
  w.x = ptx::pack_bf16x2(x[0], x[1]);
  w.y = ptx::pack_bf16x2(x[2], x[3]);
  w.z = ptx::pack_bf16x2(x[4], x[5]);
  w.w = ptx::pack_bf16x2(x[6], x[7]);
  return w;
}

}  // namespace int4
}  // namespace gqa
