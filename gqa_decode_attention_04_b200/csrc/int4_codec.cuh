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

// Codes of this lane's 8 W channels (nibble n of words[w] = channel 8 w + n) of a group held by
// 8 / W aligned lanes; pair = step (low half) | low (high half), the same in those lanes.  Every
// lane of the warp takes part; a group whose lanes have `wanted` false gets no codes, and has no say in how
// the others' are found.
//
// Both quotients, range / 15 and (x - low) / step, are the correctly rounded ones: with r = RN(1 / d),
// y = RN(a r) and the exact residual e = a - y d (one fma), RN(y + e r) is RN(a / d) (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990) where nothing
// over- or underflows; a warp with a range outside [2^-60, 2^60] takes plain divisions.  A tie of
// code + 1/2 is therefore decided as in exact arithmetic, to the even code.  The arithmetic is what
// bounds the writers (a pool of 150 MB: 28 us for its bytes), so it goes in packed pairs, and the
// codes are put together as one exact number, c0 + 16 c1 + 256 c2 + 4096 c3.
template <int W>
__device__ __forceinline__ void quantize(const float (&x)[8 * W], uint32_t (&words)[W], uint32_t& pair, bool wanted = true) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8 * W; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
#pragma unroll
  for (int d = 1; d < 8 / W; d <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, d));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, d));
  }
  const float low = bf16_round(lo);
  const float range = __fsub_rn(hi, lo);
  const bool usual = range >= 0x1p-60f && range <= 0x1p60f && fabsf(low) < INFINITY;
  if (__all_sync(0xffffffffu, usual || !wanted)) {
    constexpr float kFifteenth = 1.0f / 15.0f;
    float step = __fmul_rn(range, kFifteenth);
    step = bf16_round(__fmaf_rn(__fmaf_rn(-step, 15.0f, range), kFifteenth, step));
    pair = __float_as_uint(low) | (__float_as_uint(step) >> 16);
    const float r = __frcp_rn(step);
    const uint64_t r2 = ptx::f2_pack(r, r), step2 = ptx::f2_pack(-step, -step), low2 = ptx::f2_pack(low, low);
    const uint64_t up2 = ptx::f2_pack(12582912.0f, 12582912.0f);  // 1.5 * 2^23: adding it rounds to a whole number
#pragma unroll
    for (int w = 0; w < W; ++w) {
      float c[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t t = ptx::f2_sub(ptx::f2_pack(x[8 * w + 2 * i], x[8 * w + 2 * i + 1]), low2);
        uint64_t y = ptx::f2_mul(t, r2);
        y = ptx::f2_fma(ptx::f2_fma(y, step2, t), r2, y);
        float a, b;
        ptx::f2_unpack(y, a, b);
        a = fminf(fmaxf(a, 0.0f), 15.0f);
        b = fminf(fmaxf(b, 0.0f), 15.0f);
        ptx::f2_unpack(ptx::f2_sub(ptx::f2_add(ptx::f2_pack(a, b), up2), up2), c[2 * i], c[2 * i + 1]);
      }
      float half[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        half[i] = fmaf(4096.0f, c[4 * i + 3], fmaf(256.0f, c[4 * i + 2], fmaf(16.0f, c[4 * i + 1], c[4 * i])));
      // 2^23 + n has the whole number n in its low mantissa bits
      words[w] = __byte_perm(__float_as_uint(half[0] + 8388608.0f), __float_as_uint(half[1] + 8388608.0f), 0x5410);
    }
    return;
  }
  const float step = bf16_round(__fdiv_rn(range, 15.0f));
  const bool finite = fabsf(low) < INFINITY && step < INFINITY;  // else a NaN, an infinity, or an infinite range
  pair = finite ? __float_as_uint(low) | (__float_as_uint(step) >> 16) : 0x7fff7fffu;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    words[w] = 0;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      const float y = finite && step > 0.0f ? __fdiv_rn(__fsub_rn(x[8 * w + i], low), step) : 0.0f;
      words[w] = (words[w] << 4) | static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(y, 0.0f), 15.0f)));
    }
  }
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
