// A whole bf16 pool into the 4-bit pool and back (include/gqa_int4.h).
//
// One block per tile of 16 tokens of a (page, kv head): thread (tau, j) holds channels
// 8 j .. 8 j + 7 of token tau, first of K, then of V.  Bound: HBM (4 D bytes of bf16 and
// 9/8 D bytes of the 4-bit cache per token and kv head).
#include "int4_codec.cuh"
#include "internal.cuh"
#include "ptx.cuh"

namespace gqa {

// Source row of a tile's token: pools are [P, Hk, ps, D], tiles [P, Hk, ps / 16], so tile i
// covers rows 16 i .. 16 i + 15 of both.
template <int D>
__global__ void __launch_bounds__(2 * D) kv_quantize_int4_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                                                                 uint8_t* __restrict__ tiles) {
  using L = int4::Layout<D>;
  const int tau = threadIdx.x / L::kLanes, j = threadIdx.x % L::kLanes;
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * int4::kTile + tau) * L::kLanes + j;
  uint8_t* tile = tiles + static_cast<int64_t>(blockIdx.x) * L::kTileBytes;
  const uint4 in[2] = {__ldg(k + at), __ldg(v + at)};
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float x[8];
    int4::unpack8(in[kv], x);
    uint32_t pair;
    const uint32_t word = int4::quantize8(x, pair);
    *reinterpret_cast<uint32_t*>(tile + (kv ? L::v_word(tau, j) : L::k_word(tau, j))) = word;
    if (j % 8 == 0) *reinterpret_cast<uint32_t*>(tile + L::param(tau, kv, j / 8)) = pair;
  }
}

template <int D>
__global__ void __launch_bounds__(2 * D) kv_dequantize_int4_kernel(const uint8_t* __restrict__ tiles,
                                                                   uint4* __restrict__ k, uint4* __restrict__ v) {
  using L = int4::Layout<D>;
  const int tau = threadIdx.x / L::kLanes, j = threadIdx.x % L::kLanes;
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * int4::kTile + tau) * L::kLanes + j;
  const uint8_t* tile = tiles + static_cast<int64_t>(blockIdx.x) * L::kTileBytes;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(tile + (kv ? L::v_word(tau, j) : L::k_word(tau, j))));
    const uint32_t pair = __ldg(reinterpret_cast<const uint32_t*>(tile + L::param(tau, kv, j / 8)));
    const float step = __uint_as_float(pair << 16), low = __uint_as_float(pair & 0xffff0000u);
    float x[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      // 2^23 + code has the code in its low mantissa bits
      const float code = __uint_as_float(0x4b000000u | ((word >> (4 * n)) & 15u)) - 8388608.0f;
      x[n] = __fmaf_rn(code, step, low);
    }
    (kv ? v : k)[at] = int4::pack8(x);
  }
}

cudaError_t launch_kv_quantize_int4(const void* k, const void* v, void* tiles, int64_t num_tiles, int head_dim,
                                    cudaStream_t stream) {
  if (num_tiles == 0) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>(num_tiles);
  const uint4 *ks = static_cast<const uint4*>(k), *vs = static_cast<const uint4*>(v);
  if (head_dim == 64)
    kv_quantize_int4_kernel<64><<<grid, 128, 0, stream>>>(ks, vs, static_cast<uint8_t*>(tiles));
  else
    kv_quantize_int4_kernel<128><<<grid, 256, 0, stream>>>(ks, vs, static_cast<uint8_t*>(tiles));
  return cudaGetLastError();
}

cudaError_t launch_kv_dequantize_int4(const void* tiles, void* k, void* v, int64_t num_tiles, int head_dim,
                                      cudaStream_t stream) {
  if (num_tiles == 0) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>(num_tiles);
  uint4 *ks = static_cast<uint4*>(k), *vs = static_cast<uint4*>(v);
  if (head_dim == 64)
    kv_dequantize_int4_kernel<64><<<grid, 128, 0, stream>>>(static_cast<const uint8_t*>(tiles), ks, vs);
  else
    kv_dequantize_int4_kernel<128><<<grid, 256, 0, stream>>>(static_cast<const uint8_t*>(tiles), ks, vs);
  return cudaGetLastError();
}

}  // namespace gqa
