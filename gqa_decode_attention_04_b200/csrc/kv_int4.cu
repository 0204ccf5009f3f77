// A whole bf16 pool into the 4-bit pool and back (include/gqa_int4.h).
//
// Pools are [P, Hk, ps, D], tiles [P, Hk, ps / 16], so tile i covers rows 16 i .. 16 i + 15 of both:
// thread (tau, j) of a tile holds channels 16 j .. 16 j + 15 of token tau, first of K, then of V
// (16 channels a thread, not 8: the minimum, the step and its reciprocal are found half as often).
// A block does 256 threads' worth of tiles.
// Bound: HBM (4 D bytes of bf16 and 9/8 D bytes of the 4-bit cache per token and kv head).  9001 pages
// of 16 tokens and 8 kv heads, there and back: 273 us for 1.51 GB, 5.5 TB/s, 85 % of a copy's rate (349 us with 8
// channels a thread and plain divisions).
#include "int4_codec.cuh"
#include "internal.cuh"
#include "ptx.cuh"

namespace gqa {

namespace {
constexpr int kThreads = 256;
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_quantize_int4_kernel(const uint4* __restrict__ k,
                                                                    const uint4* __restrict__ v,
                                                                    uint8_t* __restrict__ tiles, int64_t num_tiles) {
  using L = int4::Layout<D>;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / D) + threadIdx.x / D;
  // (a whole warp is in one tile, so the shuffles are whole)
  if (i >= num_tiles) return;
  const int tau = threadIdx.x % D / (D / 16), j = 2 * (threadIdx.x % (D / 16));
  const int64_t at = (i * int4::kTile + tau) * L::kLanes + j;
  uint8_t* tile = tiles + i * L::kTileBytes;
  uint4 in[2][2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    in[0][w] = __ldg(k + at + w);
    in[1][w] = __ldg(v + at + w);
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float x[16];
    int4::unpack8(in[kv][0], *reinterpret_cast<float(*)[8]>(&x[0]));
    int4::unpack8(in[kv][1], *reinterpret_cast<float(*)[8]>(&x[8]));
    uint32_t words[2], pair;
    int4::quantize<2>(x, words, pair);
    if (kv == 0) {  // the words of channels 16 j .. lie side by side
      *reinterpret_cast<uint2*>(tile + L::k_word(tau, j)) = make_uint2(words[0], words[1]);
    } else {
      *reinterpret_cast<uint32_t*>(tile + L::v_word(tau, j)) = words[0];
      *reinterpret_cast<uint32_t*>(tile + L::v_word(tau, j + 1)) = words[1];
    }
    if (j % 8 == 0) *reinterpret_cast<uint32_t*>(tile + L::param(tau, kv, j / 8)) = pair;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_dequantize_int4_kernel(const uint8_t* __restrict__ tiles,
                                                                      uint4* __restrict__ k, uint4* __restrict__ v,
                                                                      int64_t num_tiles) {
  using L = int4::Layout<D>;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / D) + threadIdx.x / D;
  if (i >= num_tiles) return;
  const int tau = threadIdx.x % D / (D / 16), j = 2 * (threadIdx.x % (D / 16));
  const int64_t at = (i * int4::kTile + tau) * L::kLanes + j;
  const uint8_t* tile = tiles + i * L::kTileBytes;
  uint32_t word[2][2], pair[2];
  const uint2 kw = __ldg(reinterpret_cast<const uint2*>(tile + L::k_word(tau, j)));
  word[0][0] = kw.x;
  word[0][1] = kw.y;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    word[1][w] = __ldg(reinterpret_cast<const uint32_t*>(tile + L::v_word(tau, j + w)));
    pair[w] = __ldg(reinterpret_cast<const uint32_t*>(tile + L::param(tau, w, j / 8)));
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const float step = __uint_as_float(pair[kv] << 16), low = __uint_as_float(pair[kv] & 0xffff0000u);
    const uint64_t step2 = ptx::f2_pack(step, step), low2 = ptx::f2_pack(low, low);
    const uint64_t up2 = ptx::f2_pack(8388608.0f, 8388608.0f);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float x[8];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        // 2^23 + code has the code in its low mantissa bits
        const float a = __uint_as_float(0x4b000000u | ((word[kv][w] >> (8 * n)) & 15u));
        const float b = __uint_as_float(0x4b000000u | ((word[kv][w] >> (8 * n + 4)) & 15u));
        ptx::f2_unpack(ptx::f2_fma(ptx::f2_sub(ptx::f2_pack(a, b), up2), step2, low2), x[2 * n], x[2 * n + 1]);
      }
      (kv ? v : k)[at + w] = int4::pack8(x);
    }
  }
}

namespace {

unsigned blocks_of(int64_t num_tiles, int head_dim) {
  const int per = kThreads / head_dim;
  return static_cast<unsigned>((num_tiles + per - 1) / per);
}

}  // namespace

cudaError_t launch_kv_quantize_int4(const void* k, const void* v, void* tiles, int64_t num_tiles, int head_dim,
                                    cudaStream_t stream) {
  if (num_tiles == 0) return cudaSuccess;
  const unsigned grid = blocks_of(num_tiles, head_dim);
  const uint4 *ks = static_cast<const uint4*>(k), *vs = static_cast<const uint4*>(v);
  if (head_dim == 64)
    kv_quantize_int4_kernel<64><<<grid, kThreads, 0, stream>>>(ks, vs, static_cast<uint8_t*>(tiles), num_tiles);
  else
    kv_quantize_int4_kernel<128><<<grid, kThreads, 0, stream>>>(ks, vs, static_cast<uint8_t*>(tiles), num_tiles);
  return cudaGetLastError();
}

cudaError_t launch_kv_dequantize_int4(const void* tiles, void* k, void* v, int64_t num_tiles, int head_dim,
                                      cudaStream_t stream) {
  if (num_tiles == 0) return cudaSuccess;
  const unsigned grid = blocks_of(num_tiles, head_dim);
  uint4 *ks = static_cast<uint4*>(k), *vs = static_cast<uint4*>(v);
  if (head_dim == 64)
    kv_dequantize_int4_kernel<64><<<grid, kThreads, 0, stream>>>(static_cast<const uint8_t*>(tiles), ks, vs, num_tiles);
  else
    kv_dequantize_int4_kernel<128><<<grid, kThreads, 0, stream>>>(static_cast<const uint8_t*>(tiles), ks, vs, num_tiles);
  return cudaGetLastError();
}

}  // namespace gqa
