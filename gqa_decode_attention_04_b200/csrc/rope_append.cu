// Rotate q and k by position and append k and v to the paged cache, in one launch
// (include/gqa_rope.h; the 4-bit format: include/gqa_int4.h).
//
// Work: read q, k, v once, write q and the cache rows once; a handful of flops per element,
// so the bound is HBM for prompts and the launch for a decode step.  A row (one head of one
// token) is held by head_dim / 8 lanes of 16 bytes each.  In the half-split style the partner
// of a channel lies rotary_dim / 16 lanes away: the pair is brought together by shuffles of
// the packed bf16 words, so no element is read twice.  A thread keeps its cos and sin for all
// the rows it handles (the same channels of up to kRows heads of one token).
#include <cuda_fp8.h>

#include "int4_codec.cuh"
#include "internal.cuh"
#include "ptx.cuh"

namespace gqa {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t codes2(float a, float b, float s) {
  return static_cast<uint32_t>(
      __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(a, s), __fdiv_rn(b, s)), __NV_SATFINITE, __NV_E4M3));
}

}  // namespace

// One block: up to kRows * kThreads / (D / 8) rows of one token.  Rows are the q heads, then
// the k heads, then the v heads.
template <int D, int CACHE, int kRows>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeAppendParams p) {
  // A decode launched right after this one may start its prologue; it waits for this grid
  // before it reads anything that is written here.
  ptx::pdl_launch_dependents();
  constexpr int kLanes = D / 8;
  constexpr int kSlots = kThreads / kLanes;  // rows in flight
  const int t = blockIdx.x / p.chunks;
  const int first_row = (blockIdx.x - t * p.chunks) * (kSlots * kRows);
  const int j = threadIdx.x % kLanes;
  const int slot = threadIdx.x / kLanes;

  const int s = p.seq_ids != nullptr ? __ldg(p.seq_ids + t) : t;
  if (s < 0) return;  // padding
  const int pos = __ldg(p.positions + t);
  int page = -1;
  if (s < p.num_seqs && pos >= 0 && pos < p.max_positions &&
      static_cast<int64_t>(pos) < static_cast<int64_t>(p.max_blocks) * p.page_size)
    page = __ldg(p.block_table + static_cast<int64_t>(s) * p.max_blocks + pos / p.page_size);
  if (page < 0 || page >= p.num_pages) {
    if (first_row == 0 && threadIdx.x == 0) atomicOr(p.err, kErrBounds);
    return;
  }
  const int in_page = pos % p.page_size;

  const int half_lanes = p.rotary_dim / 16;  // lanes of the first half of the rotated channels
  const bool rotated = j < 2 * half_lanes;
  float c[8], sn[8];
  if (rotated) {
    const float* row = p.cos_sin + static_cast<int64_t>(pos) * p.rotary_dim;
    if (p.interleaved) {  // pairs (2 m, 2 m + 1), m = 4 j .. 4 j + 3
      const float4 a = __ldg(reinterpret_cast<const float4*>(row) + j);
      const float4 b = __ldg(reinterpret_cast<const float4*>(row + p.rotary_dim / 2) + j);
      c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
      sn[0] = b.x; sn[1] = b.y; sn[2] = b.z; sn[3] = b.w;
    } else {
      const int i = 8 * (j < half_lanes ? j : j - half_lanes);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(row + i) + h);
        const float4 b = __ldg(reinterpret_cast<const float4*>(row + p.rotary_dim / 2 + i) + h);
        c[4 * h] = a.x; c[4 * h + 1] = a.y; c[4 * h + 2] = a.z; c[4 * h + 3] = a.w;
        sn[4 * h] = b.x; sn[4 * h + 1] = b.y; sn[4 * h + 2] = b.z; sn[4 * h + 3] = b.w;
      }
    }
  }
  const bool second = !p.interleaved && j >= half_lanes;
  // the lane that holds the other half of this lane's pairs (itself where nothing is exchanged)
  const int lane = threadIdx.x & 31;
  const int partner = p.interleaved || !rotated ? lane : (second ? lane - half_lanes : lane + half_lanes);

  const int rows = p.num_heads + 2 * p.num_kv_heads;
  uint4 in[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int row = first_row + k * kSlots + slot;
    in[k] = make_uint4(0, 0, 0, 0);
    if (row < rows) {
      const uint16_t* src;
      if (row < p.num_heads) {
        src = p.q + t * p.q_stride + static_cast<int64_t>(row) * D;
      } else if (row < p.num_heads + p.num_kv_heads) {
        src = p.k + t * p.k_stride + static_cast<int64_t>(row - p.num_heads) * D;
      } else {
        src = p.v + t * p.v_stride + static_cast<int64_t>(row - p.num_heads - p.num_kv_heads) * D;
      }
      in[k] = *(reinterpret_cast<const uint4*>(src) + j);
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int row = first_row + k * kSlots + slot;
    const bool is_v = row >= p.num_heads + p.num_kv_heads;
    float x[8];
    int4::unpack8(in[k], x);
    uint4 other;
    other.x = __shfl_sync(0xffffffffu, in[k].x, partner);
    other.y = __shfl_sync(0xffffffffu, in[k].y, partner);
    other.z = __shfl_sync(0xffffffffu, in[k].z, partner);
    other.w = __shfl_sync(0xffffffffu, in[k].w, partner);
    if (rotated && !is_v) {
      if (p.interleaved) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float a = x[2 * m], b = x[2 * m + 1];
          x[2 * m] = __fsub_rn(__fmul_rn(a, c[m]), __fmul_rn(b, sn[m]));
          x[2 * m + 1] = __fadd_rn(__fmul_rn(b, c[m]), __fmul_rn(a, sn[m]));
        }
      } else {
        float y[8];
        int4::unpack8(other, y);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const float ys = __fmul_rn(y[m], sn[m]);
          x[m] = second ? __fadd_rn(__fmul_rn(x[m], c[m]), ys) : __fsub_rn(__fmul_rn(x[m], c[m]), ys);
        }
      }
    }
    uint32_t pair = 0, word = 0;
    // (the whole warp quantises if any of its rows is a cache row, so that the shuffles are whole)
    if (CACHE == kCacheInt4 && __any_sync(0xffffffffu, row >= p.num_heads && row < rows))
      word = int4::quantize8(x, pair);
    if (row >= rows) continue;
    if (row < p.num_heads) {
      *(reinterpret_cast<uint4*>(p.q_out + (static_cast<int64_t>(t) * p.num_heads + row) * D) + j) = int4::pack8(x);
      continue;
    }
    const int h = row - p.num_heads - (is_v ? p.num_kv_heads : 0);
    const int64_t page_head = static_cast<int64_t>(page) * p.num_kv_heads + h;
    if (CACHE == kCacheInt4) {
      using L = int4::Layout<D>;
      uint8_t* tile = p.k_pages + (page_head * (p.page_size / int4::kTile) + in_page / int4::kTile) * L::kTileBytes;
      const int tau = in_page % int4::kTile;
      *reinterpret_cast<uint32_t*>(tile + (is_v ? L::v_word(tau, j) : L::k_word(tau, j))) = word;
      if (j % 8 == 0) *reinterpret_cast<uint32_t*>(tile + L::param(tau, is_v, j / 8)) = pair;
    } else {
      const int64_t at = (page_head * p.page_size + in_page) * kLanes + j;
      uint8_t* pool = is_v ? p.v_pages : p.k_pages;
      if (CACHE == kCacheBf16) {
        *(reinterpret_cast<uint4*>(pool) + at) = is_v ? in[k] : int4::pack8(x);
      } else {
        const float sc = __ldg((is_v ? p.v_scales : p.k_scales) + h);
        uint2 w;
        w.x = codes2(x[0], x[1], sc) | (codes2(x[2], x[3], sc) << 16);
        w.y = codes2(x[4], x[5], sc) | (codes2(x[6], x[7], sc) << 16);
        *(reinterpret_cast<uint2*>(pool) + at) = w;
      }
    }
  }
}

namespace {

template <int D, int CACHE>
cudaError_t launch_rows(RopeAppendParams p, int sms, cudaStream_t stream) {
  const int rows = p.num_heads + 2 * p.num_kv_heads;
  constexpr int kSlots = kThreads / (D / 8);
  constexpr int kMany = 4;
  // Few tokens: one row per thread, so that the call's loads are all in flight at once on as
  // many SMs as there are rows.  Many: kMany rows per thread, which reads cos and sin once for
  // all of them.
  const int64_t chunks1 = (rows + kSlots - 1) / kSlots;
  const bool many = rows > kSlots && p.num_tokens * chunks1 > int64_t{8} * sms;
  const int per = many ? kSlots * kMany : kSlots;
  p.chunks = (rows + per - 1) / per;
  const int64_t blocks = static_cast<int64_t>(p.num_tokens) * p.chunks;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (many)
    rope_append_kernel<D, CACHE, kMany><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  else
    rope_append_kernel<D, CACHE, 1><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_cache(const RopeAppendParams& p, int cache, int sms, cudaStream_t stream) {
  if (cache == kCacheBf16) return launch_rows<D, kCacheBf16>(p, sms, stream);
  if (cache == kCacheE4m3) return launch_rows<D, kCacheE4m3>(p, sms, stream);
  return launch_rows<D, kCacheInt4>(p, sms, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams& p, int cache, int head_dim, int sms, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  return head_dim == 64 ? launch_cache<64>(p, cache, sms, stream) : launch_cache<128>(p, cache, sms, stream);
}

}  // namespace gqa
