// Rotate q and k by position and append k and v to the paged cache, in one launch
// (include/gqa_rope.h; the 4-bit format: include/gqa_int4.h).
//
// Work: read q, k, v once, write q and the cache rows once; a handful of flops per element,
// so the bound is HBM for prompts and the launch for a decode step.  A row (one head of one
// token) is held by head_dim / 8 lanes of 16 bytes each.  In the half-split style the partner
// of a channel lies rotary_dim / 16 lanes away: the pair is brought together by shuffles of
// the packed bf16 words, so no element is read twice.  A thread keeps its cos and sin for all
// the rows it handles (the same channels of several heads of one token).
//   Measured: one token of 32 + 8 heads 2.0 us and 256 of them into bf16 2.8 us (the launch, then two
// dependent loads: position, then block table and angles); 5987 tokens of 12 + 2 heads of 64 into e4m3 5.9
// us (4.1 TB/s), 16384 of 32 + 8 of 128 into bf16 69 us (5.9 TB/s, 90 % of a copy's rate), of 64 + 8 into 4
// bits, the pool read back, 146 us (5.5 TB/s, 84 %).
#include <climits>

#include <cuda_fp8.h>

#include "int4_codec.cuh"
#include "internal.cuh"
#include "ptx.cuh"

namespace gqa {

namespace {

constexpr int kThreads = 256;
// q rows of a thread whose loads are in flight together, and blocks per SM that the registers are held
// down for: 16384 tokens of 64 + 8 heads into 4 bits with the pool read back take 144 us with (4, 4), 148
// with (4, 5), 155 with (4, 3), 151 with (3, 4), 154 with (2, 4); of 32 + 8 heads into bf16 70, 75, 78, 74, 77.
// (A row's successor loaded as soon as it is turned, instead of four at a time: 162 and 80 us.)
constexpr int kBatch = 4, kBlocks = 4;

__device__ __forceinline__ uint32_t codes2(float a, float b, float s) {
  return static_cast<uint32_t>(
      __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(a, s), __fdiv_rn(b, s)), __NV_SATFINITE, __NV_E4M3));
}

}  // namespace

// A token's rows are the q heads, then the k heads, then the v heads.  MANY: 1 << p.spread_log2 q rows
// of a token are worked on side by side, each thread going on to every such-manieth, and likewise its
// k and v rows.  Otherwise one row a thread, p.chunks blocks per token.
template <int D, int CACHE, bool MANY, bool INTER>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_append_kernel(const RopeAppendParams p) {
  // The attention of a 4-bit step, launched right after this one, may start its prologue; it waits for this grid
  // before it reads anything that is written here.  (All other calls wait for the whole grid.)
  ptx::pdl_launch_dependents();
  constexpr int kLanes = D / 8;
  constexpr int kSlots = kThreads / kLanes;  // rows in flight in a block
  const int j = threadIdx.x % kLanes;
  const int slot = threadIdx.x / kLanes;
  int t, row, stride;
  if (MANY) {
    t = blockIdx.x * (kSlots >> p.spread_log2) + (slot >> p.spread_log2);
    stride = 1 << p.spread_log2;
    row = slot & (stride - 1);
  } else {
    t = blockIdx.x / p.chunks;
    row = (blockIdx.x - t * p.chunks) * kSlots + slot;
    stride = INT_MAX / 2;
  }
  // The first rows are on their way before it is known where they go, or that they are padding: what a
  // block waits for is latency.  (256 tokens into bf16 4.6 us with
  // the rows loaded after the page is known, 3.9 so; 16384 of 64 + 8 heads into 4 bits, read back, 182 and
  // 169, both before the other steps.)
  const bool here = t < p.num_tokens;
  constexpr int kQ = MANY ? kBatch : 1;
  const int cached = 2 * p.num_kv_heads;
  const uint4* q_in = reinterpret_cast<const uint4*>(p.q + t * p.q_stride) + j;
  auto load_q = [&](int r) { return here && r < p.num_heads ? q_in[r * kLanes] : make_uint4(0, 0, 0, 0); };
  auto load_cached = [&](int r) {
    uint4 in = make_uint4(0, 0, 0, 0);
    if (here && r >= 0 && r < cached) {
      const uint16_t* src = r < p.num_kv_heads ? p.k + t * p.k_stride + r * D : p.v + t * p.v_stride + (r - p.num_kv_heads) * D;
      in = *(reinterpret_cast<const uint4*>(src) + j);
    }
    return in;
  };
  const int first_cached = MANY ? row : row - p.num_heads;
  uint4 q_rows[kQ];
#pragma unroll
  for (int k = 0; k < kQ; ++k) q_rows[k] = load_q(row + k * stride);
  uint4 c_row = load_cached(first_cached);
  // (a warp may hold rows of several tokens, of which some are skipped: all its lanes stay for the shuffles)
  bool live = here;
  const int s = !live ? -1 : (p.seq_ids != nullptr ? __ldg(p.seq_ids + t) : t);
  const int pos = live ? __ldg(p.positions + t) : 0;
  live = s >= 0;  // else padding
  int page = -1, in_page = 0;
  if (live && s < p.num_seqs && pos >= 0 && pos < p.max_positions &&
      static_cast<int64_t>(pos) < static_cast<int64_t>(p.max_blocks) * p.page_size) {
    const int block = p.page_size == 1 ? pos : fast_div(pos, p.ps_magic, p.ps_shift);
    in_page = pos - block * p.page_size;
    page = __ldg(p.block_table + static_cast<int64_t>(s) * p.max_blocks + block);
  }

  const int half_lanes = p.rotary_dim / 16;  // lanes of the first half of the rotated channels
  const bool rotated = j < 2 * half_lanes;
  const bool second = !INTER && j >= half_lanes;
  // x[i] becomes x[i] c[i] + (its partner) sn[i], the sine's sign taken in; (1, 0) where nothing turns
  float c[8], sn[8];
#pragma unroll
  for (int m = 0; m < 8; ++m) c[m] = 1.0f, sn[m] = 0.0f;
  if (rotated && live && static_cast<unsigned>(pos) < static_cast<unsigned>(p.max_positions)) {
    const float* at = p.cos_sin + static_cast<int64_t>(pos) * p.rotary_dim;
    if (INTER) {  // pairs (2 m, 2 m + 1), m = 4 j .. 4 j + 3
      const float4 a = __ldg(reinterpret_cast<const float4*>(at) + j);
      const float4 b = __ldg(reinterpret_cast<const float4*>(at + p.rotary_dim / 2) + j);
      c[0] = c[1] = a.x; c[2] = c[3] = a.y; c[4] = c[5] = a.z; c[6] = c[7] = a.w;
      sn[0] = -b.x; sn[1] = b.x; sn[2] = -b.y; sn[3] = b.y; sn[4] = -b.z; sn[5] = b.z; sn[6] = -b.w; sn[7] = b.w;
    } else {
      const int i = 8 * (second ? j - half_lanes : j);
      const float sign = second ? 1.0f : -1.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(at + i) + h);
        const float4 b = __ldg(reinterpret_cast<const float4*>(at + p.rotary_dim / 2 + i) + h);
        c[4 * h] = a.x; c[4 * h + 1] = a.y; c[4 * h + 2] = a.z; c[4 * h + 3] = a.w;
        sn[4 * h] = sign * b.x; sn[4 * h + 1] = sign * b.y; sn[4 * h + 2] = sign * b.z; sn[4 * h + 3] = sign * b.w;
      }
    }
  }
  if (live && (page < 0 || page >= p.num_pages)) {
    live = false;
    if (row == 0 && j == 0) atomicOr(p.err, kErrBounds);
  }
  // the lane that holds the other half of this lane's pairs (itself where nothing is exchanged)
  const int lane = threadIdx.x & 31;
  const int partner = INTER || !rotated ? lane : (second ? lane - half_lanes : lane + half_lanes);
  auto rotate = [&](const uint4 in, float (&x)[8]) {
    int4::unpack8(in, x);
    float y[8];
    if (INTER) {
#pragma unroll
      for (int m = 0; m < 8; ++m) y[m] = x[m ^ 1];
    } else {
      uint4 other;
      other.x = __shfl_sync(0xffffffffu, in.x, partner);
      other.y = __shfl_sync(0xffffffffu, in.y, partner);
      other.z = __shfl_sync(0xffffffffu, in.z, partner);
      other.w = __shfl_sync(0xffffffffu, in.w, partner);
      int4::unpack8(other, y);
    }
    if (rotated) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        // Each product and the sum are rounded, never one fma: the products in packed pairs, the sums
        // not, which the compiler does not contract (it does contract a packed product and sum).
        float a[2], b[2];
        ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(x[2 * m], x[2 * m + 1]), ptx::f2_pack(c[2 * m], c[2 * m + 1])), a[0], a[1]);
        ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(y[2 * m], y[2 * m + 1]), ptx::f2_pack(sn[2 * m], sn[2 * m + 1])), b[0], b[1]);
        x[2 * m] = __fadd_rn(a[0], b[0]);
        x[2 * m + 1] = __fadd_rn(a[1], b[1]);
      }
    }
  };

  // ---- q
  uint4* q_out = reinterpret_cast<uint4*>(p.q_out + static_cast<int64_t>(t) * p.num_heads * D) + j;
#pragma unroll 1
  for (int r0 = row; __any_sync(0xffffffffu, r0 < p.num_heads); r0 += kQ * stride) {
#pragma unroll
    for (int k = 0; k < kQ; ++k) {
      const int r = r0 + k * stride;
      float x[8];
      rotate(q_rows[k], x);
      if (live && r < p.num_heads) q_out[r * kLanes] = int4::pack8(x);
    }
    if (!MANY) break;
#pragma unroll
    for (int k = 0; k < kQ; ++k) q_rows[k] = load_q(r0 + (kQ + k) * stride);
  }

  // ---- k, then v
#pragma unroll 1
  for (int r = first_cached; __any_sync(0xffffffffu, r >= 0 && r < cached);) {
    const uint4 next = MANY ? load_cached(r + stride) : make_uint4(0, 0, 0, 0);
    const bool is_v = r >= p.num_kv_heads;
    float x[8], turned[8];
    int4::unpack8(c_row, x);
    if (__any_sync(0xffffffffu, !is_v)) {
      rotate(c_row, turned);
#pragma unroll
      for (int m = 0; m < 8; ++m) x[m] = is_v ? x[m] : turned[m];
    }
    const bool wanted = live && r >= 0 && r < cached;
    uint32_t pair = 0, word[1] = {0};
    if (CACHE == kCacheInt4) int4::quantize<1>(x, word, pair, wanted);  // (by the whole warp: it shuffles)
    if (wanted) {
      const int h = r - (is_v ? p.num_kv_heads : 0);
      const int64_t page_head = static_cast<int64_t>(page) * p.num_kv_heads + h;
      if (CACHE == kCacheInt4) {
        using L = int4::Layout<D>;
        uint8_t* tile = p.k_pages + (page_head * (p.page_size / int4::kTile) + in_page / int4::kTile) * L::kTileBytes;
        const int tau = in_page % int4::kTile;
        *reinterpret_cast<uint32_t*>(tile + (is_v ? L::v_word(tau, j) : L::k_word(tau, j))) = word[0];
        if (j % 8 == 0) *reinterpret_cast<uint32_t*>(tile + L::param(tau, is_v, j / 8)) = pair;
      } else {
        const int64_t at = (page_head * p.page_size + in_page) * kLanes + j;
        uint8_t* pool = is_v ? p.v_pages : p.k_pages;
        if (CACHE == kCacheBf16) {
          *(reinterpret_cast<uint4*>(pool) + at) = is_v ? c_row : int4::pack8(x);
        } else {
          const float sc = __ldg((is_v ? p.v_scales : p.k_scales) + h);
          uint2 w;
          w.x = codes2(x[0], x[1], sc) | (codes2(x[2], x[3], sc) << 16);
          w.y = codes2(x[4], x[5], sc) | (codes2(x[6], x[7], sc) << 16);
          *(reinterpret_cast<uint2*>(pool) + at) = w;
        }
      }
    }
    if (!MANY) break;
    r += stride;
    c_row = next;
  }
}

namespace {

template <int D, int CACHE>
cudaError_t launch_rows(RopeAppendParams p, int sms, cudaStream_t stream) {
  const int rows = p.num_heads + 2 * p.num_kv_heads;
  constexpr int kSlots = kThreads / (D / 8);
  if (p.page_size > 1) divisor_magic(static_cast<uint32_t>(p.page_size), &p.ps_magic, &p.ps_shift);
  // As long as all rows fit on the GPU at once, one row a thread: the call's loads are all in flight
  // together.  Beyond that kBatch q rows a thread or more, which finds the token's place, cos and sin once
  // for all of them.  (Into bf16, 32 + 8 heads: 128 tokens 2.8 us one row a thread and 3.0 otherwise, 256
  // 3.7 and 3.1, 600 6.3 and 4.4; 12 + 2 heads of 64: 400 tokens 2.5 and 3.5, 800 3.9 and 3.6.)
  const int64_t per_gpu = int64_t{kThreads * kBlocks} * sms / (D / 8);
  int64_t blocks;
  const bool many = p.num_tokens * static_cast<int64_t>(rows) > per_gpu;
  if (many) {
    // Twice kBatch rows a thread while that leaves the GPU half full of threads: 16384 tokens of 32 + 8
    // heads into bf16 71 us, and 77 with kBatch; 5987 of 12 + 2 heads of 64 into e4m3 8.1, and 6.4.  The k and v
    // rows count where they are more than q's, or are all there is: 593 sequences of 8 kv heads into 4 bits
    // without rotation 4.6 us, and 23 with all 16 rows a thread (592, one row a thread: 3.3).
    p.spread_log2 = 0;
    const int most = p.num_heads > 2 * p.num_kv_heads ? p.num_heads : 2 * p.num_kv_heads;
    auto can = [&](int rows) { return (2 << p.spread_log2) <= kSlots && (2 << p.spread_log2) * rows <= most; };
    while (can(2 * kBatch)) ++p.spread_log2;
    if (static_cast<int64_t>(p.num_tokens) * (D / 8 << p.spread_log2) < int64_t{kThreads * kBlocks / 2} * sms)
      while (can(kBatch)) ++p.spread_log2;
    const int tokens = kSlots >> p.spread_log2;
    blocks = (static_cast<int64_t>(p.num_tokens) + tokens - 1) / tokens;
  } else {
    p.chunks = (rows + kSlots - 1) / kSlots;
    blocks = static_cast<int64_t>(p.num_tokens) * p.chunks;
  }
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const auto kernel = p.interleaved ? (many ? rope_append_kernel<D, CACHE, true, true> : rope_append_kernel<D, CACHE, false, true>)
                                    : (many ? rope_append_kernel<D, CACHE, true, false> : rope_append_kernel<D, CACHE, false, false>);
  kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
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
