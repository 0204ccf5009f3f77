// C ABI of the 4-bit cache and of the rotating appends (include/gqa_int4.h,
// include/gqa_rope.h): argument checks, then the launch.  Nothing is launched on a bad
// argument, and no call synchronises or allocates, but for the device's error word on the
// first call (as in gqa_decode.cu).
#include <cmath>
#include <climits>

#include "gqa_int4.h"
#include "gqa_rope.h"
#include "internal.cuh"

namespace {

using gqa::set_error;

constexpr int kTile = 16;

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

gqa_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return GQA_OK;
  return set_error(GQA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Sizes that every call on a 4-bit pool shares.
gqa_status check_pool(int num_kv_heads, int head_dim, int page_size) {
  if (num_kv_heads < 1 || head_dim < 1 || page_size < 1) return set_error(GQA_ERR_INVALID_ARG, "sizes must be positive");
  if (head_dim != 64 && head_dim != 128) return set_error(GQA_ERR_UNSUPPORTED, "head_dim %d not built (64, 128)", head_dim);
  if (page_size % kTile != 0 || page_size > 256)
    return set_error(GQA_ERR_UNSUPPORTED, "page_size %d not built (multiple of 16, <= 256)", page_size);
  return GQA_OK;
}

gqa_status check_rows(int num_pages, int num_kv_heads, int page_size, int max_blocks) {
  if (max_blocks < 1 || num_pages < 1) return set_error(GQA_ERR_INVALID_ARG, "sizes must be positive");
  if (static_cast<int64_t>(num_pages) * num_kv_heads * page_size > INT32_MAX)
    return set_error(GQA_ERR_UNSUPPORTED, "num_pages * num_kv_heads * page_size exceeds 2^31");
  if (static_cast<int64_t>(max_blocks) * page_size > INT32_MAX)
    return set_error(GQA_ERR_UNSUPPORTED, "max_blocks_per_seq * page_size exceeds 2^31");
  return GQA_OK;
}

// The append of all three caches.  q == nullptr with num_heads == 0 and rotary_dim == 0: no
// rotation (gqa_kv_append_int4).
gqa_status append(gqa::RopeAppendParams p, int cache, int head_dim, cudaStream_t stream) {
  if (p.num_tokens < 0) return set_error(GQA_ERR_INVALID_ARG, "num_tokens < 0");
  if (p.num_seqs < 0) return set_error(GQA_ERR_INVALID_ARG, "num_seqs < 0");
  const bool rotate = p.rotary_dim != 0;
  if ((rotate && p.num_heads < 1) || p.num_kv_heads < 1 || p.page_size < 1)
    return set_error(GQA_ERR_INVALID_ARG, "sizes must be positive");
  if (cache == gqa::kCacheInt4) {
    const gqa_status s = check_pool(p.num_kv_heads, head_dim, p.page_size);
    if (s != GQA_OK) return s;
  } else if (head_dim != 64 && head_dim != 128) {
    return set_error(GQA_ERR_UNSUPPORTED, "head_dim %d not built (64, 128)", head_dim);
  }
  gqa_status s = check_rows(p.num_pages, p.num_kv_heads, p.page_size, p.max_blocks);
  if (s != GQA_OK) return s;
  if (rotate) {
    if (p.rotary_dim < 16 || p.rotary_dim > head_dim || p.rotary_dim % 16 != 0)
      return set_error(GQA_ERR_INVALID_ARG, "rotary_dim %d is not a multiple of 16 in [16, %d]", p.rotary_dim, head_dim);
    if (p.max_positions < 1) return set_error(GQA_ERR_INVALID_ARG, "max_positions < 1");
  }
  const int64_t q_row = static_cast<int64_t>(p.num_heads) * head_dim, kv_row = static_cast<int64_t>(p.num_kv_heads) * head_dim;
  if (p.num_heads > INT32_MAX / 4096 || p.num_kv_heads > INT32_MAX / 4096)
    return set_error(GQA_ERR_UNSUPPORTED, "too many heads");
  if ((rotate && p.q_stride < q_row) || p.k_stride < kv_row || p.v_stride < kv_row)
    return set_error(GQA_ERR_INVALID_ARG, "a token stride is shorter than a token");
  if (p.q_stride % 8 != 0 || p.k_stride % 8 != 0 || p.v_stride % 8 != 0)
    return set_error(GQA_ERR_INVALID_ARG, "token strides must be multiples of 8 elements");
  if (p.num_tokens == 0) return GQA_OK;
  const bool two = cache != gqa::kCacheInt4, scaled = cache == gqa::kCacheE4m3;
  if (!p.k || !p.v || !p.k_pages || (two && !p.v_pages) || (scaled && (!p.k_scales || !p.v_scales)) || !p.block_table ||
      !p.positions || (rotate && (!p.q || !p.q_out || !p.cos_sin)))
    return set_error(GQA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(p.q, 16) || !aligned(p.q_out, 16) || !aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.cos_sin, 16) ||
      !aligned(p.k_pages, 16) || !aligned(p.v_pages, 16))
    return set_error(GQA_ERR_INVALID_ARG, "q, q_out, k_new, v_new, cos_sin and the pools must be 16-byte aligned");
  if (!aligned(p.k_scales, 4) || !aligned(p.v_scales, 4) || !aligned(p.block_table, 4) || !aligned(p.positions, 4) ||
      !aligned(p.seq_ids, 4))
    return set_error(GQA_ERR_INVALID_ARG, "scales and int32 arrays must be 4-byte aligned");
  if (p.seq_ids == nullptr && p.num_tokens > p.num_seqs)
    return set_error(GQA_ERR_INVALID_ARG, "without seq_ids num_tokens (%d) is at most num_seqs (%d)", p.num_tokens, p.num_seqs);
  if (rotate && p.q == p.q_out && p.q_stride != q_row)
    return set_error(GQA_ERR_INVALID_ARG, "q_out may be q only where q is contiguous");
  int sms;
  s = gqa::host_device(&p.err, &sms);
  if (s != GQA_OK) return s;
  s = cuda_status(gqa::launch_rope_append(p, cache, head_dim, sms, stream), "append launch");
  if (s == GQA_OK) gqa::host_count_launches(1);
  return s;
}

gqa::RopeAppendParams params(const void* q, const void* k_new, const void* v_new, const float* cos_sin, void* q_out,
                             void* k_pages, void* v_pages, const float* k_scales, const float* v_scales,
                             const int32_t* block_table, const int32_t* positions, const int32_t* seq_ids,
                             int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int rotary_dim,
                             int interleaved, int max_positions, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                             int page_size, int max_blocks, int num_pages) {
  gqa::RopeAppendParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k_new);
  p.v = static_cast<const uint16_t*>(v_new);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.cos_sin = cos_sin;
  p.block_table = block_table;
  p.positions = positions;
  p.seq_ids = seq_ids;
  p.k_pages = static_cast<uint8_t*>(k_pages);
  p.v_pages = static_cast<uint8_t*>(v_pages);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.num_tokens = num_tokens;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.rotary_dim = rotary_dim;
  p.interleaved = interleaved != 0;
  p.max_positions = max_positions;
  p.page_size = page_size;
  p.max_blocks = max_blocks;
  p.num_pages = num_pages;
  return p;
}

// A rotating append asks for a rotation (0 means none inside this file).
gqa_status need_rotation(int rotary_dim) {
  return rotary_dim >= 16 ? GQA_OK : set_error(GQA_ERR_INVALID_ARG, "rotary_dim %d < 16", rotary_dim);
}

gqa_status append_plain_int4(const void* k_new, const void* v_new, void* kv_pages, const int32_t* block_table,
                             const int32_t* positions, int num_seqs, int num_kv_heads, int head_dim, int page_size,
                             int max_blocks, int num_pages, void* stream) {
  const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
  return append(params(nullptr, k_new, v_new, nullptr, nullptr, kv_pages, nullptr, nullptr, nullptr, block_table,
                       positions, nullptr, num_seqs, num_seqs, 0, num_kv_heads, 0, 0, INT_MAX, 0, row, row, page_size,
                       max_blocks, num_pages),
                gqa::kCacheInt4, head_dim, static_cast<cudaStream_t>(stream));
}

// Checks of a decode call, and what it launches with.  launch == false: the checks alone.
gqa_status decode(const void* q, const void* kv_pages, const int32_t* block_table, const int32_t* seq_lens, void* out,
                  int num_seqs, int q_len, int num_heads, int num_kv_heads, int head_dim, int page_size, float scale,
                  int max_blocks, int num_pages, void* workspace, size_t workspace_bytes, void* stream, bool overlap,
                  bool launch) {
  if (num_seqs < 0) return set_error(GQA_ERR_INVALID_ARG, "num_seqs < 0");
  if (num_seqs > 65536) return set_error(GQA_ERR_UNSUPPORTED, "num_seqs > 65536");
  if (q_len < 1) return set_error(GQA_ERR_INVALID_ARG, "q_len %d < 1", q_len);
  if (num_heads < 1) return set_error(GQA_ERR_INVALID_ARG, "sizes must be positive");
  if (num_heads > INT32_MAX / 4096) return set_error(GQA_ERR_UNSUPPORTED, "too many heads");
  gqa_status s = check_pool(num_kv_heads, head_dim, page_size);
  if (s != GQA_OK) return s;
  if (num_heads % num_kv_heads != 0)
    return set_error(GQA_ERR_INVALID_ARG, "num_heads (%d) is not a multiple of num_kv_heads (%d)", num_heads, num_kv_heads);
  if (!std::isfinite(scale)) return set_error(GQA_ERR_INVALID_ARG, "scale is not finite");
  s = check_rows(num_pages, num_kv_heads, page_size, max_blocks);
  if (s != GQA_OK) return s;
  const int group = num_heads / num_kv_heads;
  if (q_len > 1 && static_cast<int64_t>(group) * q_len > 128)
    return set_error(GQA_ERR_UNSUPPORTED, "q_len %d x %d query heads per kv head exceeds 128", q_len, group);
  const int rows = group * q_len;
  const gqa::Int4Plan plan = gqa::plan_decode_int4(head_dim, rows);
  const int n_rt = (rows + 8 * plan.n_tiles - 1) / (8 * plan.n_tiles);
  if (static_cast<int64_t>(num_kv_heads) * n_rt * num_seqs > INT32_MAX)
    return set_error(GQA_ERR_UNSUPPORTED, "num_seqs x num_kv_heads x row tiles exceeds 2^31");
  if (num_seqs == 0) return GQA_OK;
  if (!q || !kv_pages || !block_table || !seq_lens || !out || !workspace)
    return set_error(GQA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(kv_pages, 16))
    return set_error(GQA_ERR_INVALID_ARG, "q, out and kv_pages must be 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4))
    return set_error(GQA_ERR_INVALID_ARG, "block_table and seq_lens must be 4-byte aligned");
  if (!aligned(workspace, 256) || workspace_bytes < GQA_INT4_WORKSPACE_BYTES)
    return set_error(GQA_ERR_INVALID_ARG, "workspace must be 256-byte aligned and of %d bytes at least",
                     GQA_INT4_WORKSPACE_BYTES);
  if (!launch) return GQA_OK;

  gqa::Int4DecodeParams p{};
  int sms;
  s = gqa::host_device(&p.err, &sms);
  if (s != GQA_OK) return s;
  const gqa::Knobs knobs = gqa::host_knobs();
  constexpr size_t kHeader = gqa::kInt4Counters * sizeof(int32_t);
  const int64_t fit = static_cast<int64_t>((GQA_INT4_WORKSPACE_BYTES - kHeader) / plan.slot_bytes);
  // no more CTAs than the longest lengths could keep busy (the lengths are device data)
  const int64_t tiles = static_cast<int64_t>(num_seqs) * num_kv_heads * n_rt *
                        (static_cast<int64_t>(max_blocks) * (page_size / kTile));
  int64_t grid = knobs.workers > 0 ? knobs.workers : static_cast<int64_t>(sms) * plan.ctas_per_sm;
  const int64_t limits[] = {fit, plan.max_ctas, (tiles + plan.warps - 1) / plan.warps};
  for (const int64_t limit : limits)
    if (grid > limit) grid = limit;

  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.pool = static_cast<const uint8_t*>(kv_pages);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.counters = static_cast<int32_t*>(workspace);
  p.slots = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kHeader);
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = group;
  p.q_len = q_len;
  p.rows = rows;
  p.n_rt = n_rt;
  p.page_size = page_size;
  p.tiles_per_page = page_size / kTile;
  p.max_blocks = max_blocks;
  p.num_pages = num_pages;
  p.scale = scale;
  p.wait_limit_ns = knobs.wait_limit_ns;
  p.arm_without_copy = knobs.arm_without_copy;
  if (p.tiles_per_page > 1) gqa::divisor_magic(static_cast<uint32_t>(p.tiles_per_page), &p.tpp_magic, &p.tpp_shift);
  s = cuda_status(gqa::launch_decode_int4(p, plan, head_dim, static_cast<int>(grid), static_cast<cudaStream_t>(stream), overlap),
                  "decode launch");
  if (s == GQA_OK) gqa::host_count_launches(1);
  return s;
}

}  // namespace

extern "C" {

gqa_status gqa_kv_quantize_int4(const void* k_pages, const void* v_pages, void* kv_pages, int num_pages,
                                int num_kv_heads, int page_size, int head_dim, void* stream) {
  if (num_pages < 0) return set_error(GQA_ERR_INVALID_ARG, "num_pages < 0");
  gqa_status s = check_pool(num_kv_heads, head_dim, page_size);
  if (s != GQA_OK || num_pages == 0) return s;
  s = check_rows(num_pages, num_kv_heads, page_size, 1);
  if (s != GQA_OK) return s;
  if (!k_pages || !v_pages || !kv_pages) return set_error(GQA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(kv_pages, 16))
    return set_error(GQA_ERR_INVALID_ARG, "the pools must be 16-byte aligned");
  const int64_t tiles = static_cast<int64_t>(num_pages) * num_kv_heads * (page_size / kTile);
  s = cuda_status(gqa::launch_kv_quantize_int4(k_pages, v_pages, kv_pages, tiles, head_dim, static_cast<cudaStream_t>(stream)),
                  "kv_quantize_int4 launch");
  if (s == GQA_OK) gqa::host_count_launches(1);
  return s;
}

gqa_status gqa_kv_dequantize_int4(const void* kv_pages, void* k_pages, void* v_pages, int num_pages, int num_kv_heads,
                                  int page_size, int head_dim, void* stream) {
  if (num_pages < 0) return set_error(GQA_ERR_INVALID_ARG, "num_pages < 0");
  gqa_status s = check_pool(num_kv_heads, head_dim, page_size);
  if (s != GQA_OK || num_pages == 0) return s;
  s = check_rows(num_pages, num_kv_heads, page_size, 1);
  if (s != GQA_OK) return s;
  if (!k_pages || !v_pages || !kv_pages) return set_error(GQA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(kv_pages, 16))
    return set_error(GQA_ERR_INVALID_ARG, "the pools must be 16-byte aligned");
  const int64_t tiles = static_cast<int64_t>(num_pages) * num_kv_heads * (page_size / kTile);
  s = cuda_status(gqa::launch_kv_dequantize_int4(kv_pages, k_pages, v_pages, tiles, head_dim, static_cast<cudaStream_t>(stream)),
                  "kv_dequantize_int4 launch");
  if (s == GQA_OK) gqa::host_count_launches(1);
  return s;
}

gqa_status gqa_kv_append_int4(const void* k_new, const void* v_new, void* kv_pages, const int32_t* block_table,
                              const int32_t* positions, int num_seqs, int num_kv_heads, int head_dim, int page_size,
                              int max_blocks_per_seq, int num_pages, void* stream) {
  return append_plain_int4(k_new, v_new, kv_pages, block_table, positions, num_seqs, num_kv_heads, head_dim, page_size,
                           max_blocks_per_seq, num_pages, stream);
}

size_t gqa_int4_workspace_bytes(void) { return GQA_INT4_WORKSPACE_BYTES; }

gqa_status gqa_paged_decode_attn_int4(const void* q, const void* kv_pages, const int32_t* block_table,
                                      const int32_t* seq_lens, void* out, int num_seqs, int num_heads,
                                      int num_kv_heads, int head_dim, int page_size, float scale,
                                      int max_blocks_per_seq, int num_pages, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  return decode(q, kv_pages, block_table, seq_lens, out, num_seqs, 1, num_heads, num_kv_heads, head_dim, page_size,
                scale, max_blocks_per_seq, num_pages, workspace, workspace_bytes, stream, false, true);
}

gqa_status gqa_paged_multi_query_attn_int4(const void* q, const void* kv_pages, const int32_t* block_table,
                                           const int32_t* seq_lens, void* out, int num_seqs, int q_len, int num_heads,
                                           int num_kv_heads, int head_dim, int page_size, float scale,
                                           int max_blocks_per_seq, int num_pages, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  return decode(q, kv_pages, block_table, seq_lens, out, num_seqs, q_len, num_heads, num_kv_heads, head_dim, page_size,
                scale, max_blocks_per_seq, num_pages, workspace, workspace_bytes, stream, false, true);
}

gqa_status gqa_decode_step_int4(const void* q, const void* k_new, const void* v_new, const float* cos_sin, void* q_rot,
                                void* kv_pages, const int32_t* block_table, const int32_t* positions,
                                const int32_t* seq_lens, void* out, int num_seqs, int num_heads, int num_kv_heads,
                                int head_dim, int rotary_dim, int interleaved, int max_positions, int page_size,
                                float scale, int max_blocks_per_seq, int num_pages, void* workspace,
                                size_t workspace_bytes, void* stream) {
  const void* attended = cos_sin != nullptr ? q_rot : q;
  // both halves are checked before anything is launched
  gqa_status s = decode(attended, kv_pages, block_table, seq_lens, out, num_seqs, 1, num_heads, num_kv_heads, head_dim,
                        page_size, scale, max_blocks_per_seq, num_pages, workspace, workspace_bytes, stream, true, false);
  if (s != GQA_OK) return s;
  if (cos_sin != nullptr)
    s = gqa_rope_kv_append_int4(q, k_new, v_new, cos_sin, q_rot, kv_pages, block_table, positions, nullptr, num_seqs,
                                num_seqs, num_heads, num_kv_heads, head_dim, rotary_dim, interleaved, max_positions,
                                static_cast<int64_t>(num_heads) * head_dim, static_cast<int64_t>(num_kv_heads) * head_dim,
                                static_cast<int64_t>(num_kv_heads) * head_dim, page_size, max_blocks_per_seq, num_pages,
                                stream);
  else
    s = append_plain_int4(k_new, v_new, kv_pages, block_table, positions, num_seqs, num_kv_heads, head_dim, page_size,
                          max_blocks_per_seq, num_pages, stream);
  if (s != GQA_OK) return s;
  // the attention reads q and the pool only after it has waited for the append
  return decode(attended, kv_pages, block_table, seq_lens, out, num_seqs, 1, num_heads, num_kv_heads, head_dim,
                page_size, scale, max_blocks_per_seq, num_pages, workspace, workspace_bytes, stream, true, true);
}

gqa_status gqa_rope_kv_append(const void* q, const void* k_new, const void* v_new, const float* cos_sin, void* q_out,
                              void* k_pages, void* v_pages, const int32_t* block_table, const int32_t* positions,
                              const int32_t* seq_ids, int num_tokens, int num_seqs, int num_heads, int num_kv_heads,
                              int head_dim, int rotary_dim, int interleaved, int max_positions, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, int page_size, int max_blocks_per_seq, int num_pages,
                              void* stream) {
  const gqa_status s = need_rotation(rotary_dim);
  if (s != GQA_OK) return s;
  return append(params(q, k_new, v_new, cos_sin, q_out, k_pages, v_pages, nullptr, nullptr, block_table, positions,
                       seq_ids, num_tokens, num_seqs, num_heads, num_kv_heads, rotary_dim, interleaved, max_positions,
                       q_stride, k_stride, v_stride, page_size, max_blocks_per_seq, num_pages),
                gqa::kCacheBf16, head_dim, static_cast<cudaStream_t>(stream));
}

gqa_status gqa_rope_kv_append_fp8(const void* q, const void* k_new, const void* v_new, const float* cos_sin,
                                  void* q_out, void* k_pages, void* v_pages, const float* k_scales,
                                  const float* v_scales, const int32_t* block_table, const int32_t* positions,
                                  const int32_t* seq_ids, int num_tokens, int num_seqs, int num_heads,
                                  int num_kv_heads, int head_dim, int rotary_dim, int interleaved, int max_positions,
                                  int64_t q_stride, int64_t k_stride, int64_t v_stride, int page_size,
                                  int max_blocks_per_seq, int num_pages, void* stream) {
  const gqa_status s = need_rotation(rotary_dim);
  if (s != GQA_OK) return s;
  return append(params(q, k_new, v_new, cos_sin, q_out, k_pages, v_pages, k_scales, v_scales, block_table, positions,
                       seq_ids, num_tokens, num_seqs, num_heads, num_kv_heads, rotary_dim, interleaved, max_positions,
                       q_stride, k_stride, v_stride, page_size, max_blocks_per_seq, num_pages),
                gqa::kCacheE4m3, head_dim, static_cast<cudaStream_t>(stream));
}

gqa_status gqa_rope_kv_append_int4(const void* q, const void* k_new, const void* v_new, const float* cos_sin,
                                   void* q_out, void* kv_pages, const int32_t* block_table, const int32_t* positions,
                                   const int32_t* seq_ids, int num_tokens, int num_seqs, int num_heads,
                                   int num_kv_heads, int head_dim, int rotary_dim, int interleaved, int max_positions,
                                   int64_t q_stride, int64_t k_stride, int64_t v_stride, int page_size,
                                   int max_blocks_per_seq, int num_pages, void* stream) {
  const gqa_status s = need_rotation(rotary_dim);
  if (s != GQA_OK) return s;
  return append(params(q, k_new, v_new, cos_sin, q_out, kv_pages, nullptr, nullptr, nullptr, block_table, positions,
                       seq_ids, num_tokens, num_seqs, num_heads, num_kv_heads, rotary_dim, interleaved, max_positions,
                       q_stride, k_stride, v_stride, page_size, max_blocks_per_seq, num_pages),
                gqa::kCacheInt4, head_dim, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
