/*
 * gqa_rope.h -- rotary position embedding of q and k fused with the append to the paged K/V
 * cache of gqa_decode.h (bf16 or e4m3 pools) or gqa_int4.h (4-bit pools).
 *
 * Row t of q, k_new, v_new is a new token of sequence s = seq_ids[t] (s = t when seq_ids is
 * NULL) at position p = positions[t].  With cos = cos_sin[p][i] and
 * sin = cos_sin[p][rotary_dim / 2 + i], i < rotary_dim / 2, channel pair (x1, x2) of every q
 * head and every k head becomes
 *
 *     x1 * cos - x2 * sin ,   x2 * cos + x1 * sin
 *
 * in fp32, each product and sum rounded on its own.  The pair is channels (i, i + rotary_dim / 2),
 * or (2 i, 2 i + 1) when interleaved != 0; channels >= rotary_dim and v pass unchanged.
 * The rotated q is rounded to bf16 into q_out; the rotated k row and the v row go to slot
 * p % page_size of page block_table[s][p / page_size]: rounded to bf16, or coded from their
 * fp32 values as gqa_kv_append_fp8 / gqa_int4.h code theirs.
 *
 *     q, q_out       [num_tokens, num_heads, head_dim]       bf16
 *     k_new, v_new   [num_tokens, num_kv_heads, head_dim]    bf16
 *     cos_sin        [max_positions, rotary_dim]             fp32
 *     positions      [num_tokens]                            int32
 *     seq_ids        [num_tokens]                            int32, or NULL
 *     block_table    [num_seqs, max_blocks_per_seq]          int32
 *
 * q_stride, k_stride, v_stride: elements between consecutive tokens (multiples of 8, at least
 * one token's elements): q, k and v may be views of one fused projection.  q_out is
 * contiguous and may be q itself when q is; otherwise it overlaps no input.
 *
 * The tokens may be one per sequence (a decode step), several (drafts) or whole prompts of
 * different lengths, in any order; no two of them may share a sequence and position (which
 * row is kept, or a mixture of both, is then unspecified).  A row with seq_ids[t] < 0 is
 * padding: skipped (its q, k_new and v_new rows may be read), its q_out row left as it was.  A seq_id >= num_seqs, a position outside
 * [0, max_blocks_per_seq * page_size) or >= max_positions, or a page id outside
 * [0, num_pages) skips the row likewise and sets GQA_ERR_DEVICE_BOUNDS in the device error
 * word.  No other byte of the pools is written.
 *
 * Requirements: head_dim in {64, 128}; page_size >= 1 (4-bit: a multiple of 16, <= 256);
 * rotary_dim a multiple of 16 in [16, head_dim]; q, q_out, k_new, v_new, cos_sin and the pools
 * 16-byte aligned; num_tokens >= 0 (0 launches nothing); num_heads >= 1.
 */
#ifndef GQA_ROPE_H_
#define GQA_ROPE_H_

#include <stdint.h>

#include "gqa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

gqa_status gqa_rope_kv_append(const void* q, const void* k_new, const void* v_new, const float* cos_sin, void* q_out,
                              void* k_pages, void* v_pages, const int32_t* block_table, const int32_t* positions,
                              const int32_t* seq_ids, int num_tokens, int num_seqs, int num_heads, int num_kv_heads,
                              int head_dim, int rotary_dim, int interleaved, int max_positions, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, int page_size, int max_blocks_per_seq,
                              int num_pages, void* stream);

/* e4m3 pools; k_scales, v_scales [num_kv_heads] fp32. */
gqa_status gqa_rope_kv_append_fp8(const void* q, const void* k_new, const void* v_new, const float* cos_sin,
                                  void* q_out, void* k_pages, void* v_pages, const float* k_scales,
                                  const float* v_scales, const int32_t* block_table, const int32_t* positions,
                                  const int32_t* seq_ids, int num_tokens, int num_seqs, int num_heads,
                                  int num_kv_heads, int head_dim, int rotary_dim, int interleaved, int max_positions,
                                  int64_t q_stride, int64_t k_stride, int64_t v_stride, int page_size,
                                  int max_blocks_per_seq, int num_pages, void* stream);

/* A 4-bit pool (gqa_int4.h). */
gqa_status gqa_rope_kv_append_int4(const void* q, const void* k_new, const void* v_new, const float* cos_sin,
                                   void* q_out, void* kv_pages, const int32_t* block_table, const int32_t* positions,
                                   const int32_t* seq_ids, int num_tokens, int num_seqs, int num_heads,
                                   int num_kv_heads, int head_dim, int rotary_dim, int interleaved, int max_positions,
                                   int64_t q_stride, int64_t k_stride, int64_t v_stride, int page_size,
                                   int max_blocks_per_seq, int num_pages, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_ROPE_H_ */
