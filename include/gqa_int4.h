/*
 * gqa_int4.h -- a 4-bit paged K/V cache for gqa_decode.h: writing it, reading it back, and
 * decode attention over it.
 *
 * For every token and kv head, K and V are cut into groups of 64 channels.  A group holds
 * its minimum and its step in bf16 and one code in 0..15 per channel:
 *
 *     low  = bf16(min x)                     step = bf16((max x - min x) / 15)
 *     code = clamp(rint((x - low) / step), 0, 15)   (0 where step is 0)
 *     cached value = code * step + low
 *
 * with every operation in IEEE fp32 (round to nearest even).  A group with a non-finite
 * member, or whose range is not finite, reads back as NaN throughout.  A token and kv head
 * takes 9/8 * head_dim bytes for K and V together (bf16: 4 * head_dim).
 *
 *     kv_pages   [num_pages, num_kv_heads, page_size / 16, 18 * head_dim]   bytes
 *
 * holds K and V in one pool, in tiles of 16 tokens of one (page, kv head); token t of a
 * sequence is token t % 16 of tile (t % page_size) / 16 of its page.  Inside a tile, with
 * groups = head_dim / 64:
 *
 *   [0, 8 D)       K codes: token tau, channel 64 r + 16 q + 8 b + n (r < groups, q < 4,
 *                  b < 2, n < 8) is nibble n of the 32-bit little-endian word at
 *                  tau * D / 2 + q * D / 8 + r * 8 + b * 4
 *   [8 D, 16 D)    V codes: token tau, channel 64 u + 8 g + n (u < groups, g < 8) is nibble
 *                  n of the word at 8 D + (g / (8 / groups)) * 512 + row * 32 +
 *                  (g % (8 / groups)) * 4 * groups + u * 4, where
 *                  row = tau / 8 * 8 + tau % 2 * 4 + tau % 8 / 2
 *   [16 D, 18 D)   token tau, K (kv = 0) or V (kv = 1), group r: the bf16 pair (step, low)
 *                  at 16 D + tau * 8 groups + kv * 4 groups + 4 r
 *
 * Each byte belongs to one token, so appending a token never touches another's bytes.  The
 * order inside a tile is the order in which the attention kernel's threads read it.
 *
 * Conventions, errors and the device error word are gqa_decode.h's.
 */
#ifndef GQA_INT4_H_
#define GQA_INT4_H_

#include <stddef.h>
#include <stdint.h>

#include "gqa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gqa_kv_quantize_int4 -- a whole bf16 pool pair into a 4-bit pool: k_pages, v_pages
 *   [num_pages, num_kv_heads, page_size, head_dim] bf16 -> kv_pages.
 * gqa_kv_dequantize_int4 -- the cached values of a whole 4-bit pool, rounded to bf16, as a
 *   pair of bf16 pools.
 * Requirements: head_dim in {64, 128}; page_size a multiple of 16 in [16, 256]; all three
 * pools 16-byte aligned; num_pages >= 0 (0 launches nothing).
 */
gqa_status gqa_kv_quantize_int4(const void* k_pages, const void* v_pages, void* kv_pages, int num_pages,
                                int num_kv_heads, int page_size, int head_dim, void* stream);
gqa_status gqa_kv_dequantize_int4(const void* kv_pages, void* k_pages, void* v_pages, int num_pages,
                                  int num_kv_heads, int page_size, int head_dim, void* stream);

/*
 * gqa_kv_append_int4 -- gqa_kv_append into a 4-bit pool: k_new, v_new [num_seqs,
 * num_kv_heads, head_dim] bf16 to positions[b].  (With the position rotation on the way:
 * gqa_rope_kv_append_int4 in gqa_rope.h.)
 */
gqa_status gqa_kv_append_int4(const void* k_new, const void* v_new, void* kv_pages, const int32_t* block_table,
                              const int32_t* positions, int num_seqs, int num_kv_heads, int head_dim, int page_size,
                              int max_blocks_per_seq, int num_pages, void* stream);

/*
 * Workspace of the attention calls below: GQA_INT4_WORKSPACE_BYTES of device memory owned by
 * the caller, 256-byte aligned, zeroed once before its first use.  Every call leaves it ready
 * for the next one, of any shape (a call that reported GQA_ERR_TIMEOUT included).  Calls that
 * may overlap in time -- on two streams, or in two graphs replayed at once -- need a workspace
 * each.
 */
#define GQA_INT4_WORKSPACE_BYTES (16 << 20)
size_t gqa_int4_workspace_bytes(void);

/*
 * gqa_paged_decode_attn_int4 -- gqa_paged_decode_attn over a 4-bit pool: the definition at
 * the top of gqa_decode.h with K_b, V_b the cached values.
 * gqa_paged_multi_query_attn_int4 -- gqa_paged_multi_query_attn likewise: q, out
 * [num_seqs, q_len, num_heads, head_dim]; q_len * (num_heads / num_kv_heads) <= 128 when
 * q_len > 1.
 *
 * Scores and sums are held in fp32.  q is scaled by a power of two per row and held in fp16,
 * which is exact for elements within 2^-28 of the row's largest; the products of the softmax
 * weights with the steps of V are rounded to fp16.  A row that sees a token and whose q holds a
 * non-finite element is NaN.  Slots at or beyond seq_lens[b] and unused pages may hold any bits.
 * Range: q, K and scale of any finite size with |scale * q| < 2^100 for every element of q and
 * scores, |scale| * sum |q| |k|, within fp32's range; V with |v| times the number of tokens up to
 * 2^115.  Beyond it an output may be anything.  Values of V below 2^-110 are off by up to 2^-136
 * absolutely per token that a row sees.
 * Time against the bf16 cache: less where sequences are long and a kv head has up to 16 query
 * rows (32 sequences of 512 to 4096 tokens, 4 rows: 33 us and 57), more in the
 * smallest calls (two sequences of 17 and 40 tokens: 6.6 us and 5.1), and more for a batch with
 * very many rows a kv head (64 sequences of 8192 tokens, 96 rows: 144 us, 57 over bf16, 83 over
 * e4m3).
 * Requirements as gqa_paged_decode_attn; q and out 16-byte aligned; out overlaps no input; num_heads at
 * most 2^19 - 1.
 */
gqa_status gqa_paged_decode_attn_int4(const void* q, const void* kv_pages, const int32_t* block_table,
                                      const int32_t* seq_lens, void* out, int num_seqs, int num_heads,
                                      int num_kv_heads, int head_dim, int page_size, float scale,
                                      int max_blocks_per_seq, int num_pages, void* workspace, size_t workspace_bytes,
                                      void* stream);
gqa_status gqa_paged_multi_query_attn_int4(const void* q, const void* kv_pages, const int32_t* block_table,
                                           const int32_t* seq_lens, void* out, int num_seqs, int q_len, int num_heads,
                                           int num_kv_heads, int head_dim, int page_size, float scale,
                                           int max_blocks_per_seq, int num_pages, void* workspace,
                                           size_t workspace_bytes, void* stream);

/*
 * gqa_decode_step_int4 -- one decode step: append this step's K/V rows at positions[b], then
 * attend over seq_lens[b] tokens; the attention launch overlaps the append.
 *   cos_sin != NULL: q and k_new are rotated on the way (gqa_rope_kv_append_int4 with
 *     rotary_dim, interleaved and max_positions; q_rot [num_seqs, num_heads, head_dim]
 *     receives the rotated q, and may be q itself).
 *   cos_sin == NULL: no rotation; rotary_dim, interleaved, max_positions and q_rot are not
 *     looked at.
 */
gqa_status gqa_decode_step_int4(const void* q, const void* k_new, const void* v_new, const float* cos_sin,
                                void* q_rot, void* kv_pages, const int32_t* block_table, const int32_t* positions,
                                const int32_t* seq_lens, void* out, int num_seqs, int num_heads, int num_kv_heads,
                                int head_dim, int rotary_dim, int interleaved, int max_positions, int page_size,
                                float scale, int max_blocks_per_seq, int num_pages, void* workspace,
                                size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_INT4_H_ */
