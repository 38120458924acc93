/*
 * bitdelta_block.h — the operators between a decoder block's delta linears
 * (include/bitdelta.h): the norms around a sub-block with its residual, the
 * rotary append of new keys and values to a paged cache, and the attention
 * that reads that cache.  With the linears they are all of a served model's
 * block but the gated activation between its last two projections:
 *
 *   x            = bitdelta_add_norm                 (input norm)
 *   qkv          = bitdelta_linear_grouped(x)        (QKV projection)
 *   q            = bitdelta_kv_append(qkv)           (rotary, cache)
 *   o            = bitdelta_attention(q)
 *   a            = bitdelta_linear_grouped(o)        (O projection)
 *   h, x         = bitdelta_add_norm(a, h)           (residual, next norm)
 *
 * The rules common to every call of bitdelta.h hold here as well: device
 * pointers owned by the caller, asynchronous on `stream`, no device memory
 * allocated, arguments checked on the host before any launch, device-side
 * faults reported by bitdelta_check_error.  bf16 tensors start on a 16-byte
 * boundary and are contiguous.
 *
 * Stream order: these kernels are launched with programmatic dependent launch
 * and touch no tensor of the caller's before the kernels ahead of them on the
 * stream have completed.
 */
#ifndef BITDELTA_BLOCK_H_
#define BITDELTA_BLOCK_H_

#include "bitdelta.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BD_RESIDUAL_BF16 = 0, BD_RESIDUAL_F32 = 1 } bd_residual_type;

/* Which elements of a head rotate together: i and i + rot_dim/2, or 2i and
 * 2i + 1. */
typedef enum { BD_ROPE_HALVES = 0, BD_ROPE_PAIRS = 1 } bd_rope_style;

/*
 * Residual addition with the norms after and before a sub-block:
 *
 *   b = y                                   (post_table NULL)
 *     = y / sqrt(mean(y²) + eps) · w_post   (else)
 *   h = residual + scale · gate · b         (gate NULL: 1)
 *   x = h / sqrt(mean(h²) + eps) · w_pre
 *
 * per row of y [M, d], all in fp32; x is formed from h before h is rounded to
 * the residual's type.
 *   residual, residual_out   [M, d] of `rtype`; residual NULL reads as zero,
 *                residual_out NULL does not store h, and the two may be the
 *                same buffer.
 *   gate         bf16, NULL, [d] (gate_stride 0) or [M, d] (gate_stride d).
 *   pre_table, post_table   device arrays [n_tab] of device pointers to bf16
 *                [d] weights: slot 0 the base model's, slot v variant v's
 *                (norm weights are kept per variant, not as 1-bit deltas).
 *                A null entry or one off a 16-byte boundary sets
 *                BD_ERR_DEVICE_BOUNDS and reads as ones.
 *   seg_offsets [n_seg+1], seg_variant [n_seg]   device int32, as in
 *                bitdelta_linear_grouped; both NULL with n_seg = 0: every row
 *                takes slot 0.  Rows of no segment are left alone, and all rows
 *                where the offsets decrease or leave [0, M], which sets
 *                BD_ERR_DEVICE_BOUNDS.  A variant
 *                id outside [0, n_tab) sets BD_ERR_DEVICE_BOUNDS and reads as
 *                slot 0.
 *   x_out        bf16 [M, d], or NULL (then pre_table may be NULL).
 * d must be a positive multiple of 8, at most 65536.
 */
bd_status bitdelta_add_norm(const uint16_t* y, int64_t M, int64_t d, const void* residual,
                            void* residual_out, bd_residual_type rtype, const uint16_t* gate,
                            int64_t gate_stride, float scale, float eps,
                            const uint16_t* const* pre_table,
                            const uint16_t* const* post_table, int32_t n_tab,
                            const int32_t* seg_offsets, const int32_t* seg_variant,
                            int32_t n_seg, uint16_t* x_out, bd_stream_t stream);

/*
 * A batch of sequences over one layer-independent page table.  Sequence s
 * brings query tokens seq_offsets[s] .. seq_offsets[s+1] - 1 of the batch's
 * n_tokens rows; kv_len[s] counts its keys including theirs, so its query
 * token i stands at position kv_len[s] - q_len[s] + i.  Keys and values of
 * position p lie in page page_table[s][p / page_size] at offset p % page_size.
 *
 * A layer's cache: k_pages and v_pages bf16 [n_pages, n_kv_heads, page_size,
 * head_dim] (a page and head is one contiguous tile; element offsets are 64
 * bits wide).
 *
 * Groups (n_group > 0): consecutive sequences group_offsets[g] ..
 * group_offsets[g+1] - 1 share their first prefix_len[g] positions, i.e. their
 * page-table rows name the same pages there.  The shared part is then read
 * once for the whole group, through the first member's row.  The attention's
 * definition does not change; sequences outside every group share nothing.
 *
 * n_q_heads must be a multiple of n_kv_heads, at most 32 times as many and at
 * most 1024; n_tokens · n_kv_heads at most 2^28, kv_len · n_kv_heads and n_pages
 * · n_kv_heads · page_size below 2^31;
 * query head h reads key head h / (n_q_heads / n_kv_heads).  head_dim 64 or
 * 128; page_size 16, 32, 64 or 128.  max_q_len and max_kv_len are host bounds
 * of the lengths in device memory; a table that breaks them, or is not
 * sorted, sets BD_ERR_DEVICE_BOUNDS.
 */
typedef struct {
  int64_t n_tokens;
  int32_t n_seq;
  int32_t max_q_len, max_kv_len;
  int32_t n_q_heads, n_kv_heads, head_dim;
  int32_t page_size;
  int64_t n_pages;
  int64_t table_stride;         /* entries per row of page_table */
  const int32_t* seq_offsets;   /* device [n_seq + 1] */
  const int32_t* kv_len;        /* device [n_seq] */
  const int32_t* page_table;    /* device [n_seq, table_stride] */
  int32_t n_group;
  const int32_t* group_offsets; /* device [n_group + 1] */
  const int32_t* prefix_len;    /* device [n_group], multiples of page_size */
} bd_attention_batch;

/*
 * Rotary positions and the cache append.  qkv bf16 [n_tokens, (n_q_heads +
 * 2·n_kv_heads)·head_dim] (query heads, key heads, value heads).  The first
 * rot_dim elements of every query and key head are rotated by the angle of
 * the token's position: (a, b) -> (a·cos − b·sin, b·cos + a·sin) in fp32,
 * rounded once.  rope: fp32 [rope_rows, rot_dim], per position rot_dim/2
 * cosines, then rot_dim/2 sines.  Query heads go to q_out bf16 [n_tokens,
 * n_q_heads, head_dim], key and value heads to the token's place in the cache.
 * A token at a negative position (kv_len < q_len), or of no sequence, is
 * padding: its query is zero and nothing is appended.  A position past rope_rows or past the page
 * table's row, or a page outside [0, n_pages), sets BD_ERR_DEVICE_BOUNDS; the
 * query is then zero and nothing is appended for that token; a batch whose
 * lengths break its bounds or are not sorted has zero queries and appends nothing.
 * rot_dim: a multiple of 16, 0 .. head_dim.
 */
bd_status bitdelta_kv_append(const bd_attention_batch* batch, const uint16_t* qkv,
                             const float* rope, int64_t rope_rows, int32_t rot_dim,
                             bd_rope_style style, uint16_t* k_pages, uint16_t* v_pages,
                             uint16_t* q_out, bd_stream_t stream);

/*
 * The attention's plan: how a batch's work is cut over the device, computed
 * on the device from the lengths alone.  It holds for every layer until the
 * lengths change.  plan: device memory of bitdelta_attention_plan_bytes(batch)
 * bytes on a 256-byte boundary.
 */
size_t bitdelta_attention_plan_bytes(const bd_attention_batch* batch);
bd_status bitdelta_attention_plan(const bd_attention_batch* batch, void* plan, size_t plan_bytes,
                                  bd_stream_t stream);

/*
 * Causal attention over the paged cache:
 *
 *   out[t, h] = Σ_{p ≤ pos(t)} softmax_p(scale · q[t, h]·k_p) · v_p
 *
 * q, out bf16 [n_tokens, n_q_heads, head_dim]; lse fp32 [n_tokens, n_q_heads]
 * (the logarithm of the softmax's denominator) or NULL.  Scores, softmax
 * statistics and sums in fp32; the softmax weights are rounded to bf16 for
 * the product with the values.  A row with no key (a negative position)
 * gives zeros and an lse of −inf, a row whose query holds a NaN gives NaN in
 * both.  Positions past a sequence's kv_len are
 * never read as values, whatever the page holds there; within kv_len, keys
 * and values are expected finite, and values below 2^57 (a row's sums are kept
 * relative to a score that may lie 2^40 below its largest).
 *   plan         as made by bitdelta_attention_plan for the same batch.  A call
 *                uses a counter in it and leaves it as it was.
 *   workspace    device memory of bitdelta_attention_workspace_bytes(batch)
 *                bytes on a 256-byte boundary.  The host knows no lengths: with
 *                groups, every 256-row tile that the batch may hold has an fp32
 *                part per key head, and every token one (a group of 16 chunks of
 *                512 tokens, 64 and 8 heads of 128, 937 MB; 64 single tokens in
 *                two groups 108 MB; without groups 101 and 20 MB).
 *   Calls that can overlap on the GPU need plans and workspaces of their own.
 * scale must be positive and at most 2^127 (times log2 e it has to be finite).
 */
size_t bitdelta_attention_workspace_bytes(const bd_attention_batch* batch);
bd_status bitdelta_attention(const bd_attention_batch* batch, void* plan, size_t plan_bytes,
                             const uint16_t* q, const uint16_t* k_pages, const uint16_t* v_pages,
                             float scale, uint16_t* out, float* lse, void* workspace,
                             size_t workspace_bytes, bd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BITDELTA_BLOCK_H_ */
