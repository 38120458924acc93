/*
 * bitdelta_decode.h — the end of a serving step, beside the decoder block's
 * operators (include/bitdelta_block.h): the next tokens from the logits, and a
 * paged cache held to a budget by the attention weight that its keys get:
 *
 *   q    = bitdelta_kv_append_at(qkv)        per layer: positions go on where an
 *   o    = bitdelta_attention(q) -> lse        eviction shortened the cache
 *          bitdelta_kv_weigh(q, lse)         adds what each key was looked at
 *   ...
 *   tok  = bitdelta_sample(logits)           per step
 *   ...
 *          bitdelta_kv_evict(keep)           per layer, when the budget is full
 *          bitdelta_kv_evict_lengths(keep)   once, after the last layer
 *
 * The rules of bitdelta.h and bitdelta_block.h hold here as well: device
 * pointers owned by the caller, asynchronous on `stream`, no device memory
 * allocated, arguments checked on the host before any launch, device-side
 * faults reported by bitdelta_check_error, no tensor touched before the kernels
 * ahead on the stream have completed.
 */
#ifndef BITDELTA_DECODE_H_
#define BITDELTA_DECODE_H_

#include "bitdelta_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A token per row of logits, from one given random number a row.
 *
 *   logits       bf16 [M, V], rows `row_stride` elements apart (>= V); rows may
 *                begin on any 2-byte boundary.
 *   u            fp32 [M], uniform in [0, 1); clamped to it.
 *   temperature  fp32 [M] or NULL (1).  0 takes the largest logit.
 *   top_k        int32 [M] or NULL; 0 and below: no cut.
 *   top_p        fp32 [M] or NULL; 1 and above: no cut.
 *   min_p        fp32 [M] or NULL; 0 and below: no cut.
 *
 * A row's tokens are taken in the order of their logits, the largest first,
 * equal ones by their index.  w = exp((logit − largest)/temperature).  Kept are
 * the first n of them, n being the least of top_k, the least number whose w sum
 * to top_p of the top_k tokens' sum, and the number with w >= min_p; one at
 * least.  The token is the first whose sum of w, with those before it, is above
 * u times the kept tokens' sum, and prob its w over that sum.
 *   tokens       int32 [M]
 *   prob         fp32 [M], or NULL
 * Sums are exact to about 2^-40 of the largest w and do not depend on the
 * order of the work.  A NaN or −inf logit is never taken; a row without
 * another gives −1 and 0.  +inf logits share all the weight.  A NaN parameter
 * or a temperature below 0 sets BD_ERR_DEVICE_BOUNDS, and its row gives −1 and 0.
 * V: 1 .. 524032.
 */
bd_status bitdelta_sample(const uint16_t* logits, int64_t M, int64_t V, int64_t row_stride,
                          const float* u, const float* temperature, const int32_t* top_k,
                          const float* top_p, const float* min_p, int32_t* tokens, float* prob,
                          bd_stream_t stream);

/*
 * bitdelta_kv_append for sequences that lost tokens to an eviction: a token in
 * slot p of sequence s is rotated by the angle of position p + pos_offset[s]
 * (device int32 [n_seq]; NULL: 0) and stored in slot p.  The position, not the
 * slot, has to lie inside rope's rows.
 */
bd_status bitdelta_kv_append_at(const bd_attention_batch* batch, const int32_t* pos_offset,
                                const uint16_t* qkv, const float* rope, int64_t rope_rows,
                                int32_t rot_dim, bd_rope_style style, uint16_t* k_pages,
                                uint16_t* v_pages, uint16_t* q_out, bd_stream_t stream);

/*
 * A layer's table of attention weights: weights fp32 and positions int32
 * [n_pages, n_kv_heads, page_size], beside its cache's slots.  For key head h
 * and slot p of a sequence
 *
 *   a = Σ_t Σ_j exp(scale · q[t, j]·k_p − lse[t, j])
 *
 * over the sequence's last `window` query tokens of this step (0: all) that see
 * the slot, and the query heads j of h.  A slot of the step's own tokens begins
 * with it (weights = a, positions = p + pos_offset[s]), any other one's weight
 * grows by a.  A group's shared slots get the sum over all members' tokens,
 * once.  Slots outside of the batch's keys are left alone.  Call it once per
 * step and layer, after the attention that gave lse; q, lse and scale as there.
 * A row whose lse is not finite adds nothing.  Sums are in fp32, in an order
 * that the batch alone decides.
 *   scale        2^-100 and more.
 *   pos_offset   device int32 [n_seq]: tokens that evictions took from the
 *                sequence; NULL: 0.
 *   workspace    device memory of bitdelta_kv_weigh_workspace_bytes(batch) bytes
 *                (0.6 MB) on a 256-byte boundary.  Calls that can overlap on the
 *                GPU need workspaces of their own.
 * A batch whose tables break its bounds, or a group with a prefix_len that is
 * not a multiple of page_size or reaches into a member's query tokens (a member
 * without any may have fewer keys), sets
 * BD_ERR_DEVICE_BOUNDS and changes nothing; a page outside [0, n_pages) sets it and
 * is skipped.  Two sequences that share a page outside of a group are not
 * supported (the page would have two writers).
 */
size_t bitdelta_kv_weigh_workspace_bytes(const bd_attention_batch* batch);
bd_status bitdelta_kv_weigh(const bd_attention_batch* batch, const uint16_t* q, const float* lse,
                            const uint16_t* k_pages, float scale, int32_t window,
                            const int32_t* pos_offset, float* weights, int32_t* positions,
                            void* workspace, size_t workspace_bytes, bd_stream_t stream);

/*
 * Eviction: a sequence of more than keep[s] keys goes down to
 *
 *   n' = max(keep[s], its group's prefix_len)      (keep[s] < 0: it stays as it is)
 *
 * slots per key head.  A group's shared slots stay.  Of the others, first those
 * with position >= kv_len[s] + pos_offset[s] − recent (the last `recent` tokens)
 * or position < sink stay, then those of the largest weight; equal ones by their
 * slot, the lowest first, a NaN weight last.  Each key head chooses for itself.
 * Attention does not depend on the order of the keys: what stays in a slot below
 * n' stays where it is, and the i-th of the others that stay (in the order of
 * slots) moves into the i-th slot below n' that came free, with its weight and
 * position.  Slots from n' on are left as they were.
 *   keep         device int32 [n_seq]
 *   weights_out, positions_out   may be weights and positions themselves, or
 *                other tables, which then get every slot below n' of every
 *                sequence of the batch (below kv_len[s] of one that stays).
 * kv_len is not changed: every layer is cut with the same lengths, and
 * bitdelta_kv_evict_lengths then sets them.  The batch's query tokens are not
 * looked at.  The tables start on 16-byte boundaries.  max_kv_len: at most 344064.
 * A kv_len outside the batch's bounds (or past its page table's row), or a page
 * outside [0, n_pages) among those that are chosen from, sets BD_ERR_DEVICE_BOUNDS
 * and leaves the sequence as it was, with its length; of other
 * weights_out and positions_out some of its slots may have been set.  Two
 * sequences that share a page outside of a group are not supported.
 */
bd_status bitdelta_kv_evict(const bd_attention_batch* batch, const int32_t* keep, int32_t recent,
                            int32_t sink, const int32_t* pos_offset, uint16_t* k_pages,
                            uint16_t* v_pages, const float* weights, const int32_t* positions,
                            float* weights_out, int32_t* positions_out, bd_stream_t stream);

/*
 * The lengths after an eviction of every layer: kv_len_out[s] = n' and
 * pos_offset[s] += kv_len[s] − n'.  kv_len_out may be the batch's own kv_len;
 * the attention's plan has to be made again.  What the eviction refuses is
 * refused here too, for the same batch, keep and n_pages: a sequence that it left as
 * it was sets BD_ERR_DEVICE_BOUNDS and keeps its length and offset (kv_len_out[s] =
 * kv_len[s]).  With n_pages = 0 or no page_table the pages are not looked at.
 */
bd_status bitdelta_kv_evict_lengths(const bd_attention_batch* batch, const int32_t* keep,
                                    int32_t* kv_len_out, int32_t* pos_offset,
                                    bd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BITDELTA_DECODE_H_ */
