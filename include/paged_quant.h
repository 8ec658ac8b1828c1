/*
 * paged_quant.h — the paged cache held in 8 bits: the write that quantises the
 * new tokens' keys and values, the read back to 16 bits, and the attention of
 * decode steps over it.  Half the bytes of a 16-bit cache, so twice the tokens
 * in the same pool and half the time where the cache's bytes bound a step.  On
 * one stream:
 *     paged_batch_tables              block tables, lengths, positions, slots
 *     paged_rope_quant_cache_write    q, k rotated; k, v stored as codes
 *     paged_decode_attn_quant         a decode step
 *   or, for a prompt's chunk,
 *     paged_quant_cache_read          the requests' pages in 16 bits
 *     paged_prefill_attn              over those pages (or _sinks)
 *
 * The cache.  A value is code x scale:
 *   k_cache, v_cache  PD_E4M3 pools, NHD or HND, any strides (innermost 1, the
 *            others multiples of 16), 16-byte aligned; K and V packed side by
 *            side are two views of one pool
 *   k_scale, v_scale  [num_blocks, page_size / 16, num_kv_heads] fp32, any
 *            strides above 0: one scale for each PD_SCALE_TOKENS = 16 tokens of a
 *            page (a block) and kv head
 * page_size is a multiple of 16.  A pool that was never written may hold
 * anything, NaN too: a request's blocks are those that its tokens were written
 * to.
 *
 * Streams, scratch, graph capture and errors are those of paged_decode.h: every
 * call is asynchronous on `stream`, allocates nothing, checks its arguments on
 * the host (PD_OK or a negative pd_status), and reports what only the device
 * can see in the status word, clamping or skipping the access.
 */
#ifndef PAGED_QUANT_H
#define PAGED_QUANT_H

#include "paged_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A further element type beside pd_dtype: 8-bit floats of 4 exponent and 3
 * mantissa bits, bias 7, largest 448, no infinities, NaN = 0x7f. */
#define PD_E4M3 4

#define PD_DEV_BAD_SCALE 0x200u /* paged_decode_attn_quant: the scale of a block with
                                   visible keys outside 2^-64 .. 2^32 */
#define PD_SCALE_TOKENS 16 /* tokens of a page that share a scale */
#define PD_RUN_DISTANCE 96 /* tokens before a run of a block's new tokens that
                              are looked through for another run of it */

/* ---- The write ----
 *
 * paged_rope_axes_cache_write into an 8-bit cache: q rotated to q_out (in its
 * own type), k rotated and v as they are, in fp32, quantised and stored at the
 * slots.  For a block (16 tokens of a page) and kv head whose new tokens have
 * the largest magnitude a,
 *     need  = 2^e, the smallest e >= -64 with a <= 448 x 2^e
 *     scale = need                  when the call writes the block's first token
 *                                   (the block starts anew: nothing it held counts)
 *           = max(scale, need)      else (an old scale that is not a positive
 *                                   finite number counts as 0)
 *     code  = x / scale rounded to the nearest code, ties to even
 * and where an old scale grew, the block's other codes are rounded to the new
 * one (code x old / new): a value is half a step of the new scale off what it was
 * held as.  A value that is written is at most 2^-4 of itself off, or 2^-10 x scale
 * where it is below 2^-6 x scale; each time that its block's scale grows after that
 * adds 2^-10 x the new scale at most, all of them together less than 2^-9 x the last
 * one.  (Scales are powers of two, so x / scale is exact, a code that stays above 2^-6
 * keeps its bits, and a call's result does not depend on how its sums are ordered.
 * The growth of an old scale that is none rounds every code.)  A scale never shrinks
 * before its block starts anew: a draft token that is taken back leaves it as it made
 * it.  Infinities are stored as 448 x scale and NaN as NaN; neither counts in a.
 *
 *   q, q_out      [T, Hq, D] fp16/bf16, or both NULL: k and v alone (num_q_heads
 *                 is then ignored); q_out may be q itself
 *   k, v          [T, Hkv, D], the type of q
 *   positions     [T], or [A, T] with rows of contiguous entries, A <= PD_MAX_AXES,
 *                 int32; cos_sin_cache as in paged_rope_cache_write; both NULL
 *                 with rot_dim = 0 (nothing is rotated: q is copied)
 *   pair_axis     [rot_dim / 2] host array of the pairs' axes, or NULL: axis 0
 *   slot_mapping  [T] int32: the cache slots, distinct, or -1 (padding: q is
 *                 rotated, nothing is stored).  The tokens of one block stand next
 *                 to one another, their slots ascending, as paged_batch_tables
 *                 lays them out; a call writes a block in one such run.  (Two runs
 *                 of a block further apart than PD_RUN_DISTANCE tokens are not
 *                 seen: what the block then holds is undefined until its first
 *                 token is written again.)
 *   rot_dim       0, or as in paged_rope_cache_write
 * Reported: a position outside the table (clamped) PD_DEV_BAD_POSITION; a slot
 * past the pool, in a run one that does not ascend (it and the rest of the run
 * are not written), or a run whose block one of the PD_RUN_DISTANCE tokens before
 * it has a slot of (it is not written): PD_DEV_BAD_SLOT. */
PD_API int paged_rope_quant_cache_write(const pd_tensor *q, const pd_tensor *k, const pd_tensor *v,
                                        const pd_tensor *positions, const pd_tensor *slot_mapping,
                                        const pd_tensor *cos_sin_cache, const uint8_t *pair_axis,
                                        pd_tensor *q_out, pd_tensor *k_cache, pd_tensor *v_cache,
                                        pd_tensor *k_scale, pd_tensor *v_scale, int num_q_heads,
                                        int num_kv_heads, int head_size, int rot_dim,
                                        int page_size, int layout, int is_neox, void *stream);

/* ---- The read ----
 *
 * Pages of requests in 16 bits: for request s and its logical page j below
 * ceil(seq_lens[s] / page_size), the tokens of page block_table[s][j] that the
 * request has go to page out_table[s][j] of a staging pool,
 *     out = code x scale, rounded once to the pool's type,
 * which paged_prefill_attn (or any call on a 16-bit pool) takes with out_table
 * as its block table.  A negative entry of either table leaves the page out
 * (pages before a window; pages staged earlier), and the slots past a request's
 * last token are left as they were.  Every entry of the tables is looked at: a
 * call over tables far wider than the requests takes longer.
 *   block_table, out_table  [S, W] int32
 *   seq_lens                [S] int32
 *   k_out, v_out            fp16/bf16 pools [num_out_blocks, ...] in the same
 *                           layout, head count and page size; out_table's entries
 *                           are distinct
 * Reported: a page id past either pool (left out) PD_DEV_BAD_PAGE; a length past
 * the table (clamped) PD_DEV_BAD_SEQLEN. */
PD_API int paged_quant_cache_read(const pd_tensor *k_cache, const pd_tensor *v_cache,
                                  const pd_tensor *k_scale, const pd_tensor *v_scale,
                                  const pd_tensor *block_table, const pd_tensor *seq_lens,
                                  const pd_tensor *out_table, pd_tensor *k_out, pd_tensor *v_out,
                                  int num_kv_heads, int head_size, int page_size, int layout,
                                  void *stream);

/* ---- Decode attention ----
 *
 * paged_decode_attn / _varlen / _sinks over an 8-bit cache: 1 to 8 query tokens
 * a request (the same number each, or by query_start), every key before a
 * token or, with window > 0, the newest `window` ones and the first `sinks`:
 *     out = softmax_k(scale * q . (k_scale k_code)) . (v_scale v_code)
 * in fp32 (the softmax weights are rounded to 16 bits for the second product),
 * rounded to q's type; 0 where no key is visible.  Scales of visible keys are
 * positive, 2^-64 to 2^32 (any such numbers, not powers of two alone; values up to
 * 448 x 2^32, where the write takes any that its input holds); others are reported
 * as PD_DEV_BAD_SCALE, and the rows that see their keys are undefined.  Keys and
 * values that some row sees are finite.  What no row sees may be anything.
 *   q, out       [S * max_query_len, Hq, D], or [T, Hq, D] with query_start
 *   block_table, seq_lens, query_start (or NULL), window, sinks, scale: as in
 *                paged_decode_attn_sinks
 *   scratch      paged_decode_scratch_bytes / _init, as for paged_decode_attn;
 *                NULL or a small one: fewer CTAs share the keys
 * The launch runs one wave of CTAs that take equal shares of all requests'
 * keys (past 448 requests a wave for each 448 of them); paged_decode_plan_quant gives
 * its numbers (path 7).  How many rows a CTA takes is chosen by the table's
 * width: the lengths are on the device. */
PD_API int paged_decode_attn_quant(const pd_tensor *q, const pd_tensor *k_cache,
                                   const pd_tensor *v_cache, const pd_tensor *k_scale,
                                   const pd_tensor *v_scale, const pd_tensor *block_table,
                                   const pd_tensor *seq_lens, const pd_tensor *query_start,
                                   pd_tensor *out, int num_q_heads, int num_kv_heads,
                                   int head_size, int page_size, int max_query_len, int window,
                                   int sinks, float scale, int layout, pd_scratch *scratch,
                                   void *stream);

/* The launch plan of that call, on the host only: rows_per_cta packed rows in
 * row_groups groups, grid_x CTAs (grid_y > 1: so many runs of sequences, each
 * with its own grid_x), merge = 1 where shares may cut a unit (0: the scratch
 * holds too few parts, every (sequence, kv head, row group) is one CTA's),
 * key_groups warps that take alternate steps of blocks, scratch_needed. */
PD_API int paged_decode_plan_quant(int num_seqs, int num_q_heads, int num_kv_heads, int head_size,
                                   int page_size, int max_query_len, int window, int sinks,
                                   int block_table_width, int num_sms, const pd_scratch *scratch,
                                   pd_plan *plan);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_QUANT_H */
