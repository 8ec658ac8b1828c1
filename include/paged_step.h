/*
 * paged_step.h — the calls around and beside paged_decode.h that a serving
 * step makes: attention over a sliding window whose first tokens stay
 * visible (sinks), the tables of a batch built on the GPU from its requests'
 * lengths, and the rotary embedding with a position per axis.  On one stream:
 *     paged_batch_tables            block tables, starts, lengths, positions, slots
 *     (the model's projections)
 *     paged_rope_axes_cache_write   q, k rotated; k, v stored at the slots
 *     paged_decode_attn_sinks       or paged_prefill_attn_sinks
 * A decode step makes no host round trip.  A prefill takes a work list that
 * paged_prefill_plan_sinks makes on the host from the host's copy of the
 * starts and lengths (known before the tables are: they are the lengths that
 * paged_batch_tables is given, summed), and that is copied to the device.
 *
 * Types, layouts, scratch, streams, graph capture and errors are those of
 * paged_decode.h: every call is asynchronous on `stream`, allocates nothing,
 * checks its arguments on the host (PD_OK or a negative pd_status), and
 * reports what only the device can see in the status word, clamping the
 * access instead of faulting.
 */
#ifndef PAGED_STEP_H
#define PAGED_STEP_H

#include "paged_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Window with sinks ----
 *
 * Attention as in paged_decode.h, but a query row that sees n keys (n = L -
 * q_len + i + 1) sees the key k of its sequence when
 *     k < n  and  (k >= n - window  or  k < sinks):
 * the first `sinks` tokens stay visible beside the sliding window of the
 * newest `window` keys.  Where both ranges meet, a key counts once.
 * window = 0 is full causal attention (sinks then change nothing), sinks = 0
 * the plain window: those calls are the ones of paged_decode.h.
 * The library reads block_table only for pages that hold visible keys: the
 * entries between the sinks' last page and the window's first one may be
 * anything (the pages may have been freed).  Keys and values that no row of
 * a request sees may be anything too; those that some row sees are finite
 * (a row's zero weight times an infinity in a key of another row is NaN). */

/* The decode call: paged_decode_attn_opts, or with query_start
 * paged_decode_attn_varlen, with sinks.
 *   query_start  [S + 1] int32 device array, or NULL (uniform: sequence s owns
 *                the rows s * max_query_len ..)
 *   sinks        >= 0 keys
 *   scratch      paged_decode_scratch_bytes / _init, as for paged_decode_attn
 *   opts         may be NULL; with sinks and a window, paths 2 and 3 are not
 *                built (PD_EINVAL), and path 6 asks for the window kernel below
 *                (PD_EINVAL where it does not serve: one sequence or more than
 *                1024, head size 512, more than 56 rows to a kv head, another
 *                knob set, too little scratch) */
PD_API int paged_decode_attn_sinks(const pd_tensor *q, const pd_tensor *k_cache,
                                   const pd_tensor *v_cache, const pd_tensor *block_table,
                                   const pd_tensor *seq_lens, const pd_tensor *query_start,
                                   pd_tensor *out, int num_q_heads, int num_kv_heads,
                                   int head_size, int page_size, int max_query_len, int window,
                                   int sinks, float scale, int layout, pd_scratch *scratch,
                                   void *stream, const pd_options *opts);

/* The launch plan of that call, on the host only.  A batch that fills the GPU
 * more than once and sets no knob is mostly planned as path 6: one wave of grid_x
 * CTAs that each take an equal share of the blocks of every (sequence, kv
 * head), cut where the shares end (grid_y = 1; seg_blocks, the most blocks of
 * one; max_segments and max_parts = grid_x).  Its scratch need is two parts
 * per CTA. */
PD_API int paged_decode_plan_sinks(int num_seqs, int num_q_heads, int num_kv_heads, int head_size,
                                   int page_size, int max_query_len, int window, int sinks,
                                   int block_table_width, int num_sms, const pd_scratch *scratch,
                                   const pd_options *opts, pd_plan *plan);

/* The prefill work list and call with sinks (paged_prefill_plan,
 * paged_prefill_attn; scratch from paged_prefill_scratch_bytes).  The plan's
 * loads are those of the window with sinks; a plan made for another window
 * or sinks gives the same outputs but for their rounding, less evenly spread
 * (tiles of other rows may be another kernel's).  At head sizes 64 to
 * 256, with up to 128 q heads to a kv head (at 128 at least 5/8 of a power of
 * two), the plan keeps its tiles whole unless they are few and long: the rows
 * of 256 / G' tokens (128 / G' at head size 256), G' the q heads to a kv head
 * rounded up to a power of two, are then a tile (info.tile_rows).  But for
 * PD_PREFILL_TILE_ROWS_D128 at head size 128 such a plan wants q's strides above
 * 0 (else PD_EALIGN), and T G' of at most 2^31 - 1. */
PD_API int paged_prefill_plan_sinks(const int32_t *query_start, const int32_t *seq_lens,
                                    int num_seqs, int num_q_heads, int num_kv_heads,
                                    int head_size, int window, int sinks, int num_sms,
                                    pd_prefill_item *items, int64_t capacity,
                                    pd_prefill_plan_info *info);
PD_API int paged_prefill_attn_sinks(const pd_tensor *q, const pd_tensor *k_cache,
                                    const pd_tensor *v_cache, const pd_tensor *block_table,
                                    const pd_tensor *seq_lens, const pd_tensor *query_start,
                                    const pd_tensor *work, const pd_prefill_plan_info *info,
                                    pd_tensor *out, int num_q_heads, int num_kv_heads,
                                    int head_size, int page_size, int window, int sinks,
                                    float scale, int layout, pd_scratch *scratch, void *stream);

/* ---- The tables of a batch ----
 *
 * For requests s = 0 .. S-1 with c_s = context_lens[s] cached tokens and q_s
 * = query_lens[s] new ones (0: no token in this step), in one launch:
 *     query_start[s]  = q_0 + .. + q_{s-1}             (query_start[S]: all)
 *     seq_lens[s]     = c_s + q_s
 *   new pages, when free_pages is given: request s takes
 *     need_s = ceil((c_s + q_s) / P) - ceil(c_s / P)
 *   pages of the list in request order, from f_s = cursor + need_0 + .. +
 *   need_{s-1} on:
 *     block_table[s][ceil(c_s / P) + j] = free_pages[f_s + j],  j < need_s
 *     next_cursor     = cursor + need_0 + .. + need_{S-1}
 *   token t = query_start[s] + i, at p = c_s + i of its sequence:
 *     positions[a][t] = p + position_delta[s]          (every axis a)
 *     slot_mapping[t] = block_table[s][p / P] * P + p % P
 *   and rows past the last request (padding): position 0, slot -1.
 * The other entries of block_table are left as they were.  With the same
 * inputs a call writes the same values again, so it may be repeated or
 * replayed; to go on, pass next_cursor's value as the next call's cursor.
 *   context_lens, query_lens  [S] int32
 *   block_table   [S, W] int32: the pages each request has (in), with the new
 *                 ones (out)
 *   query_start   [S + 1] int32 (out)      seq_lens  [S] int32 (out)
 *   positions     [A, T] or [T] int32 (out), rows contiguous, A <= PD_MAX_AXES;
 *                 T: rows of the step, padding included
 *   slot_mapping  [T] int32 (out)
 *   free_pages    [F] int32, or NULL (then the table already holds every page;
 *                 cursor and next_cursor may be NULL)
 *   cursor        [1] int32: entries of free_pages already taken
 *   next_cursor   [1] int32 (out); not cursor itself
 *   position_delta  [S] int32 or NULL: what a request's positions are ahead of
 *                 its token count (image tokens share positions: negative)
 *   page_size     any (the attention calls take multiples of 16)
 *   num_pages     pages of the pool; num_pages * page_size <= 2^31 - 1
 * No output may overlap an input (but block_table, which is both).
 * Reported: a negative length, or one past the block table (clamped; tokens
 * past the table get slot -1): PD_DEV_BAD_SEQLEN.  More tokens than T (the
 * requests are cut off there): PD_DEV_BAD_QSTART.  A page id outside the
 * pool (slot -1; a new entry is written as -1): PD_DEV_BAD_PAGE.  A list
 * that is used up (entries and slots -1; next_cursor still counts every
 * page asked for): PD_DEV_NO_PAGE. */
#define PD_DEV_NO_PAGE 0x100u /* paged_batch_tables: free_pages is used up */
#define PD_MAX_AXES 8

PD_API int paged_batch_tables(const pd_tensor *context_lens, const pd_tensor *query_lens,
                              const pd_tensor *free_pages, const pd_tensor *cursor,
                              const pd_tensor *position_delta, pd_tensor *block_table,
                              pd_tensor *query_start, pd_tensor *seq_lens, pd_tensor *positions,
                              pd_tensor *slot_mapping, pd_tensor *next_cursor, int page_size,
                              int num_pages, void *stream);

/* ---- Rotary embedding with a position per axis ----
 *
 * paged_rope_cache_write for tokens that have A positions each (time, height
 * and width of an image or video token; text has the same one on every
 * axis): rotated pair i of every head takes the angle of the axis
 * pair_axis[i],
 *     (c, s) = cos_sin_cache[positions[pair_axis[i]][t]] [i], [rot_dim / 2 + i].
 * Everything else is as there.
 *   positions  [A, T] int32 device array, rows contiguous (any distance apart,
 *              0 too: one row for every axis), 1 <= A <= PD_MAX_AXES
 *   pair_axis  [rot_dim / 2] host array (read during the call), entries < A
 * A position outside the table on any axis is clamped into it and reported
 * (PD_DEV_BAD_POSITION). */
PD_API int paged_rope_axes_cache_write(const pd_tensor *q, const pd_tensor *k, const pd_tensor *v,
                                       const pd_tensor *positions, const pd_tensor *slot_mapping,
                                       const pd_tensor *cos_sin_cache, const uint8_t *pair_axis,
                                       pd_tensor *q_out, pd_tensor *k_cache, pd_tensor *v_cache,
                                       int num_q_heads, int num_kv_heads, int head_size,
                                       int rot_dim, int page_size, int layout, int is_neox,
                                       void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_STEP_H */
