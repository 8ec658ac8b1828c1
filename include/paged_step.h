/*
 * paged_step.h — the calls around and beside paged_decode.h that a serving
 * step makes: attention over a sliding window whose first tokens stay
 * visible (sinks).
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
 *                built (PD_EINVAL) */
PD_API int paged_decode_attn_sinks(const pd_tensor *q, const pd_tensor *k_cache,
                                   const pd_tensor *v_cache, const pd_tensor *block_table,
                                   const pd_tensor *seq_lens, const pd_tensor *query_start,
                                   pd_tensor *out, int num_q_heads, int num_kv_heads,
                                   int head_size, int page_size, int max_query_len, int window,
                                   int sinks, float scale, int layout, pd_scratch *scratch,
                                   void *stream, const pd_options *opts);

/* The launch plan of that call, on the host only. */
PD_API int paged_decode_plan_sinks(int num_seqs, int num_q_heads, int num_kv_heads, int head_size,
                                   int page_size, int max_query_len, int window, int sinks,
                                   int block_table_width, int num_sms, const pd_scratch *scratch,
                                   const pd_options *opts, pd_plan *plan);

/* The prefill work list and call with sinks (paged_prefill_plan,
 * paged_prefill_attn; scratch from paged_prefill_scratch_bytes).  The plan's
 * loads are those of the window with sinks; a plan made for another window
 * or sinks gives the same outputs, less evenly spread. */
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

#ifdef __cplusplus
}
#endif

#endif /* PAGED_STEP_H */
