// Entry points of the attention over a window with sinks: the calls of
// pd_api.cu and pd_prefill.cu with the sinks passed on.
#include "paged_step.h"
#include "pd_internal.h"

using namespace pd;

extern "C" {

PD_API int paged_decode_attn_sinks(const pd_tensor *q, const pd_tensor *k_cache,
                                   const pd_tensor *v_cache, const pd_tensor *block_table,
                                   const pd_tensor *seq_lens, const pd_tensor *query_start,
                                   pd_tensor *out, int num_q_heads, int num_kv_heads,
                                   int head_size, int page_size, int max_query_len, int window,
                                   int sinks, float scale, int layout, pd_scratch *scratch,
                                   void *stream, const pd_options *opts) {
  return attn_call(q, k_cache, v_cache, block_table, seq_lens, query_start, out, num_q_heads,
                   num_kv_heads, head_size, page_size, max_query_len, window, sinks, scale, layout,
                   scratch, stream, opts);
}

PD_API int paged_decode_plan_sinks(int num_seqs, int num_q_heads, int num_kv_heads, int head_size,
                                   int page_size, int max_query_len, int window, int sinks,
                                   int block_table_width, int num_sms, const pd_scratch *scratch,
                                   const pd_options *opts, pd_plan *plan) {
  if (!plan) return PD_EINVAL;
  return attn_plan(num_seqs, num_q_heads, num_kv_heads, head_size, page_size, max_query_len,
                   window, sinks, block_table_width, num_sms, scratch, opts, plan);
}

PD_API int paged_prefill_plan_sinks(const int32_t *query_start, const int32_t *seq_lens,
                                    int num_seqs, int num_q_heads, int num_kv_heads,
                                    int head_size, int window, int sinks, int num_sms,
                                    pd_prefill_item *items, int64_t capacity,
                                    pd_prefill_plan_info *info) {
  return prefill_plan_call(query_start, seq_lens, num_seqs, num_q_heads, num_kv_heads, head_size,
                           window, sinks, num_sms, items, capacity, info);
}

PD_API int paged_prefill_attn_sinks(const pd_tensor *q, const pd_tensor *k_cache,
                                    const pd_tensor *v_cache, const pd_tensor *block_table,
                                    const pd_tensor *seq_lens, const pd_tensor *query_start,
                                    const pd_tensor *work, const pd_prefill_plan_info *info,
                                    pd_tensor *out, int num_q_heads, int num_kv_heads,
                                    int head_size, int page_size, int window, int sinks,
                                    float scale, int layout, pd_scratch *scratch, void *stream) {
  return prefill_call(q, k_cache, v_cache, block_table, seq_lens, query_start, work, info, out,
                      num_q_heads, num_kv_heads, head_size, page_size, window, sinks, scale,
                      layout, scratch, stream);
}

}  // extern "C"
