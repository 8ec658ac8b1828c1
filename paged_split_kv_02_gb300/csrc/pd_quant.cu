// Entry points of the attention over an 8-bit cache: argument checks and the
// launch plan.
#include <algorithm>
#include <cmath>

#include "pd_quant.h"

namespace pd {
namespace {

constexpr int kSmemLimit = 232448;  // dynamic shared memory of a CTA at most
constexpr int64_t kFewBytes = 24 << 20;  // of a batch's keys and values, once a row group

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct QuantPlan {
  pd_plan pub;
  int seqs_y, whole, rows_grp;
};

// Sizes are checked: S >= 1.
int make_plan(int S, int Hq, int Hkv, int D, int P, int M, int window, int sinks, int bt_width,
              int num_sms, const pd_scratch *scratch, QuantPlan *out) {
  const int64_t R = (int64_t)(Hq / Hkv) * M;
  int64_t nb_max = cdiv((int64_t)bt_width * P, kBlockKeys);
  if (window > 0)
    nb_max = std::min<int64_t>(nb_max, cdiv((int64_t)window + M - 1, kBlockKeys) + 1 +
                                           cdiv(sinks, kBlockKeys));
  // Rows of a CTA: as many as fit, so that the cache goes through the SMs as seldom as can be; but
  // where units are few, fewer, as a step and a unit's end are long with many rows.  Down to 16 rows while
  // a unit can have two CTAs (32 rows of 8 kv heads, D = 128, one request of 4,096 / 32,768 keys: 22 /
  // 37 us with 32, 15 / 34 with 16; 64 requests of 4,096, though, 167 and 200), to 8 where the reads are few
  // too (16 rows: 300 / 4,096 / 32,768 keys 11.1 / 14.3 / 24.9 us with 16, 9.3 / 12.4 / 29.2
  // with 8), or the units very few at D = 256 (2 kv heads, 30,000 keys: 28.5 and 21.5; 10 requests of
  // 8,000: 25.9 and 30.1).  All of these with tables as wide as the requests: the width is what the host
  // knows, so that a short request in a wide table gets the rows of a long one (300 keys of 16 rows: 9.4
  // us with 19 pages, 11.0 with 512 or more).  The 24 MB lie between measured 17 and 134.
  int tiles = 1;
  while (tiles < quant_max_tiles(D) && 8 * tiles < R) tiles *= 2;
  for (int t = tiles / 2; t >= 1; t /= 2) {
    const int64_t u = (int64_t)S * Hkv * cdiv(R, 8 * t);
    if (2 * u > num_sms || !scratch || scratch->counter_slots < u) break;
    if (t == 1 && u * nb_max * (kBlockKeys * 2 * D) > kFewBytes && (D < 256 || 8 * u > num_sms)) break;
    tiles = t;
  }
  const int64_t rg = cdiv(R, 8 * tiles);
  const int rows = (int)cdiv(R, rg);
  int NT = 1;
  while (8 * NT < rows) NT *= 2;
  const int NR = 8 * NT;
  const int64_t HR = Hkv * rg;
  if (HR > 65535) return PD_EINVAL;  // (units of a sequence)
  // runs of sequences whose line's places fit an int
  const int64_t per_seq = (nb_max + quant_unit_cost(D)) * HR;
  const int64_t fit = (int64_t)(INT32_MAX / 4) / per_seq;
  const int seqs = (int)std::min<int64_t>({(int64_t)S, (int64_t)kQuantSeqs, std::max<int64_t>(fit, 1)});
  const int gy = (int)cdiv(S, seqs);
  if (gy > 65535) return PD_EINVAL;
  const int64_t units = S * HR, units_y = seqs * HR;
  if (smem_bytes_quant(D, NT, seqs) > kSmemLimit) return PD_EINVAL;
  // two parts of (acc, m, l) per CTA, behind the counters
  const int64_t per_cta = 2LL * NR * (D + 2) * 4;
  int64_t G = 0;
  if (fit >= 1 && scratch && scratch->data && scratch->counter_slots >= units) {
    const int64_t cbytes = (scratch->counter_slots * 4 + 255) / 256 * 256;
    G = std::min<int64_t>(num_sms, ((int64_t)scratch->bytes - cbytes - 256) / per_cta / gy);
    G = std::min(G, cdiv(per_seq * seqs, 8));
  }
  const bool whole = G < std::min<int64_t>(units_y, std::max(1, num_sms / 4));
  if (whole) G = units_y;
  *out = QuantPlan{};
  out->seqs_y = seqs;
  out->whole = whole;
  out->rows_grp = rows;
  pd_plan &p = out->pub;
  p.path = 7;
  p.merge = whole ? 0 : 1;
  p.rows = (int)R;
  p.row_groups = (int)rg;
  p.rows_per_cta = rows;
  p.n_tiles = NT;
  p.key_groups = kQuantWarps;
  p.stages = quant_slots(D, NT);
  p.seg_blocks = (int)std::min<int64_t>(nb_max, INT32_MAX);
  p.max_segments = p.max_parts = whole ? 0 : (int)G;
  p.cluster = 1;
  p.grid_x = (int)G;
  p.grid_y = gy;
  p.block_threads = 32 * kQuantWarps;
  p.smem_bytes = smem_bytes_quant(D, NT, seqs);
  p.scratch_needed = whole ? 0 : G * gy * per_cta + 256;
  return PD_OK;
}

int check_sizes(int num_q_heads, int num_kv_heads, int head_size, int page_size, int max_query_len,
                int window, int sinks) {
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0) return PD_EINVAL;
  if (head_size != 64 && head_size != 128 && head_size != 256 && head_size != 512) return PD_EHEAD;
  if (max_query_len < 1 || max_query_len > 8) return PD_EQLEN;
  if (page_size <= 0 || page_size % kBlockKeys != 0 || window < 0 || sinks < 0) return PD_EINVAL;
  return PD_OK;
}

}  // namespace

int quant_pool(const pd_tensor *cache, const pd_tensor *scale, int layout, int Hkv, int P, int D,
               QuantPool *out) {
  const pd_tensor *t = cache, *c = scale;
  if (!t || !t->data || t->ndim != 4 || !c || !c->data || c->ndim != 3) return PD_EINVAL;
  const int hd = layout == PD_NHD ? 2 : 1, td = layout == PD_NHD ? 1 : 2;
  if (t->shape[0] < 1 || t->shape[0] > INT32_MAX || t->shape[hd] != Hkv || t->shape[td] != P ||
      t->shape[3] != D)
    return PD_EINVAL;
  if (c->shape[0] != t->shape[0] || c->shape[1] != P / PD_SCALE_TOKENS || c->shape[2] != Hkv)
    return PD_EINVAL;
  if (t->dtype != PD_E4M3 || c->dtype != PD_F32) return PD_EDTYPE;
  if (t->stride[3] != 1) return PD_EALIGN;
  for (int i = 0; i < 3; ++i) {
    if (t->stride[i] <= 0 || c->stride[i] <= 0) return PD_EINVAL;
    if (t->stride[i] % 16 != 0) return PD_EALIGN;
  }
  if (!aligned16(t->data) || (reinterpret_cast<uintptr_t>(c->data) & 3u) != 0) return PD_EALIGN;
  out->codes = static_cast<unsigned char *>(t->data);
  out->page = t->stride[0];
  out->tok = t->stride[td];
  out->head = t->stride[hd];
  out->scale = static_cast<float *>(c->data);
  out->s_page = c->stride[0];
  out->s_blk = c->stride[1];
  out->s_head = c->stride[2];
  return PD_OK;
}

}  // namespace pd

using namespace pd;

extern "C" {

PD_API int paged_decode_plan_quant(int num_seqs, int num_q_heads, int num_kv_heads, int head_size,
                                   int page_size, int max_query_len, int window, int sinks,
                                   int block_table_width, int num_sms, const pd_scratch *scratch,
                                   pd_plan *plan) {
  if (!plan || num_seqs < 1 || block_table_width < 1 || num_sms < 1) return PD_EINVAL;
  int rc = check_sizes(num_q_heads, num_kv_heads, head_size, page_size, max_query_len, window, sinks);
  if (rc != PD_OK) return rc;
  if ((int64_t)block_table_width * page_size > INT32_MAX) return PD_EINVAL;
  QuantPlan q;
  rc = make_plan(num_seqs, num_q_heads, num_kv_heads, head_size, page_size, max_query_len, window,
                 sinks, block_table_width, num_sms, scratch, &q);
  if (rc == PD_OK) *plan = q.pub;
  return rc;
}

PD_API int paged_decode_attn_quant(const pd_tensor *q, const pd_tensor *k_cache,
                                   const pd_tensor *v_cache, const pd_tensor *k_scale,
                                   const pd_tensor *v_scale, const pd_tensor *block_table,
                                   const pd_tensor *seq_lens, const pd_tensor *query_start,
                                   pd_tensor *out, int num_q_heads, int num_kv_heads,
                                   int head_size, int page_size, int max_query_len, int window,
                                   int sinks, float scale, int layout, pd_scratch *scratch,
                                   void *stream) {
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !out)
    return PD_EINVAL;
  int rc = check_sizes(num_q_heads, num_kv_heads, head_size, page_size, max_query_len, window, sinks);
  if (rc != PD_OK) return rc;
  if (!std::isfinite(scale) || (layout != PD_NHD && layout != PD_HND)) return PD_EINVAL;
  if (seq_lens->ndim != 1 || seq_lens->stride[0] != 1) return PD_EINVAL;
  if (seq_lens->dtype != PD_I32 || block_table->dtype != PD_I32) return PD_EDTYPE;
  const int64_t S = seq_lens->shape[0];
  // (of no request: any pointer)
  if (S < 0 || S > INT32_MAX || (S > 0 && (!seq_lens->data || !block_table->data))) return PD_EINVAL;
  if (block_table->ndim != 2 || block_table->shape[0] != S || block_table->shape[1] < 1 ||
      block_table->stride[1] != 1 || block_table->stride[0] < 0)
    return PD_EINVAL;
  if (block_table->shape[1] > INT32_MAX || block_table->shape[1] * (int64_t)page_size > INT32_MAX)
    return PD_EINVAL;
  int64_t T = S * max_query_len;
  if (query_start) {
    if (query_start->ndim != 1 || !query_start->data || query_start->shape[0] != S + 1 ||
        query_start->stride[0] != 1)
      return PD_EINVAL;
    if (query_start->dtype != PD_I32) return PD_EDTYPE;
    if (q->ndim != 3) return PD_EINVAL;
    T = q->shape[0];
  }
  if (T < 0 || T > INT32_MAX) return PD_EINVAL;
  if ((rc = check_rows(q, T, num_q_heads, head_size)) != PD_OK) return rc;
  if ((rc = check_rows(out, T, num_q_heads, head_size)) != PD_OK) return rc;
  if (q->dtype != out->dtype) return PD_EDTYPE;
  QuantAttnParams p{};
  if ((rc = quant_pool(k_cache, k_scale, layout, num_kv_heads, page_size, head_size, &p.k)) != PD_OK)
    return rc;
  if ((rc = quant_pool(v_cache, v_scale, layout, num_kv_heads, page_size, head_size, &p.v)) != PD_OK)
    return rc;
  if (k_cache->shape[0] != v_cache->shape[0]) return PD_EINVAL;
  if (T == 0) return PD_OK;

  int num_sms = 0;
  if ((rc = device_check(&num_sms, &p.status)) != PD_OK) return rc;
  // (no request: every row is padding)
  if (S == 0)
    return zero_padding(out, static_cast<const int32_t *>(query_start->data), 0, num_sms, stream);
  QuantPlan plan;
  rc = make_plan((int)S, num_q_heads, num_kv_heads, head_size, page_size, max_query_len, window,
                 sinks, (int)block_table->shape[1], num_sms, scratch, &plan);
  if (rc != PD_OK) return rc;
  p.q = q->data;
  p.q_s0 = q->stride[0];
  p.q_s1 = q->stride[1];
  p.out = out->data;
  p.o_s0 = out->stride[0];
  p.o_s1 = out->stride[1];
  p.block_table = static_cast<const int32_t *>(block_table->data);
  p.bt_stride = block_table->stride[0];
  p.bt_width = (int)block_table->shape[1];
  p.seq_lens = static_cast<const int32_t *>(seq_lens->data);
  p.query_start = query_start ? static_cast<const int32_t *>(query_start->data) : nullptr;
  p.num_seqs = (int)S;
  p.num_tokens = (int)T;
  p.num_pages = (int)k_cache->shape[0];
  p.Hq = num_q_heads;
  p.Hkv = num_kv_heads;
  p.G = num_q_heads / num_kv_heads;
  p.M = max_query_len;
  p.P = page_size;
  p.window = window;
  p.sinks = window > 0 ? sinks : 0;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.rg = plan.pub.row_groups;
  p.rows_grp = plan.rows_grp;
  p.seqs_y = plan.seqs_y;
  p.whole = plan.whole;
  p.min_share = 8;
  // (a step of every warp: 2048 keys of 32 / 8 heads at D = 128 in parts of 8 / 16 / 32 / 64 blocks: 9.5 / 9.4 /
  // 10.6 / 13.2 us)
  p.min_part = 8 * quant_step_blocks(head_size, plan.pub.n_tiles);
  p.bpp = page_size / kBlockKeys;
  p.by_units = FastDiv(num_kv_heads * p.rg);
  p.by_groups = FastDiv(p.rg);
  p.by_heads = FastDiv(p.G);
  p.by_page = FastDiv(p.bpp);
  p.by_ctas = FastDiv(plan.pub.grid_x);
  const int NR = 8 * plan.pub.n_tiles;
  if (!plan.whole) {
    char *base = static_cast<char *>(scratch->data);
    const int64_t cbytes = (scratch->counter_slots * 4 + 255) / 256 * 256;
    const int64_t parts = 2LL * plan.pub.grid_x * plan.pub.grid_y;
    p.counters = reinterpret_cast<int *>(base);
    p.unit_counters = (int)std::min<int64_t>(64, scratch->counter_slots / (S * num_kv_heads * p.rg));
    p.merge_bytes = 160 << 10;
    p.part_acc = reinterpret_cast<float *>(base + cbytes);
    p.part_ml = reinterpret_cast<float *>(base + cbytes + parts * NR * head_size * 4);
  }
  Launch l{};
  l.grid = dim3(plan.pub.grid_x, plan.pub.grid_y, 1);
  l.block = dim3(plan.pub.block_threads, 1, 1);
  l.smem = plan.pub.smem_bytes;
  const bool bf16 = q->dtype == PD_BF16;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  switch (head_size) {
    case 64: e = launch_quant_d64(bf16, plan.pub.n_tiles, p, l, st); break;
    case 128: e = launch_quant_d128(bf16, plan.pub.n_tiles, p, l, st); break;
    case 256: e = launch_quant_d256(bf16, plan.pub.n_tiles, p, l, st); break;
    case 512: e = launch_quant_d512(bf16, plan.pub.n_tiles, p, l, st); break;
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return PD_ECUDA;
  }
  return PD_OK;
}

}  // extern "C"
