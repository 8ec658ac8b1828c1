// Pages of an 8-bit cache as 16-bit pages of a staging pool.
//
// A block of 16 tokens, K and V of every head, is cut into slices of 512 chunks of 16
// codes, and a CTA takes every so many slices: a thread turns two chunks into values,
// its loads ahead of its stores.  A warp looks 32 of the CTA's slices up at once, a
// lane each, so that blocks past a request's end or left out of the tables (older
// than a window) cost little; but each is looked up, and tables far wider than the
// requests show: 64 requests of 300 tokens 23 us in tables of their 19 pages, 29 / 49 /
// 144 in tables of 512 / 2,048 / 8,192.
//
// Memory-bound: 1 byte read and 2 written a value.  16 requests of 2,000 to 16,384
// tokens, 8 kv heads of 128: 105 us, 6.1 TB/s, 90 % of a copy's rate (one CTA a block
// and a look for each took 120).  One of 4,090: 6.6 us, 2.5 of them a launch.
#include "pd_e4m3.cuh"
#include "pd_quant.h"
#include "pd_rope.cuh"

namespace pd {
namespace {

constexpr int kThreads = 256;
// 16 requests of 2,000 to 16,384 tokens, then 24 with 2,000 left by a window, in us: 8 / 12 / 16 / 24
// CTAs of an SM 110 / 109 / 105 / 103 and 14.3 / 14.2 / 14.5 / 15.6 (the empty blocks cost each a look).
constexpr int kCtas = 16;
// Chunks of a thread, and so of a CTA's item: 1 / 2 / 4 take 119 / 105 / 113 and 16.4 / 14.5 / 16.6 us.
constexpr int U = 2;

struct OutPool {
  unsigned short *data;
  int64_t page, tok, head;
};

struct QuantReadParams {
  QuantPool k, v;
  OutPool ko, vo;
  const int32_t *block_table, *out_table, *seq_lens;
  int64_t bt_stride, ot_stride;
  int S, width, Hkv, P, lg_row;  // lg_row: log2 of a row's 16-code chunks
  int slices;                    // of a block, one CTA's each
  int num_pages, num_out_pages;
  unsigned int *status;
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads) pd_quant_read(const __grid_constant__ QuantReadParams p) {
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  const int per_page = p.P / PD_SCALE_TOKENS;
  const int64_t per_seq = (int64_t)p.width * per_page * p.slices, total = per_seq * p.S;
  const int n = (PD_SCALE_TOKENS * p.Hkv) << p.lg_row;  // chunks of K (or V) of a block
#pragma unroll 1
  for (int64_t i0 = blockIdx.x; i0 < total; i0 += 32LL * gridDim.x) {
    // (every warp alike)
    const int64_t i = i0 + (int64_t)lane * gridDim.x;
    int len = 0, src = -1, dst = -1, blk = 0, slice = 0;
    if (i < total) {
      const int s = (int)(i / per_seq);
      const int64_t rest = i - s * per_seq;
      blk = (int)(rest / p.slices);
      slice = (int)(rest - (int64_t)blk * p.slices);
      len = __ldg(p.seq_lens + s);
      const int j = blk / per_page;
      src = __ldg(p.block_table + s * p.bt_stride + j);
      dst = __ldg(p.out_table + s * p.ot_stride + j);
      if (rest == 0 && len > (int64_t)p.width * p.P && threadIdx.x < 32) atomicOr(p.status, PD_DEV_BAD_SEQLEN);
    }
    bool there = len > blk * PD_SCALE_TOKENS && src >= 0 && dst >= 0;
    if (there && (src >= p.num_pages || dst >= p.num_out_pages)) {
      if (threadIdx.x < 32) atomicOr(p.status, PD_DEV_BAD_PAGE);
      there = false;
    }
    uint32_t todo = __ballot_sync(0xffffffffu, there);
#pragma unroll 1
    while (todo) {
      const int from = __ffs(todo) - 1;
      todo &= todo - 1;
      const int b = __shfl_sync(0xffffffffu, blk, from), sub = b % per_page;
      const int left = __shfl_sync(0xffffffffu, len, from) - b * PD_SCALE_TOKENS;  // tokens of the block
      const int64_t page = __shfl_sync(0xffffffffu, src, from), to_page = __shfl_sync(0xffffffffu, dst, from);
      const int c0 = __shfl_sync(0xffffffffu, slice, from) * (U * kThreads) + threadIdx.x;
      uint4 w[U];
      float f[U];
      unsigned short *to[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        int c = c0 + u * kThreads;
        to[u] = nullptr;
        if (c >= 2 * n) continue;
        const bool is_v = c >= n;
        if (is_v) c -= n;
        const int ch = c & ((1 << p.lg_row) - 1), r = c >> p.lg_row;
        const int tok = r & (PD_SCALE_TOKENS - 1), h = r / PD_SCALE_TOKENS;
        if (tok >= left) continue;
        const QuantPool &t = is_v ? p.v : p.k;
        const OutPool &o = is_v ? p.vo : p.ko;
        const int row = sub * PD_SCALE_TOKENS + tok;
        w[u] = __ldcs(reinterpret_cast<const uint4 *>(t.codes + page * t.page + row * t.tok + h * t.head + 16 * ch));
        f[u] = __ldg(t.scale + page * t.s_page + sub * t.s_blk + h * t.s_head);
        to[u] = o.data + to_page * o.page + row * o.tok + h * o.head + 16 * ch;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!to[u]) continue;
        const uint32_t words[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        uint32_t out[8];
        auto values = [&](auto product) {
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            float x[4];
            floats4(words[z], x);
            out[2 * z] = Elem<BF16>::from2(product(x[0]), product(x[1]));
            out[2 * z + 1] = Elem<BF16>::from2(product(x[2]), product(x[3]));
          }
        };
        if (power_of_two(f[u]))
          values([&](float x) { return x * f[u]; });
        else
          values([&](float x) { return times_marked(x, f[u]); });  // (4 bits x 24 do not fit fp32)
        uint4 *at = reinterpret_cast<uint4 *>(to[u]);
        at[0] = make_uint4(out[0], out[1], out[2], out[3]);
        at[1] = make_uint4(out[4], out[5], out[6], out[7]);
      }
    }
  }
  grid_dependents_launch();
}

void out_pool(const pd_tensor *t, int layout, OutPool *o) {
  o->data = static_cast<unsigned short *>(t->data);
  pool_strides(t, layout, &o->page, &o->tok, &o->head);
}

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" PD_API int paged_quant_cache_read(const pd_tensor *k_cache, const pd_tensor *v_cache,
                                             const pd_tensor *k_scale, const pd_tensor *v_scale,
                                             const pd_tensor *block_table, const pd_tensor *seq_lens,
                                             const pd_tensor *out_table, pd_tensor *k_out,
                                             pd_tensor *v_out, int num_kv_heads, int head_size,
                                             int page_size, int layout, void *stream) {
  if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !out_table || !k_out ||
      !v_out)
    return PD_EINVAL;
  if (num_kv_heads <= 0) return PD_EINVAL;
  if (head_size != 64 && head_size != 128 && head_size != 256 && head_size != 512) return PD_EHEAD;
  if (page_size <= 0 || page_size % PD_SCALE_TOKENS != 0 || (layout != PD_NHD && layout != PD_HND))
    return PD_EINVAL;
  int rc;
  QuantReadParams p{};
  if ((rc = quant_pool(k_cache, k_scale, layout, num_kv_heads, page_size, head_size, &p.k)) != PD_OK)
    return rc;
  if ((rc = quant_pool(v_cache, v_scale, layout, num_kv_heads, page_size, head_size, &p.v)) != PD_OK)
    return rc;
  if (k_cache->shape[0] != v_cache->shape[0]) return PD_EINVAL;
  if ((rc = check_cache_tensor(k_out, layout, num_kv_heads, page_size, head_size)) != PD_OK) return rc;
  if ((rc = check_cache_tensor(v_out, layout, num_kv_heads, page_size, head_size)) != PD_OK) return rc;
  if (k_out->dtype != v_out->dtype) return PD_EDTYPE;
  if (k_out->shape[0] != v_out->shape[0]) return PD_EINVAL;
  if (seq_lens->ndim != 1) return PD_EINVAL;
  const int64_t S = seq_lens->shape[0];
  if (S < 0 || S > INT32_MAX) return PD_EINVAL;
  if ((rc = check_i32_vector(seq_lens, S)) != PD_OK) return rc;
  for (const pd_tensor *t : {block_table, out_table}) {
    if (t->ndim != 2 || t->shape[0] != S || t->shape[1] < 1 || t->shape[1] != block_table->shape[1] ||
        t->stride[1] != 1 || t->stride[0] < 0 || (!t->data && S > 0))
      return PD_EINVAL;
    if (t->dtype != PD_I32) return PD_EDTYPE;
  }
  const int64_t W = block_table->shape[1];
  if (W > INT32_MAX || W * page_size > INT32_MAX) return PD_EINVAL;
  // (a block's chunks are ints)
  if ((int64_t)num_kv_heads * head_size > (1 << 24)) return PD_EINVAL;
  if (S == 0) return PD_OK;
  int num_sms = 0;
  if ((rc = device_check(&num_sms, &p.status)) != PD_OK) return rc;
  out_pool(k_out, layout, &p.ko);
  out_pool(v_out, layout, &p.vo);
  p.block_table = static_cast<const int32_t *>(block_table->data);
  p.out_table = static_cast<const int32_t *>(out_table->data);
  p.seq_lens = static_cast<const int32_t *>(seq_lens->data);
  p.bt_stride = block_table->stride[0];
  p.ot_stride = out_table->stride[0];
  p.S = (int)S;
  p.width = (int)W;
  p.Hkv = num_kv_heads;
  p.P = page_size;
  for (p.lg_row = 0; (16 << p.lg_row) < head_size; ++p.lg_row) {
  }
  p.num_pages = (int)k_cache->shape[0];
  p.num_out_pages = (int)k_out->shape[0];
  p.slices = (int)((2LL * num_kv_heads * head_size + U * kThreads - 1) / (U * kThreads));
  const int64_t items = S * W * (page_size / PD_SCALE_TOKENS) * p.slices;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(items < (int64_t)kCtas * num_sms ? items : (int64_t)kCtas * num_sms));
  cfg.blockDim = dim3(kThreads);
  const cudaError_t e = k_out->dtype == PD_BF16 ? cudaLaunchKernelEx(&cfg, pd_quant_read<true>, p)
                                                : cudaLaunchKernelEx(&cfg, pd_quant_read<false>, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return PD_ECUDA;
  }
  return PD_OK;
}
