// The tables of a batch built on the GPU from its requests' lengths: query
// starts, lengths, new pages from a free list, positions and cache slots, in
// one launch.
//
// The starts and the pages taken are exclusive sums over the requests.  Every
// block forms them itself, in passes of one request per thread (a block-wide
// scan of two sums), so no block waits on another: block 0 writes what
// belongs to requests, block b > 0 the kTokens tokens from (b - 1) kTokens
// on.  A token block notes each request that owns some of its tokens at the
// first of them; a running maximum over the tokens then gives every token
// its request.  A new page is written to the block table by the one token
// that opens it (the token whose position is a multiple of the page size).
//
// The work is a few bytes per token: launch latency and one chain of dependent
// loads (lengths -> sums -> page id) bound it.
#include "paged_step.h"
#include "pd_internal.h"
#include "pd_ptx.cuh"

namespace pd {
namespace {

constexpr int kThreads = 1024;
constexpr int kTokens = kThreads;  // tokens of a block

struct TablesParams {
  const int32_t *context, *query, *free_pages, *cursor, *delta;
  int32_t *table;
  int64_t bt_stride;
  int bt_width;
  int32_t *query_start, *seq_lens, *positions, *slots, *next_cursor;
  int64_t pos_stride;
  int axes, S, T, num_free, P, num_pages;
  unsigned int *status;
};

// Two running sums: tokens (held at T, so that they cannot wrap) and pages
// (wrapping, and then of requests past T only, which take none).
struct Sums {
  unsigned int tok, pages;
};

__device__ __forceinline__ Sums add(Sums a, Sums b, unsigned int T) {
  return {min(a.tok + b.tok, T), a.pages + b.pages};
}

__device__ __forceinline__ unsigned int cdiv_u(unsigned int a, unsigned int b) {
  return (a + b - 1) / b;
}

__global__ void __launch_bounds__(kThreads) pd_batch_tables(const __grid_constant__ TablesParams p) {
  __shared__ Sums warp_sums[kThreads / 32];
  __shared__ int owner[kTokens], o_start[kTokens], o_ctx[kTokens], warp_max[kThreads / 32];
  __shared__ unsigned int o_off[kTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool requests = blockIdx.x == 0;
  const int t0 = requests ? 0 : (int)(blockIdx.x - 1) * kTokens;
  const int t1 = requests ? 0 : min(p.T - t0, kTokens) + t0;
  owner[tid] = -1;
  // the lengths may be the previous kernel's outputs
  grid_dependency_wait();
  grid_dependents_launch();
  const unsigned int T = (unsigned)p.T, P = (unsigned)p.P;
  const unsigned int cap = (unsigned)p.bt_width * P;  // tokens a table row can address
  unsigned int bad = 0;
  Sums carry = {0, 0};
  // (a token block stops at the first pass that starts past its tokens)
  for (int base = 0; base < p.S && (requests || (int)carry.tok < t1); base += kThreads) {
    const int s = base + tid;
    int c_in = 0, q_in = 0;
    if (s < p.S) {
      c_in = __ldg(p.context + s);
      q_in = __ldg(p.query + s);
    }
    const unsigned int c = min((unsigned)max(c_in, 0), cap), q = min((unsigned)max(q_in, 0), T);
    const unsigned int have = cdiv_u(c, P);
    Sums x = {q, cdiv_u(min(c + q, cap), P) - have};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums y = {__shfl_up_sync(0xffffffffu, x.tok, o), __shfl_up_sync(0xffffffffu, x.pages, o)};
      if (lane >= o) x = add(y, x, T);
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    Sums w = warp_sums[lane];  // 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums y = {__shfl_up_sync(0xffffffffu, w.tok, o), __shfl_up_sync(0xffffffffu, w.pages, o)};
      if (lane >= o) w = add(y, w, T);
    }
    const Sums before = {__shfl_sync(0xffffffffu, w.tok, max(warp - 1, 0)),
                         __shfl_sync(0xffffffffu, w.pages, max(warp - 1, 0))};
    Sums end = warp ? add(before, x, T) : x;
    end = add(carry, end, T);
    // start: the sums before this request
    Sums start = {__shfl_up_sync(0xffffffffu, end.tok, 1), __shfl_up_sync(0xffffffffu, end.pages, 1)};
    if (lane == 0) start = warp ? add(carry, before, T) : carry;
    const unsigned int len = min(c + (end.tok - start.tok), cap);
    if (s < p.S) {
      if (requests) {
        p.query_start[s] = (int)start.tok;
        p.seq_lens[s] = (int)len;
        if (c_in < 0 || q_in < 0 || (unsigned)max(c_in, 0) > cap || c + (end.tok - start.tok) > cap)
          bad |= PD_DEV_BAD_SEQLEN;
        if ((unsigned)max(q_in, 0) != end.tok - start.tok) bad |= PD_DEV_BAD_QSTART;
        if (s == p.S - 1) p.query_start[p.S] = (int)end.tok;
        // the last request with tokens before T closes the pages' sum (those
        // after it take no token and no page)
        if (p.next_cursor && start.tok < T && (s == p.S - 1 || end.tok == T)) {
          const int64_t n = (int64_t)(p.cursor ? __ldg(p.cursor) : 0) +
                            (p.free_pages ? start.pages + (cdiv_u(len, P) - have) : 0u);
          *p.next_cursor = (int)min(n, (int64_t)INT32_MAX);
        }
      } else if (end.tok > start.tok && (int)end.tok > t0 && (int)start.tok < t1) {
        const int at = max((int)start.tok, t0) - t0;
        owner[at] = s;
        o_start[at] = (int)start.tok;
        o_ctx[at] = (int)c;
        o_off[at] = start.pages;
      }
    }
    const Sums all = {__shfl_sync(0xffffffffu, w.tok, 31), __shfl_sync(0xffffffffu, w.pages, 31)};
    carry = add(carry, all, T);
    __syncthreads();
  }
  if (requests) {
    if (tid == 0) {
      if (p.S == 0) p.query_start[0] = 0;
      if (p.next_cursor && (p.S == 0 || p.T == 0)) *p.next_cursor = p.cursor ? __ldg(p.cursor) : 0;
    }
    if (bad) atomicOr(p.status, bad);
    return;
  }
  // ---- the tokens: the request noted last at or before each of them --------
  __syncthreads();
  int at = owner[tid] >= 0 ? tid : -1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at = max(at, y);
  }
  if (lane == 31) warp_max[warp] = at;
  __syncthreads();
  int m = lane < warp ? warp_max[lane] : -1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  at = max(at, m);
  const int t = t0 + tid;
  if (t >= t1) return;
  int pos = 0, slot = -1;
  // (carry.tok: the tokens of all requests, or of enough of them to pass t1)
  if (t < (int)carry.tok) {
    const int s = owner[at];
    const unsigned int c = (unsigned)o_ctx[at], i = (unsigned)(t - o_start[at]);
    const unsigned int at_pos = c + i, page = at_pos / P, in = at_pos - page * P;
    pos = (int)at_pos + (p.delta ? __ldg(p.delta + s) : 0);
    if (at_pos < cap) {
      const unsigned int have = cdiv_u(c, P);
      int32_t *entry = p.table + (int64_t)s * p.bt_stride + page;
      int id;
      if (p.free_pages && page >= have) {
        const int64_t f = (int64_t)__ldg(p.cursor) + (int64_t)(o_off[at] + (page - have));
        const bool left = f >= 0 && f < p.num_free;
        id = left ? __ldg(p.free_pages + f) : -1;
        if (!left) bad |= PD_DEV_NO_PAGE;
        else if ((unsigned)id >= (unsigned)p.num_pages) bad |= PD_DEV_BAD_PAGE;
        if ((unsigned)id >= (unsigned)p.num_pages) id = -1;
        if (in == 0) *entry = id;
      } else {
        id = *entry;
        if ((unsigned)id >= (unsigned)p.num_pages) {
          bad |= PD_DEV_BAD_PAGE;
          id = -1;
        }
      }
      if (id >= 0) slot = id * p.P + (int)in;
    }
  }
  for (int a = 0; a < p.axes; ++a) p.positions[a * p.pos_stride + t] = pos;
  p.slots[t] = slot;
  if (bad) atomicOr(p.status, bad);
}

// [n] int32, contiguous (empty: any pointer)
int check_vec(const pd_tensor *t, int64_t n) {
  if (!t || t->ndim != 1 || t->shape[0] != n || (n != 0 && !t->data)) return PD_EINVAL;
  if (t->dtype != PD_I32) return PD_EDTYPE;
  if (n > 1 && t->stride[0] != 1) return PD_EALIGN;
  return PD_OK;
}

// the bytes from an int32 tensor's first element to its last
struct Span {
  const char *lo, *hi;
};
Span span_of(const pd_tensor *t) {
  int64_t last = 0, n = 1;
  for (int i = 0; i < t->ndim; ++i) {
    last += (t->shape[i] - 1) * t->stride[i];
    n *= t->shape[i];
  }
  const char *b = static_cast<const char *>(t->data);
  return n > 0 ? Span{b, b + (last + 1) * 4} : Span{nullptr, nullptr};
}

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" PD_API int paged_batch_tables(
    const pd_tensor *context_lens, const pd_tensor *query_lens, const pd_tensor *free_pages,
    const pd_tensor *cursor, const pd_tensor *position_delta, pd_tensor *block_table,
    pd_tensor *query_start, pd_tensor *seq_lens, pd_tensor *positions, pd_tensor *slot_mapping,
    pd_tensor *next_cursor, int page_size, int num_pages, void *stream) {
  if (!context_lens || !query_lens || !block_table || !query_start || !seq_lens || !positions ||
      !slot_mapping)
    return PD_EINVAL;
  if (page_size <= 0 || num_pages <= 0 || (int64_t)num_pages * page_size > INT32_MAX)
    return PD_EINVAL;
  if (context_lens->ndim != 1 || slot_mapping->ndim != 1) return PD_EINVAL;
  const int64_t S = context_lens->shape[0], T = slot_mapping->shape[0];
  if (S < 0 || S > INT32_MAX - kThreads || T < 0 || T > INT32_MAX - kTokens) return PD_EINVAL;
  int rc;
  if ((rc = check_vec(context_lens, S)) != PD_OK) return rc;
  if ((rc = check_vec(query_lens, S)) != PD_OK) return rc;
  if ((rc = check_vec(query_start, S + 1)) != PD_OK) return rc;
  if ((rc = check_vec(seq_lens, S)) != PD_OK) return rc;
  if ((rc = check_vec(slot_mapping, T)) != PD_OK) return rc;
  if (position_delta && (rc = check_vec(position_delta, S)) != PD_OK) return rc;
  if (block_table->ndim != 2 || block_table->shape[0] != S || block_table->shape[1] < 1 ||
      (S > 0 && !block_table->data))
    return PD_EINVAL;
  if (block_table->dtype != PD_I32) return PD_EDTYPE;
  if (S > 0 && block_table->shape[1] > 1 && block_table->stride[1] != 1) return PD_EALIGN;
  // (rows of their own: new pages are written to them)
  if (S > 1 && block_table->stride[0] < block_table->shape[1]) return PD_EINVAL;
  if (block_table->shape[1] > INT32_MAX || block_table->shape[1] * (int64_t)page_size > INT32_MAX)
    return PD_EINVAL;
  if (positions->ndim != 1 && positions->ndim != 2) return PD_EINVAL;
  const bool many = positions->ndim == 2;
  const int64_t axes = many ? positions->shape[0] : 1;
  if (axes < 1 || axes > PD_MAX_AXES || positions->shape[many ? 1 : 0] != T ||
      (T > 0 && !positions->data))
    return PD_EINVAL;
  if (positions->dtype != PD_I32) return PD_EDTYPE;
  if (T > 1 && positions->stride[many ? 1 : 0] != 1) return PD_EALIGN;
  if (axes > 1 && T > 0 && positions->stride[0] < T) return PD_EINVAL;
  if (free_pages) {
    if (!cursor || !next_cursor) return PD_EINVAL;
    if (free_pages->ndim != 1 || free_pages->shape[0] < 0 || free_pages->shape[0] > INT32_MAX)
      return PD_EINVAL;
    if ((rc = check_vec(free_pages, free_pages->shape[0])) != PD_OK) return rc;
  }
  if (cursor && (rc = check_vec(cursor, 1)) != PD_OK) return rc;
  if (next_cursor && (rc = check_vec(next_cursor, 1)) != PD_OK) return rc;
  // no output over an input or another output
  const pd_tensor *outs[] = {block_table, query_start, seq_lens, positions, slot_mapping, next_cursor};
  const pd_tensor *ins[] = {context_lens, query_lens, free_pages, cursor, position_delta};
  for (int i = 0; i < 6; ++i) {
    if (!outs[i]) continue;
    const Span a = span_of(outs[i]);
    auto meets = [&](const pd_tensor *t) {
      if (!t) return false;
      const Span b = span_of(t);
      return a.lo < b.hi && b.lo < a.hi;
    };
    for (const pd_tensor *t : ins)
      if (meets(t)) return PD_EINVAL;
    for (int j = i + 1; j < 6; ++j)
      if (meets(outs[j])) return PD_EINVAL;
  }

  unsigned int *status = nullptr;
  if ((rc = device_check(nullptr, &status)) != PD_OK) return rc;

  auto ptr = [](const pd_tensor *t) { return t ? static_cast<int32_t *>(t->data) : nullptr; };
  TablesParams p{};
  p.context = ptr(context_lens);
  p.query = ptr(query_lens);
  p.free_pages = ptr(free_pages);
  p.num_free = free_pages ? (int)free_pages->shape[0] : 0;
  p.cursor = ptr(cursor);
  p.delta = ptr(position_delta);
  p.table = ptr(block_table);
  p.bt_stride = block_table->stride[0];
  p.bt_width = (int)block_table->shape[1];
  p.query_start = ptr(query_start);
  p.seq_lens = ptr(seq_lens);
  p.positions = ptr(positions);
  p.pos_stride = axes > 1 ? positions->stride[0] : 0;
  p.axes = (int)axes;
  p.slots = ptr(slot_mapping);
  p.next_cursor = ptr(next_cursor);
  p.S = (int)S;
  p.T = (int)T;
  p.P = page_size;
  p.num_pages = num_pages;
  p.status = status;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(1 + (T + kTokens - 1) / kTokens));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, pd_batch_tables, p) != cudaSuccess) {
    cudaGetLastError();
    return PD_ECUDA;
  }
  return PD_OK;
}
