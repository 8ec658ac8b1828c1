// The tables of a batch built on the GPU from its requests' lengths: query
// starts, lengths, new pages from a free list, positions and cache slots, in
// one launch.
//
// The starts and the pages taken are exclusive sums over the requests.  Every
// block forms them itself, a few requests of a thread at a time and a
// block-wide scan of two sums, so no block waits on another: block 0 writes what
// belongs to requests, block b > 0 the kTokens tokens from (b - 1) kTokens on,
// four of a thread.  A token block notes each request that owns some of its
// tokens at the first of them; a running maximum over the tokens then gives
// every token its request.  A new page is written to the block table by the
// one token that opens it (the token whose position is a multiple of the page
// size).
//
// The work is a few bytes per token: launch latency and one chain of dependent
// loads (lengths -> sums -> page id) bound it.  256 requests of 1 .. 4 tokens
// take 2.9 us, 1500 with 234000 tokens on three axes 4.6 us (3.7 MB).  Up to 256
// requests take one request of a thread and 256 threads (with 512: 3.5 us),
// more take four and 512 threads (1500 requests in one pass; with 256 threads
// and two passes 5.0, eight of a thread 5.3).  One token of a thread, in blocks
// of 1024, took 3.2 and 6.1 us; four whose loads wait for one another 4.1 and 6.1.
#include "paged_step.h"
#include "pd_internal.h"
#include "pd_ptx.cuh"

namespace pd {
namespace {

constexpr int kFew = 256;   // threads, with a request each
constexpr int kMany = 512;  // threads, with kPerMany requests each per pass
constexpr int kPerMany = 4;
constexpr int kRun = 4;     // tokens of a thread

struct TablesParams {
  const int32_t *context, *query, *free_pages, *cursor, *delta;
  int32_t *table;
  int64_t bt_stride;
  int bt_width;
  int32_t *query_start, *seq_lens, *positions, *slots, *next_cursor;
  int64_t pos_stride;
  int axes, S, T, num_free, P, num_pages;
  unsigned long long magic;  // ceil(2^shift / P), shift = 31 + ceil(log2 P)
  int shift;
  unsigned int *status;
};

// n / P for n < 2^31: n x (magic P - 2^shift) < 2^31 P <= 2^shift, so the
// product's high part is exact
__device__ __forceinline__ unsigned int div_p(unsigned int n, const TablesParams &p) {
  return (unsigned int)((n * p.magic) >> p.shift);
}
__device__ __forceinline__ unsigned int cdiv_p(unsigned int n, const TablesParams &p) {
  const unsigned int q = div_p(n, p);
  return q + (q * (unsigned)p.P != n);
}

// Two running sums: tokens (held at T, so that they cannot wrap) and pages
// (wrapping, and then of requests past T only, which take none).
struct Sums {
  unsigned int tok, pages;
};

__device__ __forceinline__ Sums add(Sums a, Sums b, unsigned int T) {
  return {min(a.tok + b.tok, T), a.pages + b.pages};
}

// v[0 .. 4) to the four places from p on that lie before n, in one store
// where the address allows it
__device__ __forceinline__ void store4(int32_t *p, const int (&v)[kRun], int n) {
  if (n >= kRun && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
    *reinterpret_cast<int4 *>(p) = make_int4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kRun; ++i)
      if (i < n) p[i] = v[i];
  }
}

template <int kThreads, int kPer>
__global__ void __launch_bounds__(kThreads) pd_batch_tables(const __grid_constant__ TablesParams p) {
  constexpr int kWarps = kThreads / 32, kTokens = kThreads * kRun;
  __shared__ Sums warp_sums[kWarps];
  __shared__ int warp_max[kWarps];
  // by token: the request noted there (or -1), its start, cached tokens, pages before it
  __shared__ __align__(16) int owner[kTokens];
  __shared__ int o_start[kTokens], o_ctx[kTokens];
  __shared__ unsigned int o_off[kTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool requests = blockIdx.x == 0;
  const int t0 = requests ? 0 : (int)(blockIdx.x - 1) * kTokens;
  const int t1 = requests ? 0 : min(p.T - t0, kTokens) + t0;
  *reinterpret_cast<int4 *>(owner + kRun * tid) = make_int4(-1, -1, -1, -1);
  // the lengths may be the previous kernel's outputs
  grid_dependency_wait();
  grid_dependents_launch();
  constexpr int kRequests = kThreads * kPer;  // of a pass
  const unsigned int T = (unsigned)p.T;
  const unsigned int cap = (unsigned)p.bt_width * (unsigned)p.P;  // tokens a table row can address
  unsigned int bad = 0;
  const int cursor = p.cursor ? __ldg(p.cursor) : 0;
  Sums carry = {0, 0};
  // (a token block stops at the first pass that starts past its tokens)
  for (int base = 0; base < p.S && (requests || (int)carry.tok < t1); base += kRequests) {
    const int s0 = base + kPer * tid;
    int c_in[kPer], q_in[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c_in[i] = s0 + i < p.S ? __ldg(p.context + s0 + i) : 0;
      q_in[i] = s0 + i < p.S ? __ldg(p.query + s0 + i) : 0;
    }
    auto ctx = [&](int i) { return min((unsigned)max(c_in[i], 0), cap); };
    auto want = [&](int i) {
      const unsigned int c = ctx(i), q = min((unsigned)max(q_in[i], 0), T);
      return Sums{q, cdiv_p(min(c + q, cap), p) - cdiv_p(c, p)};
    };
    Sums own = {0, 0};
#pragma unroll
    for (int i = 0; i < kPer; ++i) own = add(own, want(i), T);
    Sums x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums y = {__shfl_up_sync(0xffffffffu, x.tok, o), __shfl_up_sync(0xffffffffu, x.pages, o)};
      if (lane >= o) x = add(y, x, T);
    }
    if (lane == 31) warp_sums[warp] = x;
    // the sums before this thread's first request
    Sums run = {__shfl_up_sync(0xffffffffu, x.tok, 1), __shfl_up_sync(0xffffffffu, x.pages, 1)};
    if (lane == 0) run = {0, 0};
    __syncthreads();
    Sums before = carry;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) before = carry;
      carry = add(carry, warp_sums[w], T);
    }
    run = add(before, run, T);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = s0 + i;
      const Sums start = run, end = add(run, want(i), T);
      run = end;
      if (s >= p.S) break;
      const unsigned int c = ctx(i), len = min(c + (end.tok - start.tok), cap);
      if (requests) {
        p.query_start[s] = (int)start.tok;
        p.seq_lens[s] = (int)len;
        if (c_in[i] < 0 || q_in[i] < 0 || (unsigned)max(c_in[i], 0) > cap ||
            c + (end.tok - start.tok) > cap)
          bad |= PD_DEV_BAD_SEQLEN;
        if ((unsigned)max(q_in[i], 0) != end.tok - start.tok) bad |= PD_DEV_BAD_QSTART;
        if (s == p.S - 1) p.query_start[p.S] = (int)end.tok;
        // the last request with tokens before T closes the pages' sum (those
        // after it take no token and no page)
        if (p.next_cursor && start.tok < T && (s == p.S - 1 || end.tok == T)) {
          const int64_t n = (int64_t)cursor +
                            (p.free_pages ? start.pages + (cdiv_p(len, p) - cdiv_p(c, p)) : 0u);
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
    __syncthreads();
  }
  if (requests) {
    if (tid == 0) {
      if (p.S == 0) p.query_start[0] = 0;
      if (p.next_cursor && (p.S == 0 || p.T == 0)) *p.next_cursor = cursor;
    }
    if (bad) atomicOr(p.status, bad);
    return;
  }
  // ---- the tokens: the request noted last at or before each of them --------
  __syncthreads();
  const int4 mine = *reinterpret_cast<const int4 *>(owner + kRun * tid);
  int at = mine.w >= 0   ? kRun * tid + 3
           : mine.z >= 0 ? kRun * tid + 2
           : mine.y >= 0 ? kRun * tid + 1
           : mine.x >= 0 ? kRun * tid
                         : -1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at = max(at, y);
  }
  if (lane == 31) warp_max[warp] = at;
  at = __shfl_up_sync(0xffffffffu, at, 1);  // before this thread's first token
  if (lane == 0) at = -1;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) at = max(at, warp_max[w]);
  const int first = t0 + kRun * tid;
  if (first >= t1) return;
  // (every load of the four tokens is under way before one is used)
  const int noted[kRun] = {mine.x, mine.y, mine.z, mine.w};
  int pos[kRun], slot[kRun], in[kRun], id[kRun], ahead[kRun];
  int32_t *opened[kRun];  // the table's entry of a page that the token opens
  bool free_page[kRun], held[kRun];
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    const int t = first + k;
    if (noted[k] >= 0) at = kRun * tid + k;
    // (carry.tok: the tokens of all requests, or of enough of them to pass t1)
    const bool live = t < t1 && t < (int)carry.tok;
    const int o = live ? at : 0;
    const int s = live ? owner[o] : 0;
    const unsigned int c = (unsigned)o_ctx[o], i = (unsigned)(t - o_start[o]);
    const unsigned int at_pos = c + i, page = div_p(at_pos, p), have = cdiv_p(c, p);
    held[k] = live && at_pos < cap;
    free_page[k] = held[k] && p.free_pages && page >= have;
    in[k] = (int)(at_pos - page * p.P);
    pos[k] = live ? (int)at_pos : 0;
    ahead[k] = live && p.delta ? __ldg(p.delta + s) : 0;
    int32_t *entry = p.table + (int64_t)s * p.bt_stride + page;
    opened[k] = free_page[k] && in[k] == 0 ? entry : nullptr;
    id[k] = -1;
    if (free_page[k]) {
      const int64_t f = (int64_t)cursor + (int64_t)(o_off[o] + (page - have));
      if (f >= 0 && f < p.num_free)
        id[k] = __ldg(p.free_pages + f);
      else {
        bad |= PD_DEV_NO_PAGE;
        held[k] = false;
      }
    } else if (held[k]) {
      id[k] = *entry;
    }
  }
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    if (held[k] && (unsigned)id[k] >= (unsigned)p.num_pages) {
      bad |= PD_DEV_BAD_PAGE;
      id[k] = -1;
    }
    if (opened[k]) *opened[k] = id[k];
    slot[k] = id[k] >= 0 ? id[k] * p.P + in[k] : -1;
    pos[k] += ahead[k];
  }
  for (int a = 0; a < p.axes; ++a) store4(p.positions + a * p.pos_stride + first, pos, t1 - first);
  store4(p.slots + first, slot, t1 - first);
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
  if (S < 0 || S > INT32_MAX - kMany * kPerMany || T < 0 || T > INT32_MAX - kMany * kRun) return PD_EINVAL;
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
  int lg = 0;
  while (((int64_t)1 << lg) < page_size) ++lg;
  p.shift = 31 + lg;
  p.magic = ((1ull << p.shift) + page_size - 1) / page_size;
  p.num_pages = num_pages;
  p.status = status;

  cudaLaunchConfig_t cfg = {};
  const int threads = S <= kFew ? kFew : kMany, tokens = threads * kRun;
  cfg.gridDim = dim3((unsigned)(1 + (T + tokens - 1) / tokens));
  cfg.blockDim = dim3(threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = S <= kFew ? cudaLaunchKernelEx(&cfg, pd_batch_tables<kFew, 1>, p)
                                  : cudaLaunchKernelEx(&cfg, pd_batch_tables<kMany, kPerMany>, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return PD_ECUDA;
  }
  return PD_OK;
}
