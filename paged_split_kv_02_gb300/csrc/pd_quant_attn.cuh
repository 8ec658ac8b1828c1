// Decode attention over an 8-bit cache.
//
// One wave of CTAs divides the keys of all requests (past 448 a wave for each 448): the
// 16-key blocks of every (sequence, kv head, row group) unit, plus a unit cost for its
// epilogue, form one line, and every CTA takes the same length of it (as pd_window.cuh
// does).  Groups without a row of a short request count as the others do.  A
// unit that the shares cut is merged by the CTA that publishes its last part.
//
// Within a CTA every warp works alone: it takes every so many steps of the CTA's
// blocks, copies K and V of each with cp.async into slots of a ring of its own and
// computes on them, with no barrier before the unit's end.  Copies of 16 bytes a lane
// gather any layout; a TMA box of one block of one head is 2 KiB at D = 128, and such
// boxes stream at 5.0 TB/s where such rings read 7.0 (12 warps, 3 slots of 4 KiB each).
//
// The products run on 16-bit floats.  Every e4m3 code is a half: a register of four
// codes becomes two of two halves each.  Keys sit on the MMA's M side: S^T = K Q^T
// and O^T += V^T P^T.  The order of the summed dims is free, so that one
// register of a K row (four codes side by side) gives both halves of an A fragment's
// row, and the transposed load of two codes a lane gives the even and the odd
// dims of a V fragment.  (The legacy MMAs of 8-bit floats are no faster: a 16 x 8 x
// 32 one takes 18.5 clocks of a sub-partition with its operands' conversions
// inside, two 16 x 8 x 16 of halves 16.2.)  bf16 queries are scaled by a power of two per row
// into the halves' range, which loses nothing above 2^-31 of the row's largest.
//
// The scales stay out of the products: S is scaled by its block's key scale in
// fp32; V's goes into the weights, a = s + log2(v_scale), p = 2^(a - max a), and
// out again in the sum l += p / v_scale, so P lies in [0, 2^15] whatever the scales
// are.  (Two scales 2^96 apart still leave the smaller one's weights 2^37 of range.)
//
// What bounds it.  Many keys of few rows: the cache's bytes, 64 requests of 4,096
// tokens, 32 / 8 heads of 128: 90 us, 6.0 TB/s, 88 % of a copy's rate.  16 rows and
// more of a kv head: conversions and MMAs, 800 clocks of a sub-partition for 16 keys of
// 256 dims and 16 rows, 518 of them the MMAs.  Short calls: the chain of one
// share, 5 us to the first keys (lengths 0.6, places 1.5, table and copies 3), 2 to 3 at a
// unit's end, 1 to publish a part and 3 to merge them, most of it code that runs once
// and is fetched while it runs: one request of 300 tokens, 16 / 4 heads of 64, 7.6 us.
#pragma once

#include <cuda_fp16.h>

#include "pd_e4m3.cuh"
#include "pd_kernel.cuh"
#include "pd_quant.h"

namespace pd {

// P = 2^(a - m), m a reference that follows the largest a: raised where a row's a
// would pass 2^15 (a half's largest is 2^16), to where the largest is 2^7, so it
// moves rarely and P loses bits of its 11 below 2^-21 of the largest alone.  The MMAs
// take 16 bits: each P is rounded, by 2^-11 of it at most, where the sum l takes it
// as it was.  An output is off by at most 2^-11 of sum p |v| / sum p, and in fact, the
// roundings being of either sign, by about a tenth more than without (fp16: 5.1e-5
// root mean square for 4.5e-5 at 300 keys; bf16 0.2 %).  Halves keep three bits more
// than the bf16 weights of the 16-bit cache's attention.
constexpr float kQuantTop = 7.f, kQuantMost = 15.f;
// 2^-64 and 2^32 as bits, the range of the scales: what is not a positive number of
// it (NaN and infinity too) lies past it as a number without a sign.  The largest of
// a piece is kept, two instructions a block, and looked at when the piece ends: 0 to
// 2.4 % of a call (a test in each step 1 to 7, one of each run of steps 0 to 5).
constexpr uint32_t kQuantLeast = (127u - 64) << 23, kQuantLargest = (127u + 32) << 23;

// 4- and 16-byte copies global -> shared by address, and this thread's groups.
__device__ __forceinline__ void copy_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D(16x8, f32) = A(16x16) * B(16x8) of halves.
__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// 4 values rounded to 16 bits
template <bool BF16>
__device__ __forceinline__ void store_four(void *dst, const float4 &v, float inv) {
  using tag = std::integral_constant<bool, BF16>;
  *reinterpret_cast<uint2 *>(dst) =
      make_uint2(pack2(v.x * inv, v.y * inv, tag{}), pack2(v.z * inv, v.w * inv, tag{}));
}

__device__ __forceinline__ void add_scaled(float4 &o, float f, const float4 &a) {
  o.x = fmaf(f, a.x, o.x);
  o.y = fmaf(f, a.y, o.y);
  o.z = fmaf(f, a.z, o.z);
  o.w = fmaf(f, a.w, o.w);
}

// The keys of a sequence that its rows see, in 16-key blocks.
struct QuantSeq {
  int L, q0, ml;               // keys, first q / out row, query tokens
  int u_lo, u_hi;              // union of its rows' windows
  int sk_nb, sk_gap;           // blocks of the sinks, blocks left out after them
  int nb;                      // blocks with visible keys
  int all_lo, all_hi, all_sk;  // of those, [all_lo, all_hi) and [0, all_sk) are seen whole by every row
};

__device__ __forceinline__ QuantSeq quant_seq(int L, int q0, int ml, int window, int sinks) {
  QuantSeq r;
  r.L = L;
  r.q0 = q0;
  r.ml = ml;
  const int n0 = ml > 0 ? max(L - ml + 1, 0) : 0, n1 = ml > 0 ? L : 0;  // keys of the first, the last row
  r.u_hi = n1;
  r.u_lo = window > 0 ? max(0, n0 - window) : 0;
  const int first = r.u_lo / kBlockKeys, last = (n1 + kBlockKeys - 1) / kBlockKeys;
  r.sk_nb = window > 0 ? (min(sinks, n1) + kBlockKeys - 1) / kBlockKeys : 0;
  r.sk_gap = max(0, first - r.sk_nb);
  r.nb = n1 > r.u_lo ? last - r.sk_gap : 0;
  const int v_lo = window > 0 ? max(0, n1 - window) : 0;
  const int whole = (v_lo + kBlockKeys - 1) / kBlockKeys - r.sk_gap;
  r.all_lo = r.sk_gap > 0 ? max(r.sk_nb, whole) : whole;
  r.all_hi = n0 / kBlockKeys - r.sk_gap;
  r.all_sk = window > 0 ? min(sinks, n0) / kBlockKeys : 0;
  return r;
}

// n / d for n >= 0 below 2^31 and a quotient below 2^16 (the approximate one is at
// most one off).
__device__ __forceinline__ int div_near(int n, int d) {
  int q = __float2int_rz(__fdividef((float)n, (float)d));
  const int r = n - q * d;
  if (r < 0) --q;
  if (r >= d) ++q;
  return q;
}

// A run of steps of a warp within a piece: its copies' cursor.
struct QuantRun {
  int k;                // piece
  int first, mine;      // the warp's first step of it, and its number of them
  int base;             // the run's first of those
  int b0, b1, sk_nb, sk_gap;
  int s, h;
};

// A piece of a CTA's share: some or all blocks of one unit.
struct QuantPiece {
  QuantSeq r;
  int s, h, g;          // sequence, kv head, row group
  int b0, b1;           // its blocks of the unit
  int part, parts, first_cta;
};

static_assert(sizeof(QuantRun) == kQuantRunBytes && sizeof(QuantPiece) <= kQuantPieceBytes, "their shared memory");

template <int D, int NT, bool BF16>
__global__ void __launch_bounds__(32 * kQuantWarps, 1) pd_quant_decode(const __grid_constant__ QuantAttnParams p) {
  constexpr int NW = kQuantWarps;
  constexpr int TB = quant_step_blocks(D, NT), NS = quant_slots(D, NT);
  constexpr int BLOCK = 16 * D;               // bytes of K (or V) of a block
  constexpr int SLOT = quant_slot_bytes(D, NT);  // TB blocks of K, and their scales, or of V
  constexpr int CPR = D / 16;                 // 16-byte chunks of a row
  constexpr int RPI = 32 / CPR;               // rows that 32 lanes copy at once (D = 512: 1)
  constexpr int COPIES = D / 32;              // copies of a lane for K (or V) of a block
  constexpr int NR = 8 * NT;                  // rows of the CTA, padded
  constexpr int PASSES = quant_passes(D, NT), DC = D / PASSES, CPP = CPR / PASSES;
  constexpr int SWIZZLE = DC >= 32 ? 24 : DC - 8;  // of the columns of the warps' sums
  constexpr int COST = quant_unit_cost(D);
  constexpr int SPC = 32 / TB;                // steps whose page ids a warp holds
  constexpr int NTHR = 32 * NW;
  constexpr int kPieces = kQuantPieces;       // pieces whose place is known at a time

  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char *ring = smem + warp * (NS * SLOT);
  uint2 *qfrag = reinterpret_cast<uint2 *>(smem + NW * NS * SLOT);         // [2][CPR][NT][32]
  float *rowsc = reinterpret_cast<float *>(qfrag + 2 * CPR * NT * 32);     // [2][NR]
  int *rowhi = reinterpret_cast<int *>(rowsc + 2 * NR);                    // [2][NR]
  float2 *ml_of = reinterpret_cast<float2 *>(rowhi + 2 * NR);              // [NR][NW] (m, l) of the warps
  QuantPiece *pieces = reinterpret_cast<QuantPiece *>(ml_of + NR * NW);    // [kPieces], by piece % kPieces
  QuantPiece *cut_piece = pieces + kPieces;                                // [2]
  QuantRun *runs = reinterpret_cast<QuantRun *>(cut_piece + 2) + 2 * warp;  // [NW][2]
  int *sums = reinterpret_cast<int *>(runs - 2 * warp + 2 * NW);           // [NW]
  int *free_slot = sums + NW;                                              // [NW]
  volatile int *flag = free_slot + NW;                                     // [8]
  int *lens = free_slot + NW + 8;                                          // [seqs]
  int *starts = lens + p.seqs_y;                                           // [seqs + 1]
  int *blocks = starts + p.seqs_y + 1;                                     // [seqs] with visible keys
  // of the sequences that have some, in order: which, and their places on the line
  int *order = blocks + p.seqs_y;                                          // [seqs]
  int *place = order + p.seqs_y;                                           // [seqs]

  const int s_first = blockIdx.y * p.seqs_y, S = min(p.seqs_y, p.num_seqs - s_first);
  const int HR = p.Hkv * p.rg;  // units of a sequence

  grid_dependency_wait();

  // ---- the lengths, clamped and reported; their places on the line -----------
  // (a thread has a run of sequences)
  const int per = (S + NTHR - 1) / NTHR, i0 = min(tid * per, S), i1 = min(i0 + per, S);
  const int G = gridDim.x;
  int sum = 0, full = 0;  // its blocks, and its sequences that have some
  {
    const int cap = p.bt_width * p.P;
    unsigned int bad = 0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      int L = __ldg(p.seq_lens + s_first + i), ml = p.M;
      if (p.query_start) {
        const int a = __ldg(p.query_start + s_first + i), b = __ldg(p.query_start + s_first + i + 1);
        const int q0 = min(max(a, 0), p.num_tokens), q1 = min(max(b, 0), p.num_tokens);
        ml = min(max(q1 - q0, 0), p.M);
        starts[i] = q0;
        starts[i + 1] = q1;  // (what the next one writes there too)
        if (a < 0 || b > p.num_tokens || b < a || b - a > p.M) bad |= PD_DEV_BAD_QSTART;
      }
      if (L > cap) bad |= PD_DEV_BAD_SEQLEN;
      L = min(max(L, 0), cap);
      const int nb = quant_seq(L, 0, ml, p.window, p.sinks).nb;
      lens[i] = L;
      blocks[i] = nb;
      sum += nb;
      full += nb > 0;
    }
    if (bad && blockIdx.x == 0) atomicOr(p.status, bad);
  }
  // sums over the CTA's threads: inclusive, and of all
  auto scan = [&](int v, int *all) -> int {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      if (i == warp) v += total;
      total += sums[i];
    }
    *all = total;
    return v;
  };
  if (tid == 0) {
    flag[0] = 1;
    flag[1] = flag[2] = 0;
  }
  auto seq_of = [&](int i) -> QuantSeq {
    int q0 = (s_first + i) * p.M, ml = p.M;
    if (p.query_start) {
      q0 = starts[i];
      ml = min(max(starts[i + 1] - q0, 0), p.M);
    }
    return quant_seq(lens[i], q0, ml, p.window, p.sinks);
  };

  // ---- this CTA's share -------------------------------------------------------
  // A length of the line, from any place of a unit to any of another (a unit counts
  // COST beside its blocks); or, where units are few and it costs little, of a
  // line on which every unit has a whole number of shares: no CTA then ends two units.
  // (whole: a CTA has a unit, there being no scratch for parts.)
  int U, N, unit0, n_pieces;
  int rank = scan(full, &U) - full;
  scan(sum, &N);
  U *= HR;  // units with blocks, and the blocks
  N *= HR;
  int share = p.by_ctas.div(N + U * COST + G - 1), even = 0;
  if (2 * U <= G && U > 0) {
    // parts of s blocks take N / s + U CTAs at most; of one sequence, whose units are alike, no more than
    // G (approximate quotients, rounded up past their error)
    const int m = S == 1 ? U * div_near(G, U) : G - U;
    const int s = (int)(1.f + 1.00001f * __fdividef((float)N, (float)m));
    if (s <= share + COST) even = max(s, p.min_part);
  }
  share = even > 0 ? even : max(share, p.min_share);
  auto cost_of = [&](int nb) { return even > 0 ? (div_near(nb - 1, share) + 1) * share : nb + COST; };
  sum = 0;
#pragma unroll 1
  for (int i = i0; i < i1; ++i)
    if (blocks[i] > 0) sum += cost_of(blocks[i]) * HR;
  int W, line_at = scan(sum, &W) - sum;
  const int x0 = (int)min((int64_t)blockIdx.x * share, (int64_t)W), x1 = (int)min((int64_t)x0 + share, (int64_t)W);
  // the sequences' places, and the units that the share's first and last place are in
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    const int nb = blocks[i];
    if (nb == 0) continue;
    order[rank] = i;
    place[rank] = line_at;
    const int cost = cost_of(nb), next = line_at + cost * HR;
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      const int x = e ? x1 - 1 : x0;
      if (x0 >= x1 || x < line_at || x >= next) continue;
      const int k = div_near(x - line_at, cost), in = x - line_at - k * cost;
      // (not a first unit whose blocks lie before the share; and does the last one go on behind it)
      flag[e] = rank * HR + k + (!e && in >= nb ? 1 : 0);
      if (e) flag[2] = in + 1 < nb;
    }
    line_at = next;
    ++rank;
  }
  __syncthreads();
  if (p.whole) {
    unit0 = (int)((int64_t)U * blockIdx.x / G);
    n_pieces = (int)((int64_t)U * (blockIdx.x + 1) / G) - unit0;
  } else {
    unit0 = flag[0];
    n_pieces = flag[1] - unit0 + 1;
  }
  // a unit that goes on behind the share comes first, so that its part is out early
  const bool tail = n_pieces > 1 && flag[2] && !p.whole;

  using Piece = QuantPiece;
  auto piece_at = [&](int k) -> Piece {
    const int u = unit0 + (tail ? (k == 0 ? n_pieces - 1 : k - 1) : k);
    Piece q;
    const int j = p.by_units.div(u), hr = u - j * HR, i = order[j];
    q.s = s_first + i;
    q.h = p.by_groups.div(hr);
    q.g = hr - q.h * p.rg;
    q.r = seq_of(i);
    const int nb = q.r.nb;
    q.b0 = 0;
    q.b1 = nb;
    q.part = 0;
    q.parts = 1;
    q.first_cta = blockIdx.x;
    if (!p.whole) {
      const int a = place[j] + hr * cost_of(nb);
      q.b0 = max(x0 - a, 0);
      q.b1 = min(x1 - a, nb);
      if (q.b1 - q.b0 < nb) {
        q.first_cta = div_near(a, share);
        q.part = (int)blockIdx.x - q.first_cta;
        q.parts = div_near(a + nb - 1, share) - q.first_cta + 1;
      }
    }
    return q;
  };
  if (tid < min(n_pieces, kPieces - 1)) pieces[tid] = piece_at(tid);
  __syncthreads();

  // ---- the copies: a cursor over the steps of this warp ----------------------
  // Step st of a piece is blocks b0 + st TB ..; a warp takes steps first, first +
  // NW, .., the first one moving on with the pieces so that odd ones are spread.
  // The page ids of a run of up to SPC steps are held, one block a lane; the run
  // after it is looked up while this one is copied.  What a run does not change
  // from step to step lies in shared memory: registers are for the products.
  auto enter = [&](QuantRun &c, int k) {
    c.k = k;
    c.base = c.mine = 0;
    if (k >= n_pieces) return;
    const Piece &q = pieces[k & (kPieces - 1)];
    const int steps = (q.b1 - q.b0 + TB - 1) / TB;
    c.first = (warp + k) & (NW - 1);
    c.mine = (steps + NW - 1 - c.first) / NW;
    c.b0 = q.b0;
    c.b1 = q.b1;
    c.sk_nb = q.r.sk_nb;
    c.sk_gap = q.r.sk_gap;
    c.s = q.s;
    c.h = q.h;
  };
  auto fetch_ids = [&](const QuantRun &c) -> int {
    if (c.k >= n_pieces) return 0;
    const int b = c.b0 + (c.first + (c.base + lane / TB) * NW) * TB + lane % TB;
    if (c.base + lane / TB >= c.mine || b >= c.b1) return 0;
    const int sb = b >= c.sk_nb ? b + c.sk_gap : b;
    return __ldg(p.block_table + (int64_t)c.s * p.bt_stride + p.by_page.div(sb));
  };
  int which = 0;        // the present run; the next one lies beside it
  int at = 0, end = 0;  // steps of it
  int ids_ahead = 0;
  bool look = false;    // the next run is still to be looked up
  // of the present run, a block a lane: where its K, V and their scales are (K at -1: there is none)
  int64_t k_at = -1, v_at = -1, ks_at = 0, vs_at = 0;
  // the run after c: of its piece, or of the next one that has a step for this warp (a
  // piece has a block, so one of NW pieces has: kPieces cover all that a warp looks ahead)
  auto look_ahead = [&](QuantRun c) {
    c.base += SPC;
    while (c.k < n_pieces && c.base >= c.mine) enter(c, c.k + 1);
    ids_ahead = fetch_ids(c);
    __syncwarp();
    if (lane == 0) runs[which ^ 1] = c;
    __syncwarp();
  };
  auto next_run = [&]() {
    which ^= 1;
    const QuantRun &c = runs[which];
    at = 0;
    end = c.k < n_pieces ? min(SPC, c.mine - c.base) : 0;
    look = true;
    const int b = c.b0 + (c.first + (c.base + lane / TB) * NW) * TB + lane % TB;
    k_at = v_at = -1;
    if (lane / TB < end && b < c.b1) {
      int page = ids_ahead;
      if ((unsigned)page >= (unsigned)p.num_pages) {
        atomicOr(p.status, PD_DEV_BAD_PAGE);  // report, read page 0
        page = 0;
      }
      const int sb = b >= c.sk_nb ? b + c.sk_gap : b;
      const int sub = sb - (int)p.by_page.div(sb) * p.bpp;
      k_at = page * p.k.page + c.h * p.k.head + (sub * kBlockKeys) * p.k.tok;
      v_at = page * p.v.page + c.h * p.v.head + (sub * kBlockKeys) * p.v.tok;
      ks_at = page * p.k.s_page + sub * p.k.s_blk + c.h * p.k.s_head;
      vs_at = page * p.v.s_page + sub * p.v.s_blk + c.h * p.v.s_head;
    }
  };
  {
    QuantRun c{};
    c.k = n_pieces > 0 ? -1 : 0;
    look_ahead(c);
    next_run();
  }
  const int c_row = lane / CPR, c_ch = lane % CPR;  // (D = 512: row 0, chunk = lane)
  auto place_of = [&](int row, int ch) -> uint32_t {
    return D >= 128 ? row * D + ((ch ^ (row & 7)) << 4) : row * D + ((ch ^ ((row >> 1) & 3)) << 4);
  };
  const unsigned char *k_lane = p.k.codes + c_row * p.k.tok + c_ch * 16;
  const unsigned char *v_lane = p.v.codes + c_row * p.v.tok + c_ch * 16;
  int in_slot = 0;     // the slot that the next copies go to
  const uint32_t ring_at = smem_u32(ring);
  // the next slot's copies: the present step's K and scales, or its V and on to the next step
  auto issue = [&](bool is_v) {
    if (at < end) {
      const int64_t tok = is_v ? p.v.tok : p.k.tok;
      const uint32_t slot = ring_at + in_slot * SLOT;
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        const int64_t from = __shfl_sync(0xffffffffu, is_v ? v_at : k_at, at * TB + b);
        if (from >= 0) {
          const unsigned char *src = (is_v ? v_lane : k_lane) + from;
          if (tok == D) {
            // (rows one after the other: offsets are constants)
#pragma unroll
            for (int j = 0; j < COPIES; ++j)
              copy_async16(slot + b * BLOCK + place_of(c_row + j * RPI, c_ch), src + j * (RPI * D));
          } else {
#pragma unroll
            for (int j = 0; j < COPIES; ++j)
              copy_async16(slot + b * BLOCK + place_of(c_row + j * RPI, c_ch), src + (int64_t)(j * RPI) * tok);
          }
        }
      }
      if (!is_v) {
        // a lane a scale: K's and V's of a block side by side (of one that is not there: 1, which is
        // in the range)
        const int from = at * TB + (lane >> 1) % TB;
        const int64_t there = __shfl_sync(0xffffffffu, k_at, from);
        const int64_t ks = __shfl_sync(0xffffffffu, ks_at, from), vs = __shfl_sync(0xffffffffu, vs_at, from);
        if (lane < 2 * TB) {
          if (there >= 0)
            copy_async4(slot + TB * BLOCK + lane * 4, lane & 1 ? p.v.scale + vs : p.k.scale + ks);
          else
            reinterpret_cast<float *>(ring + in_slot * SLOT + TB * BLOCK)[lane] = 1.f;
        }
      } else {
        ++at;
        if (look) {
          look_ahead(runs[which]);
          look = false;
        }
        if (at == end) next_run();
      }
    }
    if (++in_slot == NS) in_slot = 0;
    copy_commit();
  };

  // ---- Q of a piece: halves in fragment order, row scales, row ends ----------
  using T = std::conditional_t<BF16, __nv_bfloat16, __half>;
  const T *qbase = static_cast<const T *>(p.q);
  T *obase = static_cast<T *>(p.out);
  constexpr int QV = D >= 128 ? D / 128 : 1;
  auto row_live = [&](const Piece &q, int rr) {
    return rr < p.rows_grp && q.g * p.rows_grp + rr < q.r.ml * p.G;
  };
  uint2 qw[NT][QV];  // a warp's rows: warp, warp + NW, ..
  static_assert(NW == 8, "a warp has NT rows of Q");
  auto fetch_q = [&](const Piece &q) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int rr = warp + NW * n;
      const bool live = row_live(q, rr);
      const int pr = q.g * p.rows_grp + rr;
      const int t = live ? (int)p.by_heads.div(pr) : 0, jq = live ? pr - t * p.G : 0;
      const uint2 *src = reinterpret_cast<const uint2 *>(
          qbase + (int64_t)(q.r.q0 + t) * p.q_s0 + (int64_t)(q.h * p.G + jq) * p.q_s1);
#pragma unroll
      for (int v = 0; v < QV; ++v)
        qw[n][v] = live && (D >= 128 || lane < D / 4) ? __ldg(src + v * 32 + lane) : make_uint2(0u, 0u);
    }
  };
  auto put_q = [&](const Piece &q, int buf) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int rr = warp + NW * n;
      float f = 1.f;
      if constexpr (BF16) {
        // the row's largest magnitude to [2^14, 2^15)
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < QV; ++v)
          top = max(max(max(qw[n][v].x & 0x7fffu, (qw[n][v].x >> 16) & 0x7fffu),
                        max(qw[n][v].y & 0x7fffu, (qw[n][v].y >> 16) & 0x7fffu)), top);
        top = __reduce_max_sync(0xffffffffu, top);
        // 2^(14 - e), e the exponent of the largest, within fp32's range
        const int e = min(max((int)(top >> 7) - 127, -100), 127);
        const float up = __int_as_float((14 - e + 127) << 23);
        f = __int_as_float((e - 14 + 127) << 23);
        auto halves = [&](uint32_t b) -> uint32_t {
          return pack2(__uint_as_float(b << 16) * up, __uint_as_float(b & 0xffff0000u) * up,
                       std::integral_constant<bool, false>{});
        };
#pragma unroll
        for (int v = 0; v < QV; ++v) qw[n][v] = make_uint2(halves(qw[n][v].x), halves(qw[n][v].y));
      }
#pragma unroll
      for (int v = 0; v < QV; ++v) {
        const int d4 = v * 32 + lane;  // dims 4 d4 ..
        if (D >= 128 || lane < D / 4)
          qfrag[((buf * CPR + (d4 >> 2)) * NT + n) * 32 + warp * 4 + (d4 & 3)] = qw[n][v];
      }
      if (lane == 0) {
        rowsc[buf * NR + rr] = f * p.scale_log2;
        rowhi[buf * NR + rr] =
            row_live(q, rr) ? max(q.r.L - q.r.ml + (int)p.by_heads.div(q.g * p.rows_grp + rr) + 1, 0) : 0;
      }
    }
  };
  const int g8 = lane >> 2, t4 = lane & 3;
  const int a_row = lane & 15, a_hi = lane >> 4;  // the rows and chunk of ldmatrix's addresses
  auto sees = [&](int key, int lo, int hi) { return key < hi && (key >= lo || key < p.sinks); };
  int out_slot = 0;   // the slot of the next step's K
  int n_cut = 0;      // cut units of this share whose part is out
  int cut_old0 = 0, cut_old1 = 0;

  // the rows of a unit in q and out, and the scratch slot of a part of it
  auto out_row = [&](const Piece &q, int rr) -> T * {
    const int pr = q.g * p.rows_grp + rr, t = p.by_heads.div(pr), jq = pr - t * p.G;
    return obase + (int64_t)(q.r.q0 + t) * p.o_s0 + (int64_t)(q.h * p.G + jq) * p.o_s1;
  };
  // Parts of a unit are merged in groups, and then the groups, where they are many: one
  // CTA pulls parts at about 80 GB/s, so 152 parts of 16 KiB take it 30 us, in 13
  // groups two times 2.5.  Each group has a counter beside the unit's.
  auto group_size = [&](const Piece &q) -> int {
    if (p.unit_counters < 3 || q.parts * (NR * D / 32) <= p.merge_bytes / 128) return q.parts;
    int g = 2;
    while (g * g < q.parts) ++g;
    return max(g, (q.parts + p.unit_counters - 2) / (p.unit_counters - 1));
  };
  auto counter_of = [&](const Piece &q, int group) -> int * {
    const int64_t unit = (int64_t)((q.s * p.Hkv + q.h) * p.rg + q.g) * p.unit_counters;
    return p.counters + unit + (group_size(q) < q.parts ? 1 + group : 0);
  };
  auto slot_of = [&](const Piece &q, int part) -> int64_t {
    const int64_t c = (int64_t)blockIdx.y * gridDim.x + q.first_cta + part;
    return part == 0 ? 2 * c + 1 : 2 * c;
  };

  // (from -1 on: the first copies and the first Q)
#pragma unroll 1
  for (int k = n_pieces > 0 ? -1 : 0; k < n_pieces; ++k) {
    const int buf = k & 1;
    const Piece &q = pieces[k & (kPieces - 1)];
    const uint2 *qf = qfrag + buf * CPR * NT * 32 + lane;
    const int first = (warp + k) & (NW - 1);
    const int mine = k < 0 ? 0 : ((q.b1 - q.b0 + TB - 1) / TB + NW - 1 - first) / NW;
    const bool more = k + 1 < n_pieces;
    constexpr bool EARLY = NT * QV <= 2;  // the next Q is fetched while this piece runs
    if (more && (EARLY || k < 0)) fetch_q(pieces[(k + 1) & (kPieces - 1)]);
    float acc[CPR][NT][4];
#pragma unroll
    for (int c = 0; c < CPR; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[c][n][0] = acc[c][n][1] = acc[c][n][2] = acc[c][n][3] = 0.f;
    // rows 8 n + 2 t4, + 1 of this thread: P's reference (m - kQuantTop; a row
    // without one yet, 0), its sum, the scale of its scores
    float mu[NT][2], l[NT][2], rs[NT][2];
    bool has[NT][2];
    constexpr bool QREG = NT * CPR <= 16;  // Q's fragments in registers
    uint2 qr[QREG ? CPR : 1][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float2 r = *reinterpret_cast<const float2 *>(rowsc + buf * NR + 8 * n + 2 * t4);
      const int2 hi = *reinterpret_cast<const int2 *>(rowhi + buf * NR + 8 * n + 2 * t4);
      rs[n][0] = r.x;
      rs[n][1] = r.y;
      has[n][0] = hi.x <= 0;  // (a row without keys needs none)
      has[n][1] = hi.y <= 0;
      mu[n][0] = mu[n][1] = l[n][0] = l[n][1] = 0.f;
      if constexpr (QREG) {
#pragma unroll
        for (int c = 0; c < CPR; ++c) qr[c][n] = qf[(c * NT + n) * 32];
      }
    }
    bool settled = false;  // every row has its reference
    uint32_t past = 0;     // how far scales lie past their range, as numbers
    uint32_t pb[TB][NT][2];
    if (k < 0) {
#pragma unroll 1
      for (int i = 0; i < NS - 1; ++i) issue(i & 1);
    }
#pragma unroll 1
    for (int st = 0; st < mine; ++st) {
      copy_wait<NS - 2>();
      __syncwarp();
      issue((NS - 1) & 1);
      const uint32_t kb = ring_at + out_slot * SLOT;
      const int blk = q.b0 + (first + st * NW) * TB;
      // (else some row does not see them whole, or the piece does not have them)
      const bool whole = blk + TB <= q.b1 && ((blk >= q.r.all_lo && blk + TB <= q.r.all_hi) || blk + TB <= q.r.all_sk);
      const float2 *scales = reinterpret_cast<const float2 *>(ring + out_slot * SLOT + TB * BLOCK);
      if (++out_slot == NS) out_slot = 0;

      // S^T = K Q^T (in two sums where few products are independent)
      constexpr bool TWO = TB * NT <= 2;
      float sc[TB][NT][4], sd[TB][NT][4];
#pragma unroll
      for (int c = 0; c < CPR; c += 2) {
        uint2 qa[NT], qb[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          qa[n] = QREG ? qr[QREG ? c : 0][n] : qf[(c * NT + n) * 32];
          qb[n] = QREG ? qr[QREG ? c + 1 : 0][n] : qf[((c + 1) * NT + n) * 32];
        }
        uint32_t x[TB][4], y[TB][4];
#pragma unroll
        for (int b = 0; b < TB; ++b) {
          // (rows 0-7, 8-15) of chunk c, then of chunk c + 1
          uint32_t w[4];
          ldsm_x4(kb + b * BLOCK + place_of(a_row, c + a_hi), w);
          halves_of(w[0], x[b][0], x[b][2]);
          halves_of(w[1], x[b][1], x[b][3]);
          halves_of(w[2], y[b][0], y[b][2]);
          halves_of(w[3], y[b][1], y[b][3]);
        }
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (c == 0)
              mma_first(sc[b][n], x[b], qa[n].x, qa[n].y);
            else
              mma_16816<false>(sc[b][n], x[b], qa[n].x, qa[n].y);
          }
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (!TWO)
              mma_16816<false>(sc[b][n], y[b], qb[n].x, qb[n].y);
            else if (c == 0)
              mma_first(sd[b][n], y[b], qb[n].x, qb[n].y);
            else
              mma_16816<false>(sd[b][n], y[b], qb[n].x, qb[n].y);
          }
      }
      if constexpr (TWO) {
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[b][n][e] += sd[b][n][e];
      }

      // x = a - mu = log2 of P
      float inv[TB];
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        const float2 kv = scales[b];
        past = __viaddmax_u32(__float_as_uint(kv.x), 0u - kQuantLeast, past);
        past = __viaddmax_u32(__float_as_uint(kv.y), 0u - kQuantLeast, past);
        const float lg = __log2f(kv.y);
        inv[b] = sfu_rcp(kv.y);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float f0 = rs[n][0] * kv.x, f1 = rs[n][1] * kv.x, g0 = lg - mu[n][0], g1 = lg - mu[n][1];
          sc[b][n][0] = fmaf(sc[b][n][0], f0, g0);
          sc[b][n][1] = fmaf(sc[b][n][1], f1, g1);
          sc[b][n][2] = fmaf(sc[b][n][2], f0, g0);
          sc[b][n][3] = fmaf(sc[b][n][3], f1, g1);
        }
      }
      if (!whole) {
#pragma unroll
        for (int b = 0; b < TB; ++b) {
          const int i = blk + b;
          const bool there = i < q.b1;
          const int ka = (i >= q.r.sk_nb ? i + q.r.sk_gap : i) * kBlockKeys + g8, kb8 = ka + 8;
          if (!there) inv[b] = 0.f;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int2 hi = *reinterpret_cast<const int2 *>(rowhi + buf * NR + 8 * n + 2 * t4);
            const int lo0 = p.window > 0 ? max(0, hi.x - p.window) : 0;
            const int lo1 = p.window > 0 ? max(0, hi.y - p.window) : 0;
            if (!there || !sees(ka, lo0, hi.x)) sc[b][n][0] = -INFINITY;
            if (!there || !sees(ka, lo1, hi.y)) sc[b][n][1] = -INFINITY;
            if (!there || !sees(kb8, lo0, hi.x)) sc[b][n][2] = -INFINITY;
            if (!there || !sees(kb8, lo1, hi.y)) sc[b][n][3] = -INFINITY;
          }
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          top = fmaxf(fmaxf(top, fmaxf(sc[b][n][0], sc[b][n][1])), fmaxf(sc[b][n][2], sc[b][n][3]));
      if (!settled || __any_sync(0xffffffffu, top > kQuantMost)) {
        // the rows' references up to their largest a
        float al[NT][2];
        bool all = true;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = -INFINITY;
#pragma unroll
            for (int b = 0; b < TB; ++b) mx = fmaxf(mx, fmaxf(sc[b][n][e], sc[b][n][e + 2]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const bool any = mx > -INFINITY;
            const float up = !any ? 0.f : has[n][e] ? fmaxf(mx - kQuantTop, 0.f) : mx - kQuantTop;
            al[n][e] = has[n][e] ? sfu_exp2(-up) : 1.f;  // (nothing summed before the first)
            has[n][e] |= any;
            all &= has[n][e];
            mu[n][e] += up;
            l[n][e] *= al[n][e];
#pragma unroll
            for (int b = 0; b < TB; ++b) {
              sc[b][n][e] -= up;
              sc[b][n][e + 2] -= up;
            }
          }
        settled = __all_sync(0xffffffffu, all);
#pragma unroll
        for (int c = 0; c < CPR; ++c)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[c][n][0] *= al[n][0];
            acc[c][n][1] *= al[n][1];
            acc[c][n][2] *= al[n][0];
            acc[c][n][3] *= al[n][1];
          }
      }
      // P
#pragma unroll
      for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float p0 = sfu_exp2(sc[b][n][0]), p1 = sfu_exp2(sc[b][n][1]);
          const float p2 = sfu_exp2(sc[b][n][2]), p3 = sfu_exp2(sc[b][n][3]);
          l[n][0] = fmaf(p0 + p2, inv[b], l[n][0]);
          l[n][1] = fmaf(p1 + p3, inv[b], l[n][1]);
          pb[b][n][0] = movmatrix_trans(pack2(p0, p1, std::integral_constant<bool, false>{}));
          pb[b][n][1] = movmatrix_trans(pack2(p2, p3, std::integral_constant<bool, false>{}));
        }

      copy_wait<NS - 2>();
      __syncwarp();
      issue(NS & 1);
      const uint32_t vb = ring_at + out_slot * SLOT;
      // O^T += V^T P^T
      if (!whole) {
        // V of keys that no row sees (stale or NaN slots), or that are not there: zeros
#pragma unroll 1
        for (int j = lane; j < TB * kBlockKeys * CPR; j += 32) {
          const int i = blk + j / (kBlockKeys * CPR), tok = j / CPR % kBlockKeys;
          const int key = (i >= q.r.sk_nb ? i + q.r.sk_gap : i) * kBlockKeys + tok;
          if (i >= q.b1 || !sees(key, q.r.u_lo, q.r.u_hi))
            *reinterpret_cast<uint4 *>(ring + out_slot * SLOT + j * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
      }
      if (++out_slot == NS) out_slot = 0;
#pragma unroll
      for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int c = 0; c < CPR; c += 2) {
          // (keys 0-7, 8-15) of chunk c, then of chunk c + 1: two keys' codes of
          // dims 2 g8, 2 g8 + 1 a register
          uint32_t w[4];
          ldsm_x4_trans(vb + b * BLOCK + place_of(a_row, c + a_hi), w);
          uint32_t x[4], y[4];
          halves_of(__byte_perm(w[0], 0u, 0x3120), x[0], x[1]);
          halves_of(__byte_perm(w[1], 0u, 0x3120), x[2], x[3]);
          halves_of(__byte_perm(w[2], 0u, 0x3120), y[0], y[1]);
          halves_of(__byte_perm(w[3], 0u, 0x3120), y[2], y[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_16816<false>(acc[c][n], x, pb[b][n][0], pb[b][n][1]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_16816<false>(acc[c + 1][n], y, pb[b][n][0], pb[b][n][1]);
        }
    }

    // ---- the piece's end: the warps' sums added, rows stored or published ----
    // A warp's sums go to its ring's free slot (the one that the next copies are
    // for), DC columns at a time.
    if (more && !EARLY && k >= 0) fetch_q(pieces[(k + 1) & (kPieces - 1)]);
    if (k < 0) {
      put_q(pieces[0], 0);
      __syncthreads();
      continue;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
      }
      if (lane < 4) {
        // (of a row without a visible key here: no maximum)
        ml_of[(8 * n + 2 * lane) * NW + warp] = make_float2(l[n][0] > 0.f ? mu[n][0] : -INFINITY, l[n][0]);
        ml_of[(8 * n + 2 * lane + 1) * NW + warp] = make_float2(l[n][1] > 0.f ? mu[n][1] : -INFINITY, l[n][1]);
      }
    }
    if (past > kQuantLargest - kQuantLeast && lane == 0) atomicOr(p.status, PD_DEV_BAD_SCALE);
    if (lane == 0) free_slot[warp] = (warp * NS + in_slot) * SLOT;
    const bool cut = q.parts > 1;
    __syncwarp();  // (every lane has read the slot)
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
      // column d of row r at d ^ 8 (r / 2 % 4) (but for few columns): a warp's stores hit
      // every bank once
      float *mine_at = reinterpret_cast<float *>(ring + in_slot * SLOT);
#pragma unroll
      for (int c = 0; c < CPP; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int r0 = 8 * n + 2 * t4, d = (16 * c + 2 * g8) ^ ((t4 << 3) & SWIZZLE);
          const float(&a)[4] = acc[ps * CPP + c][n];
          *reinterpret_cast<float2 *>(mine_at + r0 * DC + d) = make_float2(a[0], a[2]);
          *reinterpret_cast<float2 *>(mine_at + (r0 + 1) * DC + d) = make_float2(a[1], a[3]);
        }
      __syncthreads();
#pragma unroll 1
      for (int it = tid; it < NR * (DC / 4); it += NTHR) {
        const int rr = it / (DC / 4), d4 = it - rr * (DC / 4);
        if (!row_live(q, rr)) continue;
        // the row's (m, l) of the warps, their weights and their sum
        float2 t[NW];
#pragma unroll
        for (int w = 0; w < NW; w += 2) {
          const float4 x = *reinterpret_cast<const float4 *>(ml_of + rr * NW + w);
          t[w] = make_float2(x.x, x.y);
          t[w + 1] = make_float2(x.z, x.w);
        }
        float M = t[0].x, ls = 0.f;
#pragma unroll
        for (int w = 1; w < NW; ++w) M = fmaxf(M, t[w].x);
        const float mm = M == -INFINITY ? 0.f : M;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float f = exp2_or_zero(t[w].x, mm);
          ls = fmaf(f, t[w].y, ls);
          add_scaled(o, f,
                     *reinterpret_cast<const float4 *>(smem + free_slot[w] +
                                                       4 * (rr * DC + ((4 * d4) ^ (((rr >> 1 & 3) << 3) & SWIZZLE)))));
        }
        const int d = ps * DC + 4 * d4;
        if (!cut) {
          store_four<BF16>(out_row(q, rr) + d, o, ls > 0.f ? sfu_rcp(ls) : 0.f);
        } else {
          const int64_t to = slot_of(q, q.part) * NR + rr;
          __stcg(reinterpret_cast<float4 *>(p.part_acc + to * D + d), o);
          if (d == 0) __stcg(reinterpret_cast<float2 *>(p.part_ml + to * 2), make_float2(M, ls));
        }
      }
      if (ps == PASSES - 1) {
        if (more) put_q(pieces[(k + 1) & (kPieces - 1)], buf ^ 1);
        // (the place of the piece before this one is free)
        if (tid == NTHR - 1 && k + kPieces - 1 < n_pieces) pieces[(k - 1) & (kPieces - 1)] = piece_at(k + kPieces - 1);
      }
      __syncthreads();
    }
    if (cut) {
      // every thread's stores, the barrier above, one release by one thread; the
      // count's answer is looked at when the share is done
      if (tid == 0) {
        const int old = atomic_add_acq_rel_gpu(counter_of(q, q.part / group_size(q)), 1);
        if (n_cut == 0) cut_old0 = old; else cut_old1 = old;
      }
      if (tid == 32) cut_piece[n_cut] = q;  // (read behind later barriers)
      ++n_cut;
    }
  }
  grid_dependents_launch();

  // ---- cut units whose last part is this CTA's: merged ------------------------
  // n parts from part `from` on, `step` apart: to the output, or back as part `from`.
  // Neighbouring lanes take turns at the parts of an item (a row's 4 columns).
  auto merge = [&](const Piece &q, int rows, int from, int n, int step, bool last) {
    constexpr int CH = 8;  // parts whose loads are in flight
    const int items = rows * (D / 4);
    int lg = 0;
    while (lg < 3 && (items << lg) * 2 <= NTHR) ++lg;
    const int slices = 1 << lg, slice = tid & (slices - 1);
#pragma unroll 1
    for (int it = tid >> lg; it < items; it += NTHR >> lg) {
      const int rr = it / (D / 4), d = 4 * (it - rr * (D / 4));
      float M = -INFINITY, ls = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int c0 = slice; c0 < n; c0 += CH * slices) {
        float2 t[CH];
        float4 a[CH];
#pragma unroll
        for (int w = 0; w < CH; ++w) {
          const int c = c0 + w * slices;
          t[w] = make_float2(-INFINITY, 0.f);
          a[w] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c < n) {
            const int64_t at = slot_of(q, from + c * step) * NR + rr;
            t[w] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + at * 2));
            a[w] = __ldcg(reinterpret_cast<const float4 *>(p.part_acc + at * D + d));
          }
        }
        float mn = M;
#pragma unroll
        for (int w = 0; w < CH; ++w) mn = fmaxf(mn, t[w].x);
        const float mm = mn == -INFINITY ? 0.f : mn, al = exp2_or_zero(M, mm);
        M = mn;
        ls *= al;
        o = make_float4(o.x * al, o.y * al, o.z * al, o.w * al);
#pragma unroll
        for (int w = 0; w < CH; ++w) {
          const float f = exp2_or_zero(t[w].x, mm);
          ls = fmaf(f, t[w].y, ls);
          add_scaled(o, f, a[w]);
        }
      }
#pragma unroll 1
      for (int k = 1; k < slices; k *= 2) {
        // (a sum of two is the same in either order: both lanes alike)
        const float Mo = __shfl_xor_sync(0xffffffffu, M, k), mn = fmaxf(M, Mo);
        const float f = exp2_or_zero(M, mn == -INFINITY ? 0.f : mn);
        M = mn;
        ls *= f;
        ls += __shfl_xor_sync(0xffffffffu, ls, k);
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
        o.x += __shfl_xor_sync(0xffffffffu, o.x, k);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, k);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, k);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, k);
      }
      if (slice != 0) continue;
      if (last) {
        store_four<BF16>(out_row(q, rr) + d, o, ls > 0.f ? sfu_rcp(ls) : 0.f);
      } else {
        __stcg(reinterpret_cast<float4 *>(p.part_acc + (slot_of(q, from) * NR + rr) * D + d), o);
        if (d == 0) ml_of[rr] = make_float2(M, ls);  // (others still read the part's)
      }
    }
  };
  if (n_cut > 0) __syncthreads();
#pragma unroll 1
  for (int c = 0; c < n_cut; ++c) {
    const int g = group_size(cut_piece[c]), parts = cut_piece[c].parts, group = cut_piece[c].part / g;
    const bool grouped = g < parts;
    int old = c == 0 ? cut_old0 : cut_old1;
#pragma unroll 1
    for (int level = grouped ? 0 : 1; level < 2; ++level) {
      const Piece &q = cut_piece[c];
      const int n = !grouped ? parts : level == 0 ? min(g, parts - group * g) : (parts + g - 1) / g;
      __syncthreads();
      if (tid == 0) {
        if (old < 0 || old >= n) atomicOr(p.status, PD_DEV_BAD_SCRATCH);  // not zero at the start
        flag[4] = old == n - 1;
        if (old == n - 1) atomicExch(level == 0 ? counter_of(q, group) : counter_of(q, -1), 0);
      }
      __syncthreads();
      if (!flag[4]) break;
      const int rows = min(p.rows_grp, q.r.ml * p.G - q.g * p.rows_grp);
      const int from = level == 0 ? group * g : 0, step = grouped && level == 1 ? g : 1;
      merge(q, rows, from, n, step, level == 1);
      if (level == 0) {
        __syncthreads();
        if (tid < rows)
          __stcg(reinterpret_cast<float2 *>(p.part_ml + (slot_of(q, from) * NR + tid) * 2), ml_of[tid]);
        __syncthreads();
        if (tid == 0) old = atomic_add_acq_rel_gpu(counter_of(q, -1), 1);
      }
    }
  }

  // rows of sequences without a visible key, and those at and past the last request's
  // end (padding of a captured batch): zeros
  auto zero_rows = [&](int t0, int t1, int first, int step) {
    const int per_row = p.Hq * (D / 8);
    const int64_t n = (int64_t)(t1 - t0) * per_row;
    for (int64_t i = first; i < n; i += step) {
      const int t = t0 + (int)(i / per_row), rem = (int)(i - (int64_t)(t - t0) * per_row);
      const int hq = rem / (D / 8), c = rem - hq * (D / 8);
      *reinterpret_cast<uint4 *>(obase + (int64_t)t * p.o_s0 + (int64_t)hq * p.o_s1 + c * 8) =
          make_uint4(0u, 0u, 0u, 0u);
    }
  };
#pragma unroll 1
  for (int i = blockIdx.x; i < S; i += G) {
    const QuantSeq r = seq_of(i);
    if (r.nb == 0) zero_rows(r.q0, r.q0 + r.ml, tid, NTHR);
  }
  if (p.query_start && blockIdx.y == gridDim.y - 1)
    zero_rows(starts[S], p.num_tokens, blockIdx.x * NTHR + tid, G * NTHR);
}

template <int D, int NT, bool BF16>
cudaError_t launch_quant_t(const QuantAttnParams &p, const Launch &l, cudaStream_t stream) {
  auto kern = pd_quant_decode<D, NT, BF16>;
  static SmemLimit limit;
  const cudaError_t e = allow_smem(limit, kern, l.smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = l.grid;
  cfg.blockDim = l.block;
  cfg.dynamicSmemBytes = l.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace pd
