// Decode attention over an 8-bit cache.
//
// One wave of CTAs divides the keys of all requests: the 16-key blocks of every
// (sequence, kv head, row group) unit, plus a unit cost for its epilogue, form one
// line, and every CTA takes the same length of it (as pd_window.cuh does).  A
// unit that the shares cut is merged by the CTA that publishes its last part.
//
// Within a CTA every warp works alone: it takes every so many steps of the CTA's
// blocks, copies them with cp.async into a ring of its own and computes on them,
// with no barrier before the unit's end.  Copies of 16 bytes a lane gather any
// layout; a TMA box of one block of one head is 2 KiB at D = 128, and such boxes
// stream at 5.0 TB/s where these rings read 7.0 (12 warps, 3 stages of 4 KiB each).
//
// The products run on 16-bit floats.  Every e4m3 code is a half: a register of four
// codes becomes two of two halves each.  Keys sit on the MMA's M side: S^T = K Q^T
// and O^T += V^T P^T.  The order of the summed dims is free, so that one
// register of a K row (four codes side by side) gives both halves of an A fragment's
// row, and the transposed load of two codes a lane gives the even and the odd
// dims of a V fragment.  bf16 queries are scaled by a power of two per row
// into the halves' range, which loses nothing above 2^-31 of the row's largest.
//
// The scales stay out of the products: S is scaled by its block's key scale in
// fp32; V's goes into the weights, a = s + log2(v_scale), p = 2^(a - max a), and
// out again in the sum l += p / v_scale, so P lies in [0, 2^15] whatever the scales
// are, and is rounded once, to 11 bits.
#pragma once

#include <cuda_fp16.h>

#include "pd_kernel.cuh"
#include "pd_quant.h"

namespace pd {

// What a unit counts in the line beside its blocks.
constexpr int kQuantUnitCost = 12;
constexpr float kQuantTop = 15.f;  // log2 of the largest P

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

// Four e4m3 codes as halves: bytes 0, 1 and bytes 2, 3.
__device__ __forceinline__ void halves_of(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// 4 values rounded to 16 bits
template <bool BF16>
__device__ __forceinline__ void store_four(void *dst, const float4 &v, float inv) {
  using tag = std::integral_constant<bool, BF16>;
  *reinterpret_cast<uint2 *>(dst) =
      make_uint2(pack2(v.x * inv, v.y * inv, tag{}), pack2(v.z * inv, v.w * inv, tag{}));
}

// The keys of a sequence that its rows see, in 16-key blocks.
struct QuantSeq {
  int L, q0, ml;               // keys, first q / out row, query tokens
  int u_lo, u_hi, v_lo, v_hi;  // union / intersection of its rows' windows
  int sk_nb, sk_gap;           // blocks of the sinks, blocks left out after them
  int nb;                      // blocks with visible keys
};

__device__ __forceinline__ QuantSeq quant_seq(int L, int q0, int ml, int window, int sinks) {
  QuantSeq r;
  r.L = L;
  r.q0 = q0;
  r.ml = ml;
  const int n0 = ml > 0 ? max(L - ml + 1, 0) : 0, n1 = ml > 0 ? L : 0;
  r.u_hi = n1;
  r.v_hi = n0;
  r.u_lo = window > 0 ? max(0, n0 - window) : 0;
  r.v_lo = window > 0 ? max(0, n1 - window) : 0;
  const int first = r.u_lo / kBlockKeys, last = (n1 + kBlockKeys - 1) / kBlockKeys;
  r.sk_nb = window > 0 ? (min(sinks, n1) + kBlockKeys - 1) / kBlockKeys : 0;
  r.sk_gap = max(0, first - r.sk_nb);
  r.nb = n1 > r.u_lo ? last - r.sk_gap : 0;
  return r;
}

template <int D, int NT, bool BF16>
__global__ void __launch_bounds__(32 * quant_max_warps(D, NT), 1)
    pd_quant_decode(const __grid_constant__ QuantAttnParams p) {
  constexpr int TB = quant_step_blocks(D, NT), NS = quant_stages(D, NT);
  constexpr int BLOCK = 16 * D;               // bytes of K (or V) of a block
  constexpr int STAGE = quant_stage_bytes(D, NT);  // TB x (K, V, scales)
  constexpr int CPR = D / 16;                 // 16-byte chunks of a row
  constexpr int RPI = 32 / CPR;               // rows that 32 lanes copy at once (D = 512: 1)
  constexpr int COPIES = D / 32;              // copies of a lane for K (or V) of a block
  constexpr int NR = 8 * NT;                  // rows of the CTA, padded
  constexpr int PASSES = quant_passes(D, NT), DC = D / PASSES, CPP = CPR / PASSES;
  constexpr int SPC = 32 / TB;                // steps whose page ids a warp holds

  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nthr = blockDim.x, NW = nthr >> 5;
  unsigned char *ring = smem + warp * (NS * STAGE);
  float *cp = reinterpret_cast<float *>(smem + NW * NS * STAGE);  // [NW][NR][DC] (swizzled)
  float2 *ml_of = reinterpret_cast<float2 *>(cp + NW * NR * DC);  // [NW][NR] (m, l)
  uint2 *qfrag = reinterpret_cast<uint2 *>(ml_of + NW * NR);      // [2][CPR][NT][32]
  float *rowsc = reinterpret_cast<float *>(qfrag + 2 * CPR * NT * 32);  // [2][NR]
  int *rowhi = reinterpret_cast<int *>(rowsc + 2 * NR);                 // [2][NR]
  int *sums = rowhi + 2 * NR;                                           // [32]
  volatile int *flag = sums + 32;                                       // [32]
  int *lens = sums + 64;                                                // [seqs]
  int *starts = lens + p.seqs_y;                                        // [seqs + 1]
  int *place = starts + p.seqs_y + 1;                                   // [seqs + 1]

  const int s_first = blockIdx.y * p.seqs_y, S = min(p.seqs_y, p.num_seqs - s_first);
  const int HR = p.Hkv * p.rg;  // units of a sequence

  grid_dependency_wait();

  // ---- the lengths, clamped and reported ------------------------------------
  {
    const int cap = p.bt_width * p.P;
    unsigned int bad = 0;
    for (int i = tid; i < S; i += nthr) {
      const int L = __ldg(p.seq_lens + s_first + i);
      if (L > cap) bad |= PD_DEV_BAD_SEQLEN;
      lens[i] = min(max(L, 0), cap);
    }
    if (p.query_start) {
      for (int i = tid; i <= S; i += nthr) {
        const int s = s_first + i;
        const int a = __ldg(p.query_start + s);
        const int b = s < p.num_seqs ? __ldg(p.query_start + s + 1) : a;
        starts[i] = min(max(a, 0), p.num_tokens);
        if (a < 0 || a > p.num_tokens || b < a || (s < p.num_seqs && b - a > p.M)) bad |= PD_DEV_BAD_QSTART;
      }
    }
    if (bad && blockIdx.x == 0) atomicOr(p.status, bad);
  }
  __syncthreads();
  auto seq_of = [&](int i) -> QuantSeq {
    int q0 = (s_first + i) * p.M, ml = p.M;
    if (p.query_start) {
      q0 = starts[i];
      ml = min(max(starts[i + 1] - q0, 0), p.M);
    }
    return quant_seq(lens[i], q0, ml, p.window, p.sinks);
  };

  // ---- this CTA's share: units [unit0, unit0 + n_pieces) of the line --------
  int unit0 = 0, n_pieces = 0;
  uint32_t x0 = 0, x1 = 0, share = 1;
  if (p.whole) {
    const int64_t U = (int64_t)S * HR;
    unit0 = (int)(U * blockIdx.x / gridDim.x);
    n_pieces = (int)(U * (blockIdx.x + 1) / gridDim.x) - unit0;
  } else {
    // places of the sequences: an exclusive sum over threads of runs of them
    const int per = (S + nthr - 1) / nthr, i0 = min(tid * per, S), i1 = min(i0 + per, S);
    int sum = 0;
    for (int i = i0; i < i1; ++i) sum += (seq_of(i).nb + kQuantUnitCost) * HR;
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int base = 0, W = 0;
    for (int i = 0; i < NW; ++i) {
      const int v = sums[i];
      if (i < warp) base += v;
      W += v;
    }
    int at = base + inc - sum;
    for (int i = i0; i < i1; ++i) {
      place[i] = at;
      at += (seq_of(i).nb + kQuantUnitCost) * HR;
    }
    if (tid == 0) place[S] = W;
    __syncthreads();
    share = max((uint32_t)p.min_share, ((uint32_t)W + gridDim.x - 1) / gridDim.x);
    x0 = min((uint64_t)blockIdx.x * share, (uint64_t)W);
    x1 = min((uint64_t)x0 + share, (uint64_t)W);
    // the unit that a place of the line is in
    auto unit_at = [&](uint32_t x, bool first) -> int {
      int lo = 0, hi = S - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((uint32_t)place[mid] <= x) lo = mid; else hi = mid - 1;
      }
      const uint32_t off = x - (uint32_t)place[lo];
      const int nb = seq_of(lo).nb, cost = nb + kQuantUnitCost;
      const int k = (int)(off / (uint32_t)cost), in = (int)(off - (uint32_t)k * cost);
      // (a first unit whose blocks, or whose place if it has none, lie before the share)
      return lo * HR + k + (first && in > 0 && in >= nb ? 1 : 0);
    };
    if (x1 > x0) {
      unit0 = unit_at(x0, true);
      n_pieces = unit_at(x1 - 1, false) - unit0 + 1;
    }
  }

  // A piece of the share: some or all blocks of one unit.
  struct Piece {
    QuantSeq r;
    int i, h, g;          // sequence (of this line), kv head, row group
    int b0, b1;           // its blocks of the unit
    int part, parts, first_cta;
  };
  // A unit that goes on behind the share comes first, so that its part is out early.
  bool tail = false;
  auto piece_at = [&](int k) -> Piece {
    const int u = unit0 + (tail ? (k == 0 ? n_pieces - 1 : k - 1) : k);
    Piece q;
    q.i = u / HR;
    const int hr = u - q.i * HR;
    q.h = hr / p.rg;
    q.g = hr - q.h * p.rg;
    q.r = seq_of(q.i);
    q.b0 = 0;
    q.b1 = q.r.nb;
    q.part = 0;
    q.parts = 1;
    q.first_cta = blockIdx.x;
    if (!p.whole) {
      const uint32_t a = (uint32_t)place[q.i] + (uint32_t)hr * (q.r.nb + kQuantUnitCost);
      if (x0 > a) q.b0 = (int)(x0 - a);
      if (x1 < a + q.r.nb) q.b1 = (int)(x1 - a);
      if (q.b1 - q.b0 < q.r.nb) {
        q.first_cta = (int)(a / share);
        q.part = (int)blockIdx.x - q.first_cta;
        q.parts = (int)((a + q.r.nb - 1) / share) - q.first_cta + 1;
      }
    }
    return q;
  };
  if (!p.whole && n_pieces > 1) {
    const Piece q = piece_at(n_pieces - 1);
    tail = q.b1 < q.r.nb;
  }

  // ---- the copies: a cursor over the steps of this warp ----------------------
  // Step st of a piece is blocks b0 + st TB ..; a warp takes steps first, first +
  // NW, .., the first one moving on with the pieces so that odd ones are spread.
  struct Cursor {
    int k;                // piece
    int first, mine;      // of its steps
    int at, base;         // next step of mine, the first whose page ids are held
    int b0, b1, sk_nb, sk_gap;
    int s, h;
  };
  auto enter = [&](Cursor &c, int k) {
    c.k = k;
    c.at = c.base = 0;
    c.mine = 0;
    if (k >= n_pieces) return;
    const Piece q = piece_at(k);
    const int steps = (q.b1 - q.b0 + TB - 1) / TB;
    c.first = (warp + k) % NW;
    c.mine = c.first < steps ? (steps - 1 - c.first) / NW + 1 : 0;
    c.b0 = q.b0;
    c.b1 = q.b1;
    c.sk_nb = q.r.sk_nb;
    c.sk_gap = q.r.sk_gap;
    c.s = s_first + q.i;
    c.h = q.h;
  };
  const int bpp = p.P / kBlockKeys;  // blocks of a page
  const int lg_bpp = (bpp & (bpp - 1)) == 0 ? __ffs(bpp) - 1 : -1;
  // the page ids of the cursor's next SPC steps, one block a lane
  auto fetch_ids = [&](const Cursor &c) -> int {
    if (c.k >= n_pieces) return 0;
    const int b = c.b0 + (c.first + (c.base + lane / TB) * NW) * TB + lane % TB;
    if (c.base + lane / TB >= c.mine || b >= c.b1) return 0;
    const int sb = b >= c.sk_nb ? b + c.sk_gap : b;
    return __ldg(p.block_table + (int64_t)c.s * p.bt_stride + (lg_bpp >= 0 ? sb >> lg_bpp : sb / bpp));
  };
  // the next run of steps with page ids: of this piece, or of the next one
  // that has a step for this warp
  auto next_run = [&](Cursor &c) {
    c.base += SPC;
    c.at = c.base;
    while (c.k < n_pieces && c.base >= c.mine) enter(c, c.k + 1);
  };
  Cursor cur, ahead;
  enter(cur, 0);
  while (cur.k < n_pieces && cur.mine == 0) enter(cur, cur.k + 1);
  int ids = fetch_ids(cur);
  ahead = cur;
  next_run(ahead);
  int ids_ahead = fetch_ids(ahead);
  const int c_row = lane / CPR, c_ch = lane % CPR;  // (D = 512: row 0, chunk = lane)
  const int64_t k_off = c_row * p.k.tok + c_ch * 16, v_off = c_row * p.v.tok + c_ch * 16;
  auto place_of = [&](int row, int ch) -> uint32_t {
    return D >= 128 ? row * D + ((ch ^ (row & 7)) << 4) : row * D + ((ch ^ ((row >> 1) & 3)) << 4);
  };
  int in_slot = 0;  // the slot that the next step goes to
  const uint32_t ring_at = smem_u32(ring);
  auto issue = [&]() {
    if (cur.k < n_pieces) {
      const int blk = cur.b0 + (cur.first + cur.at * NW) * TB;
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        int page = __shfl_sync(0xffffffffu, ids, (cur.at - cur.base) * TB + b);
        if (blk + b < cur.b1) {
          const int sb = blk + b >= cur.sk_nb ? blk + b + cur.sk_gap : blk + b;
          const int sub = lg_bpp >= 0 ? sb & (bpp - 1) : sb % bpp;
          if ((unsigned)page >= (unsigned)p.num_pages) {
            if (lane == 0) atomicOr(p.status, PD_DEV_BAD_PAGE);  // report, read page 0
            page = 0;
          }
          const uint32_t dst = ring_at + in_slot * STAGE + b * (2 * BLOCK);
          const unsigned char *ksrc = p.k.codes + page * p.k.page + (int64_t)(sub * kBlockKeys) * p.k.tok +
                                      cur.h * p.k.head + k_off;
          const unsigned char *vsrc = p.v.codes + page * p.v.page + (int64_t)(sub * kBlockKeys) * p.v.tok +
                                      cur.h * p.v.head + v_off;
#pragma unroll
          for (int i = 0; i < COPIES; ++i)
            copy_async16(dst + place_of(c_row + i * RPI, c_ch), ksrc + (int64_t)(i * RPI) * p.k.tok);
#pragma unroll
          for (int i = 0; i < COPIES; ++i)
            copy_async16(dst + BLOCK + place_of(c_row + i * RPI, c_ch), vsrc + (int64_t)(i * RPI) * p.v.tok);
          if (lane < 2) {
            const QuantPool &t = lane ? p.v : p.k;
            copy_async4(ring_at + in_slot * STAGE + TB * (2 * BLOCK) + b * 8 + lane * 4,
                        t.scale + page * t.s_page + sub * t.s_blk + cur.h * t.s_head);
          }
        }
      }
      if (++in_slot == NS) in_slot = 0;
      if (++cur.at - cur.base == SPC || cur.at == cur.mine) {
        cur = ahead;
        ids = ids_ahead;
        if (ahead.k < n_pieces) next_run(ahead);
        ids_ahead = fetch_ids(ahead);
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) issue();

  // ---- Q of a piece: halves in fragment order, row scales, row ends ----------
  using T = std::conditional_t<BF16, __nv_bfloat16, __half>;
  const T *qbase = static_cast<const T *>(p.q);
  T *obase = static_cast<T *>(p.out);
  constexpr int QV = D >= 128 ? D / 128 : 1;
  const int lg_g = (p.G & (p.G - 1)) == 0 ? __ffs(p.G) - 1 : -1;
  auto token_of = [&](int r) { return lg_g >= 0 ? r >> lg_g : r / p.G; };  // packed row -> token
  auto row_live = [&](const Piece &q, int rr) {
    return rr < p.rows_grp && q.g * p.rows_grp + rr < q.r.ml * p.G;
  };
  auto load_q = [&](const Piece &q, int buf) {
    for (int rr = warp; rr < NR; rr += NW) {
      const bool live = row_live(q, rr);
      const int pr = q.g * p.rows_grp + rr;
      const int t = live ? token_of(pr) : 0, jq = live ? pr - t * p.G : 0;
      const uint2 *src = reinterpret_cast<const uint2 *>(
          qbase + (int64_t)(q.r.q0 + t) * p.q_s0 + (int64_t)(q.h * p.G + jq) * p.q_s1);
      uint2 w[QV];
#pragma unroll
      for (int v = 0; v < QV; ++v)
        w[v] = live && (D >= 128 || lane < D / 4) ? __ldg(src + v * 32 + lane) : make_uint2(0u, 0u);
      float f = 1.f;
      if constexpr (BF16) {
        // the row's largest magnitude to [2^14, 2^15)
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < QV; ++v)
          top = max(max(max(w[v].x & 0x7fffu, (w[v].x >> 16) & 0x7fffu),
                        max(w[v].y & 0x7fffu, (w[v].y >> 16) & 0x7fffu)), top);
        top = __reduce_max_sync(0xffffffffu, top);
        // 2^(14 - e), e the exponent of the largest, within fp32's range
        const int e = min(max((int)(top >> 7) - 127, -100), 127);
        const float up = __int_as_float((14 - e + 127) << 23);
        f = __int_as_float((e - 14 + 127) << 23);
#pragma unroll
        for (int v = 0; v < QV; ++v) {
          auto half2_of = [&](uint32_t b) -> uint32_t {
            const float lo = __uint_as_float(b << 16) * up, hi = __uint_as_float(b & 0xffff0000u) * up;
            return pack2(lo, hi, std::integral_constant<bool, false>{});
          };
          w[v] = make_uint2(half2_of(w[v].x), half2_of(w[v].y));
        }
      }
#pragma unroll
      for (int v = 0; v < QV; ++v) {
        const int d4 = v * 32 + lane;  // dims 4 d4 ..
        if (D >= 128 || lane < D / 4)
          qfrag[((buf * CPR + (d4 >> 2)) * NT + (rr >> 3)) * 32 + (rr & 7) * 4 + (d4 & 3)] = w[v];
      }
      if (lane == 0) {
        rowsc[buf * NR + rr] = f * p.scale_log2;
        rowhi[buf * NR + rr] = live ? max(q.r.L - q.r.ml + t + 1, 0) : 0;
      }
    }
  };

  const int g8 = lane >> 2, t4 = lane & 3;
  const int a_row = lane & 15, a_hi = lane >> 4;  // the rows and chunk of ldmatrix's addresses
  auto sees = [&](int key, int lo, int hi) { return key < hi && (key >= lo || key < p.sinks); };
  int out_slot = 0;   // the slot of the next step to compute on
  int n_cut = 0;      // cut units of this share whose part is out
  int cut_k[2], cut_old[2];
  cut_k[0] = cut_k[1] = 0;
  cut_old[0] = cut_old[1] = 0;

  // the rows of a unit in q and out, and the scratch slot of a part of it
  auto out_row = [&](const Piece &q, int rr) -> T * {
    const int pr = q.g * p.rows_grp + rr, t = token_of(pr), jq = pr - t * p.G;
    return obase + (int64_t)(q.r.q0 + t) * p.o_s0 + (int64_t)(q.h * p.G + jq) * p.o_s1;
  };
  auto slot_of = [&](const Piece &q, int part) -> int64_t {
    const int64_t c = (int64_t)blockIdx.y * gridDim.x + q.first_cta + part;
    return part == 0 ? 2 * c + 1 : 2 * c;
  };

  if (n_pieces > 0) load_q(piece_at(0), 0);
  __syncthreads();

  for (int k = 0; k < n_pieces; ++k) {
    const Piece q = piece_at(k);
    const int buf = k & 1;
    const uint2 *qf = qfrag + buf * CPR * NT * 32 + lane;
    const int steps = (q.b1 - q.b0 + TB - 1) / TB;
    const int first = (warp + k) % NW;
    const int mine = first < steps ? (steps - 1 - first) / NW + 1 : 0;
    float acc[CPR][NT][4];
#pragma unroll
    for (int c = 0; c < CPR; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[c][n][0] = acc[c][n][1] = acc[c][n][2] = acc[c][n][3] = 0.f;
    // rows 8 n + 2 t4, + 1 of this thread
    float m[NT][2], l[NT][2], rs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float2 r = *reinterpret_cast<const float2 *>(rowsc + buf * NR + 8 * n + 2 * t4);
      rs[n][0] = r.x;
      rs[n][1] = r.y;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }
#pragma unroll 1
    for (int st = 0; st < mine; ++st) {
      copy_wait<NS - 2>();
      __syncwarp();
      issue();
      const uint32_t stage = ring_at + out_slot * STAGE;
      const float2 *scales = reinterpret_cast<const float2 *>(ring + out_slot * STAGE + TB * (2 * BLOCK));
      if (++out_slot == NS) out_slot = 0;
      const int blk = q.b0 + (first + st * NW) * TB;
      const int nbt = min(TB, q.b1 - blk);

      // S^T = K Q^T
      float sc[TB][NT][4];
#pragma unroll
      for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[b][n][0] = sc[b][n][1] = sc[b][n][2] = sc[b][n][3] = 0.f;
#pragma unroll
      for (int c = 0; c < CPR; c += 2) {
        uint2 qa[NT], qb[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          qa[n] = qf[(c * NT + n) * 32];
          qb[n] = qf[((c + 1) * NT + n) * 32];
        }
#pragma unroll
        for (int b = 0; b < TB; ++b) {
          if (b < nbt) {
            // (rows 0-7, 8-15) of chunk c, then of chunk c + 1
            uint32_t w[4];
            ldsm_x4(stage + b * (2 * BLOCK) + place_of(a_row, c + a_hi), w);
            uint32_t x[4], y[4];
            halves_of(w[0], x[0], x[2]);
            halves_of(w[1], x[1], x[3]);
            halves_of(w[2], y[0], y[2]);
            halves_of(w[3], y[1], y[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_16816<false>(sc[b][n], x, qa[n].x, qa[n].y);
              mma_16816<false>(sc[b][n], y, qb[n].x, qb[n].y);
            }
          }
        }
      }

      // scale, mask, running maximum of a = s + log2(v_scale)
      float mx[NT][2], inv[TB];
#pragma unroll
      for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = -INFINITY;
      int key0[TB];
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        const int i = blk + b;
        key0[b] = (i >= q.r.sk_nb ? i + q.r.sk_gap : i) * kBlockKeys;
        inv[b] = 0.f;
        if (b >= nbt) {
#pragma unroll
          for (int n = 0; n < NT; ++n) sc[b][n][0] = sc[b][n][1] = sc[b][n][2] = sc[b][n][3] = -INFINITY;
          continue;
        }
        const float2 kv = scales[b];
        const float lg = __log2f(kv.y);
        inv[b] = sfu_rcp(kv.y);
        // (does every row see all 16 keys)
        const bool all = key0[b] + kBlockKeys <= q.r.v_hi &&
                         (key0[b] >= q.r.v_lo || key0[b] + kBlockKeys <= p.sinks);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float f0 = rs[n][0] * kv.x, f1 = rs[n][1] * kv.x;
          sc[b][n][0] = fmaf(sc[b][n][0], f0, lg);
          sc[b][n][1] = fmaf(sc[b][n][1], f1, lg);
          sc[b][n][2] = fmaf(sc[b][n][2], f0, lg);
          sc[b][n][3] = fmaf(sc[b][n][3], f1, lg);
          if (!all) {
            const int2 hi = *reinterpret_cast<const int2 *>(rowhi + buf * NR + 8 * n + 2 * t4);
            const int lo0 = p.window > 0 ? max(0, hi.x - p.window) : 0;
            const int lo1 = p.window > 0 ? max(0, hi.y - p.window) : 0;
            const int ka = key0[b] + g8, kb = ka + 8;
            if (!sees(ka, lo0, hi.x)) sc[b][n][0] = -INFINITY;
            if (!sees(ka, lo1, hi.y)) sc[b][n][1] = -INFINITY;
            if (!sees(kb, lo0, hi.x)) sc[b][n][2] = -INFINITY;
            if (!sees(kb, lo1, hi.y)) sc[b][n][3] = -INFINITY;
          }
          mx[n][0] = fmaxf(mx[n][0], fmaxf(sc[b][n][0], sc[b][n][2]));
          mx[n][1] = fmaxf(mx[n][1], fmaxf(sc[b][n][1], sc[b][n][3]));
        }
      }
      bool grew = false;
      float mu[NT][2], al[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx[n][e] = fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], o));
          const float mn = fmaxf(m[n][e], mx[n][e]);
          mu[n][e] = (mn == -INFINITY ? 0.f : mn) - kQuantTop;
          al[n][e] = sfu_exp2(m[n][e] - (mn == -INFINITY ? 0.f : mn));  // m = -inf -> 0
          grew |= al[n][e] != 1.f;
          m[n][e] = mn;
          l[n][e] *= al[n][e];
        }
      if (__any_sync(0xffffffffu, grew)) {
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

      // P, then O^T += V^T P^T
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        if (b >= nbt) continue;
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float p0 = sfu_exp2(sc[b][n][0] - mu[n][0]), p1 = sfu_exp2(sc[b][n][1] - mu[n][1]);
          const float p2 = sfu_exp2(sc[b][n][2] - mu[n][0]), p3 = sfu_exp2(sc[b][n][3] - mu[n][1]);
          l[n][0] = fmaf(p0 + p2, inv[b], l[n][0]);
          l[n][1] = fmaf(p1 + p3, inv[b], l[n][1]);
          pb[n][0] = movmatrix_trans(pack2(p0, p1, std::integral_constant<bool, false>{}));
          pb[n][1] = movmatrix_trans(pack2(p2, p3, std::integral_constant<bool, false>{}));
        }
        // zero V of keys that no row sees (stale or NaN slots)
        const bool vmask = !(key0[b] >= q.r.u_lo && key0[b] + kBlockKeys <= q.r.u_hi);
        uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
        if (vmask) {
          const int ke = key0[b] + 2 * t4;
          mlo = (sees(ke, q.r.u_lo, q.r.u_hi) ? 0x0000ffffu : 0u) |
                (sees(ke + 1, q.r.u_lo, q.r.u_hi) ? 0xffff0000u : 0u);
          mhi = (sees(ke + 8, q.r.u_lo, q.r.u_hi) ? 0x0000ffffu : 0u) |
                (sees(ke + 9, q.r.u_lo, q.r.u_hi) ? 0xffff0000u : 0u);
        }
        const uint32_t vb = stage + b * (2 * BLOCK) + BLOCK;
#pragma unroll
        for (int c = 0; c < CPR; c += 2) {
          // (keys 0-7, 8-15) of chunk c, then of chunk c + 1: two keys' codes of
          // dims 2 g8, 2 g8 + 1 a register
          uint32_t w[4];
          ldsm_x4_trans(vb + place_of(a_row, c + a_hi), w);
          uint32_t x[4], y[4];
          halves_of(__byte_perm(w[0], 0u, 0x3120), x[0], x[1]);
          halves_of(__byte_perm(w[1], 0u, 0x3120), x[2], x[3]);
          halves_of(__byte_perm(w[2], 0u, 0x3120), y[0], y[1]);
          halves_of(__byte_perm(w[3], 0u, 0x3120), y[2], y[3]);
          if (vmask) {
            x[0] &= mlo; x[1] &= mlo; x[2] &= mhi; x[3] &= mhi;
            y[0] &= mlo; y[1] &= mlo; y[2] &= mhi; y[3] &= mhi;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_16816<false>(acc[c][n], x, pb[n][0], pb[n][1]);
            mma_16816<false>(acc[c + 1][n], y, pb[n][0], pb[n][1]);
          }
        }
      }
    }

    // ---- the piece's end: the warps' sums added, rows stored or published ----
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
      }
      if (lane < 4) {
        ml_of[warp * NR + 8 * n + 2 * lane] = make_float2(m[n][0], l[n][0]);
        ml_of[warp * NR + 8 * n + 2 * lane + 1] = make_float2(m[n][1], l[n][1]);
      }
    }
    const bool cut = q.parts > 1;
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
      // column d of row r at d ^ 8 (r / 2 % 4): a warp's stores hit every bank once
      float *mine_at = cp + warp * (NR * DC);
#pragma unroll
      for (int c = 0; c < CPP; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int r0 = 8 * n + 2 * t4, d = (16 * c + 2 * g8) ^ (t4 << 3);
          const float(&a)[4] = acc[ps * CPP + c][n];
          *reinterpret_cast<float2 *>(mine_at + r0 * DC + d) = make_float2(a[0], a[2]);
          *reinterpret_cast<float2 *>(mine_at + (r0 + 1) * DC + d) = make_float2(a[1], a[3]);
        }
      __syncthreads();
      if (ps == 0 && k + 1 < n_pieces) load_q(piece_at(k + 1), buf ^ 1);
      for (int it = tid; it < NR * (DC / 4); it += nthr) {
        const int rr = it / (DC / 4), d4 = it - rr * (DC / 4);
        if (!row_live(q, rr)) continue;
        float M = -INFINITY;
        for (int w = 0; w < NW; ++w) M = fmaxf(M, ml_of[w * NR + rr].x);
        const float mm = M == -INFINITY ? 0.f : M;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float ls = 0.f;
        for (int w = 0; w < NW; ++w) {
          const float2 t = ml_of[w * NR + rr];
          const float f = exp2_or_zero(t.x, mm);
          const float4 a = *reinterpret_cast<const float4 *>(cp + (w * NR + rr) * DC +
                                                              ((4 * d4) ^ (((rr >> 1) & 3) << 3)));
          ls = fmaf(f, t.y, ls);
          o.x = fmaf(f, a.x, o.x);
          o.y = fmaf(f, a.y, o.y);
          o.z = fmaf(f, a.z, o.z);
          o.w = fmaf(f, a.w, o.w);
        }
        const int d = ps * DC + 4 * d4;
        if (!cut) {
          store_four<BF16>(out_row(q, rr) + d, o, ls > 0.f ? 1.f / ls : 0.f);
        } else {
          const int64_t at = slot_of(q, q.part) * NR + rr;
          __stcg(reinterpret_cast<float4 *>(p.part_acc + at * D + d), o);
          if (d == 0) __stcg(reinterpret_cast<float2 *>(p.part_ml + at * 2), make_float2(M, ls));
        }
      }
      __syncthreads();
    }
    if (cut) {
      // every thread's stores, the barrier above, one release by one thread; the
      // count's answer is looked at when the share is done
      if (tid == 0) {
        const int u = ((s_first + q.i) * p.Hkv + q.h) * p.rg + q.g;
        const int old = atomic_add_acq_rel_gpu(p.counters + u, 1);
        if (n_cut == 0) cut_old[0] = old; else cut_old[1] = old;
      }
      if (n_cut == 0) cut_k[0] = k; else cut_k[1] = k;
      ++n_cut;
    }
  }
  grid_dependents_launch();

  // ---- cut units whose last part is this CTA's: merged ------------------------
  for (int c = 0; c < n_cut; ++c) {
    const Piece q = piece_at(c == 0 ? cut_k[0] : cut_k[1]);
    if (tid == 0) {
      const int old = c == 0 ? cut_old[0] : cut_old[1];
      if (old < 0 || old >= q.parts) atomicOr(p.status, PD_DEV_BAD_SCRATCH);  // not zero at the start
      flag[c] = old == q.parts - 1;
      if (old == q.parts - 1) {
        const int u = ((s_first + q.i) * p.Hkv + q.h) * p.rg + q.g;
        atomicExch(p.counters + u, 0);
      }
    }
    __syncthreads();
    if (!flag[c]) continue;
    constexpr int CH = 8;  // parts whose loads are in flight
    for (int it = tid; it < NR * (D / 4); it += nthr) {
      const int rr = it / (D / 4), d = 4 * (it - rr * (D / 4));
      if (!row_live(q, rr)) continue;
      float M = -INFINITY, ls = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c0 = 0; c0 < q.parts; c0 += CH) {
        float2 t[CH];
        float4 a[CH];
#pragma unroll
        for (int w = 0; w < CH; ++w) {
          const int64_t at = slot_of(q, min(c0 + w, q.parts - 1)) * NR + rr;
          t[w] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + at * 2));
          a[w] = __ldcg(reinterpret_cast<const float4 *>(p.part_acc + at * D + d));
          if (c0 + w >= q.parts) t[w] = make_float2(-INFINITY, 0.f);
        }
        float mn = M;
#pragma unroll
        for (int w = 0; w < CH; ++w) mn = fmaxf(mn, t[w].x);
        const float mm = mn == -INFINITY ? 0.f : mn;
        const float al = exp2_or_zero(M, mm);
        ls *= al;
        o.x *= al; o.y *= al; o.z *= al; o.w *= al;
        M = mn;
#pragma unroll
        for (int w = 0; w < CH; ++w) {
          const float f = exp2_or_zero(t[w].x, mm);
          ls = fmaf(f, t[w].y, ls);
          o.x = fmaf(f, a[w].x, o.x);
          o.y = fmaf(f, a[w].y, o.y);
          o.z = fmaf(f, a[w].z, o.z);
          o.w = fmaf(f, a[w].w, o.w);
        }
      }
      store_four<BF16>(out_row(q, rr) + d, o, ls > 0.f ? 1.f / ls : 0.f);
    }
  }

  if (p.query_start && blockIdx.y == gridDim.y - 1) {
    // rows at and past the last request's end (padding of a captured batch)
    // see no key: zeros
    const int t0 = starts[S], per_row = p.Hq * (D / 8);
    const int64_t n = (int64_t)(p.num_tokens - t0) * per_row;
    for (int64_t i = (int64_t)blockIdx.x * nthr + tid; i < n; i += (int64_t)gridDim.x * nthr) {
      const int t = t0 + (int)(i / per_row), rem = (int)(i - (int64_t)(t - t0) * per_row);
      const int hq = rem / (D / 8), c = rem - hq * (D / 8);
      *reinterpret_cast<uint4 *>(obase + (int64_t)t * p.o_s0 + (int64_t)hq * p.o_s1 + c * 8) =
          make_uint4(0u, 0u, 0u, 0u);
    }
  }
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
