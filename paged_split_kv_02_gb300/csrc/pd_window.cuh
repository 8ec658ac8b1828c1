// Batched decode over a window with sinks, every CTA an equal share.
//
// With a window, a (sequence, kv head) is a few hundred to a few thousand keys:
// a CTA each (pd_kernel.cuh) spends as long on its prologue (lengths, page
// ids, first copies) and epilogue as on its keys, and lengths that differ
// leave the last wave uneven.  Here one wave of CTAs divides all of them: the
// 16-key blocks of every (sequence, kv head) unit, plus a unit cost for its
// epilogue, form one line, and every CTA takes the same length of it, so a CTA
// has some whole units and at most one cut at each end.  Its producer warp
// streams from unit to unit without a pause while the consumers finish the
// last one; a unit that was cut is merged by the CTA that publishes its last
// part (each part in its CTA's own scratch slot, a counter per unit).
//
// The products are those of pd_kernel.cuh's mma.sync consumers: keys on the
// MMA's M side, S^T = K Q^T and O^T += V^T P^T, Q's fragments in registers (so
// head sizes up to 256), all sums in fp32.  P is rounded to the input type, the
// one rounding before the output's: the MMA takes 16-bit operands, and a pair of
// them (P and its remainder) would double the PV products.  It adds a tenth to
// the output's error, rms against 64 bits of the rms output: 64 sequences,
// window 1024, bf16 0.00182, of the output's rounding alone 0.00166.
//
// Memory-bound: K and V of the visible keys are read once.  Measured with
// CUDA events over graph replays (32 / 8 heads, D = 128, bf16, P = 16), in us,
// the bytes at the measured copy rate / this kernel / a CTA per unit and
// segment: 64 sequences, window 1024: 34 / 43 / 52; 32 of 1..4 tokens, window
// 4096: 55 / 66 / 79; 8, window 4096: 16 / 24 / 35; 128, window 128: 10 / 23 /
// 39.  What is left: about 4 us before the first keys arrive (lengths, page
// ids, the first copies), about 3 after the last (the sums, a part's count and
// the merge), and the pause of the warp groups between units.
#pragma once

#include "pd_kernel.cuh"

namespace pd {

// Everything of a sequence that a unit of it needs.
struct SeqRange {
  int L, q0, ml;               // keys, first q / out row, query tokens
  int rows;                    // packed rows, ml * G
  int u_lo, u_hi, v_lo, v_hi;  // union / intersection of its rows' windows
  int sk_nb, sk_gap;           // blocks of the sinks, blocks left out after them
  int nb;                      // 16-key blocks with visible keys
};

__device__ __forceinline__ SeqRange seq_range(int L, int q0, int ml, const Params &p) {
  SeqRange r;
  r.L = L;
  r.q0 = q0;
  r.ml = ml;
  r.rows = ml * p.G;
  const int n0 = ml > 0 ? max(L - ml + 1, 0) : 0, n1 = ml > 0 ? L : 0;
  r.u_hi = n1;
  r.v_hi = n0;
  r.u_lo = max(0, n0 - p.window);
  r.v_lo = max(0, n1 - p.window);
  const int first = r.u_lo / kBlockKeys, last = (n1 + kBlockKeys - 1) / kBlockKeys;
  r.sk_nb = (min(p.sinks, n1) + kBlockKeys - 1) / kBlockKeys;
  r.sk_gap = max(0, first - r.sk_nb);
  r.nb = n1 > r.u_lo ? last - r.sk_gap : 0;
  return r;
}

// Runs of 2 or 4 columns: of the sums in shared memory, of the output, of the
// published parts (L2 only).
__device__ __forceinline__ void load_run(float (&v)[4], const float *p) {
  const float4 w = *reinterpret_cast<const float4 *>(p);
  v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
}
__device__ __forceinline__ void load_run(float (&v)[2], const float *p) {
  const float2 w = *reinterpret_cast<const float2 *>(p);
  v[0] = w.x; v[1] = w.y;
}
__device__ __forceinline__ void fetch_run(float (&v)[4], const float *p) {
  const float4 w = __ldcg(reinterpret_cast<const float4 *>(p));
  v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
}
__device__ __forceinline__ void fetch_run(float (&v)[2], const float *p) {
  const float2 w = __ldcg(reinterpret_cast<const float2 *>(p));
  v[0] = w.x; v[1] = w.y;
}
__device__ __forceinline__ void publish_run(float *p, const float (&v)[4]) {
  __stcg(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
}
__device__ __forceinline__ void publish_run(float *p, const float (&v)[2]) {
  __stcg(reinterpret_cast<float2 *>(p), make_float2(v[0], v[1]));
}
template <bool BF16>
__device__ __forceinline__ void store_run(void *p, const float (&v)[4], float inv) {
  const float o[4] = {v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
  store4<BF16>(p, o);
}
template <bool BF16>
__device__ __forceinline__ void store_run(void *p, const float (&v)[2], float inv) {
  *reinterpret_cast<uint32_t *>(p) =
      pack2(v[0] * inv, v[1] * inv, std::integral_constant<bool, BF16>{});
}

// a / b for a quotient below 2^16 (an exact one: the approximate quotient is at
// most one off)
__device__ __forceinline__ int div_small(int a, int b) {
  int q = __float2int_rz(__fdividef((float)a, (float)b));
  const int r = a - q * b;
  if (r < 0) --q;
  if (r >= b) ++q;
  return q;
}

// A piece of a CTA's share: some or all blocks of one unit.
struct Piece {
  SeqRange r;
  int s, h;              // its unit
  int b0, b1;            // its blocks of the unit (none: a unit without visible keys)
  int part, parts;       // parts of the unit, one per CTA that has blocks of it
  int first_cta;         // the CTA of part 0
};

template <int D, bool BF16>
__global__ void __launch_bounds__(32 * (kWindowWarps + 1), 1)
    pd_window_decode(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ Params p) {
  static_assert(D <= 256, "Q's fragments stay in registers");
  using tag = std::integral_constant<bool, BF16>;
  using T = std::conditional_t<BF16, __nv_bfloat16, __half>;
  constexpr int BLOCK_BYTES = kBlockKeys * D * 2;
  constexpr int STAGE = kStageBytes;
  constexpr int TB = STAGE / 2 / BLOCK_BYTES;  // 16-key blocks per stage
  constexpr int KS = D / 16;                   // mma k-steps over d, and m-tiles of O^T

  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem =
      smem_raw + ((kSmemAlign - (smem_u32(smem_raw) & (kSmemAlign - 1))) & (kSmemAlign - 1));
  const int NS = p.NS, NT = p.NT, KG = p.KG, NC = NT * KG, NT8 = NT * 8;
  unsigned char *ring = smem;
  float *cp = reinterpret_cast<float *>(ring + NS * STAGE);  // [KG][NT8][D] (swizzled columns)
  float *mrow = cp + (size_t)KG * NT8 * D;                   // [KG][NT8]
  float *lrow = mrow + KG * NT8;
  uint64_t *full = reinterpret_cast<uint64_t *>(lrow + KG * NT8);
  uint64_t *empty = full + NS;
  int *sums = reinterpret_cast<int *>(empty + NS);  // per warp, of the line's length
  volatile int *flags = sums + kWindowWarps + 1;  // [0] abort
  volatile int *cut = flags + 4;                  // [2][8], the share's cut units: s, h, part, parts,
                                                  // first CTA, whether its part was the last
  int *pids = const_cast<int *>(cut) + 16;        // [kBlockIds]
  int *lens = pids + kBlockIds;                   // [S]
  int *starts = lens + p.num_seqs;           // [S + 1], with query_start

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = p.num_seqs, Hkv = p.Hkv;

  if (warp == 0) {
    if (lane < NS) {
      mbar_init(smem_u32(full + lane), 1);
      mbar_init(smem_u32(empty + lane), NT);
    }
    if (lane == 31) flags[0] = 0;
    fence_mbar_init();
  }
  if (warp == NC && lane == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  // (with p.early the lengths, the table and the older keys are read before
  // the previous grid on the stream has completed)
  if (!p.early) grid_dependency_wait();

  // ---- the lengths, clamped and reported, and the line's length -------------
  const int cap = p.bt_width * p.P;
  unsigned int bad = 0;
  for (int s = tid; s < S; s += blockDim.x) {
    const int L = __ldg(p.seq_lens + s);
    if (L > cap) bad |= PD_DEV_BAD_SEQLEN;
    lens[s] = min(max(L, 0), cap);
  }
  if (p.query_start) {
    for (int s = tid; s <= S; s += blockDim.x) {
      const int a = __ldg(p.query_start + s);
      const int b = s < S ? __ldg(p.query_start + s + 1) : a;
      starts[s] = min(max(a, 0), p.num_tokens);
      if (a < 0 || a > p.num_tokens || b < a || (s < S && b - a > p.M)) bad |= PD_DEV_BAD_QSTART;
    }
  }
  if (bad && blockIdx.x == 0) atomicOr(p.status, bad);
  __syncthreads();
  auto range_of = [&](int s) -> SeqRange {
    int q0 = s * p.M, ml = p.M;
    if (p.query_start) {
      q0 = starts[s];
      ml = min(max(starts[s + 1] - q0, 0), p.M);
    }
    return seq_range(lens[s], q0, ml, p);
  };
  // (the line's length fits an int: the planner sees to it)
  {
    int sum = 0;
    for (int s = tid; s < S; s += blockDim.x) sum += range_of(s).nb + kUnitCost;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sums[warp] = sum;
  }
  __syncthreads();
  int W = 0;
  for (int i = 0; i <= NC; ++i) W += sums[i];
  W *= Hkv;
  const int share = max(p.min_share, (W + (int)gridDim.x - 1) / (int)gridDim.x);
  if ((int64_t)blockIdx.x * share >= W) return;
  int x = blockIdx.x * share;
  const int x1 = min(W - x, share) + x;
  // the sequence of a place of the line, and where its units begin; of this
  // share's first place (s_cur, A) and of its last (s_end, A_end)
  int s_cur = 0, A = 0, s_end = 0, A_end = 0;
  for (int base = 0, sum = 0; base < S; base += 32) {
    const int s = base + lane;
    int c = s < S ? (range_of(s).nb + kUnitCost) * Hkv : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += y;
    }
    // sequences of these that end at or before the place
    const int n0 = __popc(__ballot_sync(0xffffffffu, s < S && sum + c <= x));
    const int n1 = __popc(__ballot_sync(0xffffffffu, s < S && sum + c <= x1 - 1));
    const int c0 = __shfl_sync(0xffffffffu, c, max(n0 - 1, 0));
    const int c1 = __shfl_sync(0xffffffffu, c, max(n1 - 1, 0));
    if (sum <= x) {
      s_cur = base + n0;
      A = n0 > 0 ? sum + c0 : sum;
    }
    s_end = base + n1;
    A_end = n1 > 0 ? sum + c1 : sum;
    if (n1 < 32) break;
    sum += __shfl_sync(0xffffffffu, c, 31);
  }
  SeqRange cur = range_of(s_cur);
  // blocks [b0, b1) of unit (s, h), which begins at place a of the line
  auto make_piece = [&](Piece &q, const SeqRange &r, int s, int h, int a) {
    q.r = r;
    q.s = s;
    q.h = h;
    q.b0 = max(min(x - a, r.nb), 0);
    q.b1 = min(x1 - a, r.nb);
    q.part = 0;
    q.parts = 1;
    q.first_cta = blockIdx.x;
    if (q.b1 > q.b0 && (q.b0 > 0 || q.b1 < r.nb)) {
      q.first_cta = div_small(a, share);
      q.part = (int)blockIdx.x - q.first_cta;
      q.parts = div_small(a + r.nb - 1, share) - q.first_cta + 1;
    }
  };
  // A unit cut at the end of the share comes first, then the rest in order: a
  // cut unit's parts are then published while whole units still stream, and
  // its merge does not wait for the end of every share.
  bool tail = false;
  int walk_end = x1;
  Piece tail_piece;
  {
    const SeqRange r = range_of(s_end);
    const int h = div_small(x1 - 1 - A_end, r.nb + kUnitCost);
    const int a = A_end + h * (r.nb + kUnitCost);
    if (a > x && x1 - a < r.nb) {
      make_piece(tail_piece, r, s_end, h, a);
      tail = true;
      walk_end = a;
    }
  }
  // the next piece of this CTA's share (every warp walks them alike); false
  // at its end
  int at = x;
  auto next_piece = [&](Piece &q) -> bool {
    if (tail) {
      tail = false;
      q = tail_piece;
      return true;
    }
    while (at < walk_end) {
      const int cost = cur.nb + kUnitCost;
      const int h = div_small(at - A, cost);
      const int a = A + h * cost;  // the unit: [a, a + cost), blocks first
      make_piece(q, cur, s_cur, h, a);
      const bool mine = cur.nb > 0 ? q.b1 > q.b0 : at == a;
      at = a + cost;
      if (at < walk_end && h == Hkv - 1) {
        A = at;
        cur = range_of(++s_cur);
      }
      if (mine) return true;
    }
    return false;
  };
  const int lg_g = (p.G & (p.G - 1)) == 0 ? __ffs(p.G) - 1 : -1;  // G a power of two
  auto token_of = [&](int rr) { return lg_g >= 0 ? rr >> lg_g : rr / p.G; };  // packed row -> token

  if (warp == NC) {
    // ================= producer: the page gather ===========================
    const uint64_t pol = policy_evict_first();
    const int bpp = p.P / kBlockKeys;  // 16-key blocks per page
    const int lg_bpp = (bpp & (bpp - 1)) == 0 ? __ffs(bpp) - 1 : -1;
    bool waited = !p.early, stop = false;
    int issued = 0, slot = 0, phase = 0;  // stages issued; ring slot and round parity of the next
    Piece q;
    while (!stop && next_piece(q)) {
      const int n = q.b1 - q.b0, ntile = (n + TB - 1) / TB;
      const int32_t *bt_row = p.block_table + (int64_t)q.s * p.bt_stride;
      // block i of the piece in its sequence
      auto seq_block = [&](int i) -> int {
        const int b = q.b0 + i;
        return b >= q.r.sk_nb ? b + q.r.sk_gap : b;
      };
      // (p.early: keys at and past `fresh` may come from the previous grid)
      const int fresh = max(q.r.L - p.M, 0);
      int pid_base = -kBlockIds;
      for (int j = 0; j < ntile; ++j) {
        if (j * TB >= pid_base + kBlockIds) {
          // physical pages of the next kBlockIds blocks
          pid_base = j * TB;
          __syncwarp();
          const int m = min(kBlockIds, n - pid_base);
#pragma unroll 4
          for (int i = lane; i < m; i += 32) {
            const int b = seq_block(pid_base + i);
            pids[i] = __ldg(bt_row + (lg_bpp >= 0 ? b >> lg_bpp : b / bpp));
          }
          __syncwarp();
        }
        const int nbt = min(TB, n - j * TB);
        if (!waited && (seq_block(j * TB + nbt - 1) + 1) * kBlockKeys > fresh) {
          grid_dependency_wait();
          waited = true;
        }
        if (issued >= NS) {
          int ok = 1;
          if (lane == 0) ok = mbar_wait_bounded(smem_u32(empty + slot), phase ^ 1);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) {
            if (lane == 0) {
              flags[0] = 1;
              atomicOr(p.status, PD_DEV_WAIT_TIMEOUT);
            }
            stop = true;
          }
        }
        if (stop || flags[0]) {
          stop = true;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(smem_u32(full + slot), nbt * 2 * BLOCK_BYTES);
        __syncwarp();
        if (lane < 2 * nbt) {
          // one copy per 16-key block of K or V
          const int kv = lane >= nbt, b = lane - kv * nbt;
          const int blk = seq_block(j * TB + b);
          const int key_in_page = (lg_bpp >= 0 ? blk & (bpp - 1) : blk % bpp) * kBlockKeys;
          int phys = pids[j * TB + b - pid_base];
          if ((unsigned)phys >= (unsigned)p.num_pool_blocks) {
            atomicOr(p.status, PD_DEV_BAD_PAGE);  // a page id outside the pool: report, read page 0
            phys = 0;
          }
          const uint32_t dst =
              smem_u32(ring + slot * STAGE + kv * (TB * BLOCK_BYTES) + b * BLOCK_BYTES);
          tma_load_5d(dst, kv ? &tmV : &tmK, smem_u32(full + slot), 0, key_in_page, 0, q.h, phys, pol);
        }
        ++issued;
        if (++slot == NS) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    // the next grid may launch as soon as the consumers say so too
    grid_dependents_launch();
    // leave no copy in flight: wait (bounded) for the last stages issued
    if (lane == 0) {
      for (int j = max(0, issued - NS); j < issued; ++j)
        if (!mbar_wait_bounded(smem_u32(full + j % NS), (j / NS) & 1))
          atomicOr(p.status, PD_DEV_WAIT_TIMEOUT);
    }
    return;
  }

  // ================= consumers ==============================================
  if (p.early) grid_dependency_wait();  // before q and any write
  const int nthr = NC * 32;
  auto consumers_sync = [&]() { asm volatile("bar.sync 1, %0;" ::"r"(nthr) : "memory"); };
  // Warp (t_n, g_k) owns the 8 packed rows of n-tile t_n and the stages in the
  // slots g_k, g_k + KG, ..: every phase of a slot's barriers is one group's.
  // (A parity tells two phases apart, no more: a group that skipped a phase of
  // a slot would take the one before it for the one it waits for.)
  const int t_n = warp % NT, g_k = warp / NT;
  const int r0 = t_n * 8 + 2 * (lane & 3), r1 = r0 + 1;
  const T *qbase = static_cast<const T *>(p.q);
  T *obase = static_cast<T *>(p.out);

  // Q's fragments of a unit, straight from its rows (the B operand: row lane /
  // 4 of the n-tile, dims 16 ks + 2 (lane % 4), + 1 and those + 8)
  uint32_t qf[KS][2];
  auto load_q = [&](const Piece &q) {
    const int rr = t_n * 8 + (lane >> 2);
    const bool live = rr < q.r.rows;
    const int i = live ? token_of(rr) : 0, jq = live ? rr - i * p.G : 0;
    const uint32_t *src = reinterpret_cast<const uint32_t *>(
        qbase + (int64_t)(q.r.q0 + i) * p.q_s0 + (int64_t)(q.h * p.G + jq) * p.q_s1 +
        2 * (lane & 3));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qf[ks][0] = live ? __ldg(src + 8 * ks) : 0u;
      qf[ks][1] = live ? __ldg(src + 8 * ks + 4) : 0u;
    }
  };

  const int k_row = lane & 15, k_hi = lane >> 4;                              // K ldmatrix roles
  const int v_row = (lane & 7) + ((lane >> 4) << 3), v_hi = (lane >> 3) & 1;  // V^T roles
  int slot = 0, phase = 0, turn = 0;  // slot of the next stage, its round's parity, slot % KG
  bool dead = false;        // a wait of this warp gave up: no more stages

  // the rows of a unit, and the scratch slot of a part of it: a CTA has at
  // most one unit that began before its share (slot 0) and one that goes on
  // behind it (slot 1)
  auto out_row = [&](const Piece &u, int rr) -> T * {
    const int i = token_of(rr), jq = rr - i * p.G;
    return obase + (int64_t)(u.r.q0 + i) * p.o_s0 + (int64_t)(u.h * p.G + jq) * p.o_s1;
  };
  auto slot_of = [&](const Piece &u, int part) -> int64_t {
    return part == 0 ? 2 * (int64_t)u.first_cta + 1 : 2 * (int64_t)(u.first_cta + part);
  };
  constexpr int kMaxGroups = kWindowGroups;
  constexpr int kW = D >= 128 ? 4 : 2, kV = D / (32 * kW);
  // a unit's parts from every CTA, normalised and stored
  auto merge_unit = [&](const Piece &u) {
    // rows and parts whose loads are in flight at once (fewer at D = 256, where
    // more registers here cost the main loop its own: 31 us against 23 for 48
    // sequences of 16 rows; bulk copies of the parts to shared memory are no
    // faster)
    constexpr int kRows = D == 256 ? 2 : 3, kChunk = D == 256 ? 2 : 4;
    for (int r0_ = warp; r0_ < u.r.rows; r0_ += kRows * NC) {
      float M[kRows], ls[kRows], a[kRows][kV][kW];
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        M[k] = -INFINITY;
        ls[k] = 0.f;
#pragma unroll
        for (int v = 0; v < kV; ++v)
#pragma unroll
          for (int e = 0; e < kW; ++e) a[k][v][e] = 0.f;
      }
      for (int c0 = 0; c0 < u.parts; c0 += kChunk) {
        float2 ml[kRows][kChunk];
        float b[kRows][kChunk][kV][kW];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
          for (int w = 0; w < kChunk; ++w) {
            const int rr = min(r0_ + k * NC, u.r.rows - 1);
            const bool there = c0 + w < u.parts;
            const int64_t place = slot_of(u, there ? c0 + w : 0) * NT8 + rr;
            ml[k][w] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + place * 2));
            if (!there) ml[k][w] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int v = 0; v < kV; ++v)
              fetch_run(b[k][w][v], p.part_acc + place * D + 32 * kW * v + kW * lane);
          }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          float cm = M[k];
#pragma unroll
          for (int w = 0; w < kChunk; ++w) cm = fmaxf(cm, ml[k][w].x);
          const float mu = cm == -INFINITY ? 0.f : cm;
          const float sc = exp2_or_zero(M[k], mu);
          ls[k] *= sc;
#pragma unroll
          for (int v = 0; v < kV; ++v)
#pragma unroll
            for (int e = 0; e < kW; ++e) a[k][v][e] *= sc;
#pragma unroll
          for (int w = 0; w < kChunk; ++w) {
            const float f = exp2_or_zero(ml[k][w].x, mu);  // (0 past the last part)
            ls[k] += f * ml[k][w].y;
#pragma unroll
            for (int v = 0; v < kV; ++v)
#pragma unroll
              for (int e = 0; e < kW; ++e) a[k][v][e] += f * b[k][w][v][e];
          }
          M[k] = cm;
        }
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int rr = r0_ + k * NC;
        if (rr < u.r.rows) {
          const float inv = ls[k] > 0.f ? sfu_rcp(ls[k]) : 0.f;
          T *dst = out_row(u, rr) + kW * lane;
#pragma unroll
          for (int v = 0; v < kV; ++v) store_run<BF16>(dst + 32 * kW * v, a[k][v], inv);
        }
      }
    }
  };
  // The cut units of this share (two at most) that are counted in but not
  // looked at yet: merged where this CTA's part was the last.
  int n_cut = 0, n_seen = 0;
  int count0 = 0, count1 = 0;  // thread 0: the units' counts before this CTA's parts
  auto merge_cut = [&]() {
    if (tid == 0) {
      for (int k = n_seen; k < n_cut; ++k) {
        const int old = k == 0 ? count0 : count1, parts = cut[8 * k + 3];
        const bool last = old == parts - 1;
        if (last) atomicExch(p.counters + 2 * ((int64_t)cut[8 * k] * Hkv + cut[8 * k + 1]), 0);
        if (old < 0 || old >= parts) atomicOr(p.status, PD_DEV_BAD_SCRATCH);  // not zero at the start
        cut[8 * k + 5] = last;
      }
    }
    consumers_sync();
    for (int k = n_seen; k < n_cut; ++k) {
      if (!cut[8 * k + 5]) continue;
      Piece u;
      u.s = cut[8 * k];
      u.h = cut[8 * k + 1];
      u.part = cut[8 * k + 2];
      u.parts = cut[8 * k + 3];
      u.first_cta = cut[8 * k + 4];
      u.b0 = u.b1 = 0;
      u.r = range_of(u.s);
      merge_unit(u);
    }
    n_seen = n_cut;
  };

  Piece q;
  bool have = next_piece(q);
  if (have) load_q(q);
  while (have) {
    const SeqRange &r = q.r;
    const int n = q.b1 - q.b0, ntile = (n + TB - 1) / TB;
    // visible keys of this thread's two rows (none for padding rows)
    int lo0 = 0, hi0 = 0, lo1 = 0, hi1 = 0;
    if (r0 < r.rows) {
      hi0 = max(r.L - r.ml + token_of(r0) + 1, 0);
      lo0 = max(0, hi0 - p.window);
    }
    if (r1 < r.rows) {
      hi1 = max(r.L - r.ml + token_of(r1) + 1, 0);
      lo1 = max(0, hi1 - p.window);
    }
    auto sees = [&](int k, int lo, int hi) -> bool { return k < hi && (k >= lo || k < p.sinks); };
    float acc[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int j = 0; j < ntile; ++j) {
      const int at_slot = slot, at_phase = phase;
      const bool mine = turn == g_k;
      if (++turn == KG) turn = 0;
      if (++slot == NS) {
        slot = turn = 0;
        phase ^= 1;
      }
      if (dead || !mine) continue;
      // one verdict for the warp, so no lane leaves the shuffles alone
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(full + at_slot), at_phase))) {
        if (lane == 0) {
          flags[0] = 1;
          atomicOr(p.status, PD_DEV_WAIT_TIMEOUT);
        }
        dead = true;
        continue;
      }
      const int nbt = min(TB, n - j * TB);
      const uint32_t kbase = smem_u32(ring + at_slot * STAGE);
      const uint32_t vbase = kbase + TB * BLOCK_BYTES;
      // first key of the stage's block b
      auto block_key = [&](int b) -> int {
        const int i = q.b0 + j * TB + b;
        return (i >= r.sk_nb ? i + r.sk_gap : i) * kBlockKeys;
      };

      // S^T = K Q^T for every block of the stage
      float sc[TB][4];
#pragma unroll
      for (int b = 0; b < TB; ++b) sc[b][0] = sc[b][1] = sc[b][2] = sc[b][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int chunk = 2 * ks + k_hi;
        const uint32_t off = (chunk >> 3) * 2048 + k_row * 128 + (((chunk & 7) ^ (k_row & 7)) << 4);
#pragma unroll
        for (int b = 0; b < TB; ++b) {
          if (b < nbt) {
            uint32_t a[4];
            ldsm_x4(kbase + b * BLOCK_BYTES + off, a);
            mma_16816<BF16>(sc[b], a, qf[ks][0], qf[ks][1]);
          }
        }
      }

      // scale, mask, running max
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        if (b >= nbt) {
          sc[b][0] = sc[b][1] = sc[b][2] = sc[b][3] = -INFINITY;
        } else {
          const int key0 = block_key(b);
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[b][e] *= p.scale_log2;
          // (does every row see all 16 keys)
          if (!(key0 + kBlockKeys <= r.v_hi && (key0 >= r.v_lo || key0 + kBlockKeys <= p.sinks))) {
            const int ka = key0 + (lane >> 2), kb = ka + 8;
            if (!sees(ka, lo0, hi0)) sc[b][0] = -INFINITY;
            if (!sees(ka, lo1, hi1)) sc[b][1] = -INFINITY;
            if (!sees(kb, lo0, hi0)) sc[b][2] = -INFINITY;
            if (!sees(kb, lo1, hi1)) sc[b][3] = -INFINITY;
          }
        }
        mx0 = fmaxf(mx0, fmaxf(sc[b][0], sc[b][2]));
        mx1 = fmaxf(mx1, fmaxf(sc[b][1], sc[b][3]));
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
      }
      const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
      const float mu0 = mn0 == -INFINITY ? 0.f : mn0;
      const float mu1 = mn1 == -INFINITY ? 0.f : mn1;
      const float al0 = sfu_exp2(m0 - mu0), al1 = sfu_exp2(m1 - mu1);  // m = -inf -> 0
      m0 = mn0;
      m1 = mn1;
      if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          acc[i][0] *= al0;
          acc[i][1] *= al1;
          acc[i][2] *= al0;
          acc[i][3] *= al1;
        }
      }
      l0 *= al0;
      l1 *= al1;

      // P = exp2(S - m); PV
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        if (b < nbt) {
          const float p0 = sfu_exp2(sc[b][0] - mu0), p1 = sfu_exp2(sc[b][1] - mu1);
          const float p2 = sfu_exp2(sc[b][2] - mu0), p3 = sfu_exp2(sc[b][3] - mu1);
          l0 += p0 + p2;
          l1 += p1 + p3;
          const uint32_t pb0 = movmatrix_trans(pack2(p0, p1, tag{}));
          const uint32_t pb1 = movmatrix_trans(pack2(p2, p3, tag{}));
          const int key0 = block_key(b);
          const bool vmask = !(key0 >= r.u_lo && key0 + kBlockKeys <= r.u_hi);
          uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
          if (vmask) {
            // zero V of keys that no row sees (stale or NaN slots)
            const int ke = key0 + 2 * (lane & 3);
            mlo = (sees(ke, r.u_lo, r.u_hi) ? 0x0000ffffu : 0u) |
                  (sees(ke + 1, r.u_lo, r.u_hi) ? 0xffff0000u : 0u);
            mhi = (sees(ke + 8, r.u_lo, r.u_hi) ? 0x0000ffffu : 0u) |
                  (sees(ke + 9, r.u_lo, r.u_hi) ? 0xffff0000u : 0u);
          }
          const uint32_t vb = vbase + b * BLOCK_BYTES;
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            const int chunk = 2 * mt + v_hi;
            uint32_t a[4];
            ldsm_x4_trans(vb + (chunk >> 3) * 2048 + v_row * 128 + (((chunk & 7) ^ (v_row & 7)) << 4),
                          a);
            if (vmask) {
              a[0] &= mlo;
              a[1] &= mlo;
              a[2] &= mhi;
              a[3] &= mhi;
            }
            mma_16816<BF16>(acc[mt], a, pb0, pb1);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(empty + at_slot));
    }
    // full row sums: the 8 lanes of one (lane & 3) class hold one row pair
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }

    // ---- the warp groups' sums to shared memory; the next unit's Q on its way
    {
      float *dst = cp + (size_t)g_k * NT8 * D;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        const int d = mt * 16 + (lane >> 2);
        dst[r0 * D + psw(d, r0)] = acc[mt][0];
        dst[r1 * D + psw(d, r1)] = acc[mt][1];
        dst[r0 * D + psw(d + 8, r0)] = acc[mt][2];
        dst[r1 * D + psw(d + 8, r1)] = acc[mt][3];
      }
      if (lane < 4) {
        mrow[g_k * NT8 + r0] = m0;
        mrow[g_k * NT8 + r1] = m1;
        lrow[g_k * NT8 + r0] = l0;
        lrow[g_k * NT8 + r1] = l1;
      }
    }
    const Piece done = q;
    have = next_piece(q);
    if (have)
      load_q(q);
    else
      grid_dependents_launch();  // (the next grid's CTAs wait until this one has completed)
    consumers_sync();

    // ---- rows of the piece: normalised and stored, or published as a part ---
    // a warp takes a row at a time, a lane kV runs of kW columns
    for (int rr = warp; rr < done.r.rows; rr += NC) {
      float mg[kMaxGroups], lg[kMaxGroups], b[kMaxGroups][kV][kW];
#pragma unroll
      for (int g = 0; g < kMaxGroups; ++g) {
        const int at_row = (g < KG ? g : 0) * NT8 + rr;
        mg[g] = g < KG ? mrow[at_row] : -INFINITY;
        lg[g] = g < KG ? lrow[at_row] : 0.f;
#pragma unroll
        for (int v = 0; v < kV; ++v)
          load_run(b[g][v], cp + (size_t)at_row * D + psw(32 * kW * v + kW * lane, rr));
      }
      float ms = mg[0];
#pragma unroll
      for (int g = 1; g < kMaxGroups; ++g) ms = fmaxf(ms, mg[g]);
      const float mu = ms == -INFINITY ? 0.f : ms;
      float a[kV][kW] = {}, ls = 0.f;
#pragma unroll
      for (int g = 0; g < kMaxGroups; ++g) {
        const float w = exp2_or_zero(mg[g], mu);
        ls += w * lg[g];
#pragma unroll
        for (int v = 0; v < kV; ++v)
#pragma unroll
          for (int e = 0; e < kW; ++e) a[v][e] += w * b[g][v][e];
      }
      if (done.parts == 1) {
        const float inv = ls > 0.f ? sfu_rcp(ls) : 0.f;
        T *dst = out_row(done, rr) + kW * lane;
#pragma unroll
        for (int v = 0; v < kV; ++v) store_run<BF16>(dst + 32 * kW * v, a[v], inv);
      } else {
        const int64_t mine = slot_of(done, done.part) * NT8 + rr;
        float *dst = p.part_acc + mine * D + kW * lane;
#pragma unroll
        for (int v = 0; v < kV; ++v) publish_run(dst + 32 * kW * v, a[v]);
        if (lane == 0) __stcg(reinterpret_cast<float2 *>(p.part_ml + mine * 2), make_float2(ms, ls));
      }
    }
    consumers_sync();  // the sums are free for the next piece
    if (done.parts > 1) {
      // every thread's stores, the barrier above, one release by one thread;
      // the last part's acquire then covers all of them.  The count's answer
      // is looked at after the next whole unit, or at the end.
      if (tid == 0) {
        cut[8 * n_cut] = done.s;
        cut[8 * n_cut + 1] = done.h;
        cut[8 * n_cut + 2] = done.part;
        cut[8 * n_cut + 3] = done.parts;
        cut[8 * n_cut + 4] = done.first_cta;
        const int old =
            atomic_add_acq_rel_gpu(p.counters + 2 * ((int64_t)done.s * Hkv + done.h), 1);
        if (n_cut == 0)
          count0 = old;
        else
          count1 = old;
      }
      ++n_cut;
    }
    if (n_cut > n_seen && (!have || done.parts == 1)) merge_cut();
  }

  if (p.query_start && blockIdx.x == 0) {
    // rows at and past the last request's end (padding of a captured batch)
    // see no key: zeros
    const int t0 = starts[S], per_row = p.Hq * (D / 8);
    for (int64_t i = tid; i < (int64_t)(p.num_tokens - t0) * per_row; i += nthr) {
      const int t = t0 + (int)(i / per_row), rem = (int)(i - (int64_t)(t - t0) * per_row);
      const int hq = rem / (D / 8), c = rem - hq * (D / 8);
      *reinterpret_cast<uint4 *>(obase + (int64_t)t * p.o_s0 + (int64_t)hq * p.o_s1 + c * 8) =
          make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

template <int D, bool BF16>
cudaError_t launch_window_t(const CUtensorMap &tk, const CUtensorMap &tv, const Params &p,
                            const Launch &l, cudaStream_t stream) {
  auto kern = pd_window_decode<D, BF16>;
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
  return cudaLaunchKernelEx(&cfg, kern, tk, tv, p);
}

}  // namespace pd
