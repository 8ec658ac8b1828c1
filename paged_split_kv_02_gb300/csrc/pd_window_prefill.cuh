// Prefill over a window with sinks at head sizes 64 to 256, tile after tile.
//
// The tiles, stages, products and softmax are those of pd_kernel.cuh's
// tensor-memory prefill (256 packed rows as two halves that share every K/V
// stage, at head size 256 one half of 128 rows; S, P and O in tensor memory).  A window makes a tile short: at 1024
// keys 17 stages of 64 keys, ~1.1 us each, beside ~11 us of starting the CTA,
// reading the work item and lengths, loading Q, filling the ring and storing
// O.  Here a CTA keeps its tensor memory and ring and runs through a list of
// tiles (one CTA per SM, item i of CTA b is the list's b + i G, every kv head
// of an item beside each other), so that most of that is under the tile before:
//   * the producer warp reads the next item and its lengths ahead, hands them
//     to the other warps through two slots in shared memory, and goes on
//     streaming K and V into the ring;
//   * the S warp, once the last S of a tile is done, brings the next tile's Q
//     with TMA copies (two boxes of 64 dims per half: 128 / G tokens of the
//     kv head's G q heads are the half's 128 packed rows in order) and starts
//     on its S while the softmax finishes the tile before;
//   * the softmax warps store O straight from tensor memory, a 4 x 4 exchange
//     of 16-byte pieces among lanes making 64-byte runs of a row.
// Barriers are counted through the tiles: stage g of the CTA uses S / P buffer
// g & 1, ring slot g % NS.
//
// A half's softmax has two warps on each scheduler and is bound by latency, so
// what a stage does not need is kept out of it: which stages need a mask, and
// which may hold V to zero, are ranges of stages worked out per tile (four
// blocks' tests per stage cost ~200 of ~1200 cycles); a masked stage takes the
// same exponentials as the others and clears P by the row's visible keys, and
// with sinks only a tile's first stage takes a max (a masked stage 1900 cycles,
// 3000 with its own max and tests); the row sums follow the hand-over of P.
//
// P is rounded to the input type, as the MMA's 16-bit operand (two operands, P
// and its remainder, would double the PV products), and the row sums take it as
// rounded, so that O is a mean by the weights used.  Error, rms against 64 bits
// of the rms output: window 1024 bf16 0.00185, of the output's rounding alone
// 0.00166; window 700 at head size 64 fp16 0.00024 and 0.00021.
//
// Measured (CUDA events over graph replays, bf16, P = 16; in brackets a CTA per
// tile, at head size 64 tiles of 64 rows on mma.sync): 4 requests of 2048 tokens
// after 2048, 32 / 8 heads of 128, window 1024, 4 sinks 142 us (206); 2 of 8192,
// window 4096, 64 sinks 678 us (800), 64 % of the tensor peak; 1276 ragged
// tokens, 16 / 4 heads of 64, window 700 17.7 us (30.6); 1024 tokens, 32 / 8
// heads of 256, window 1024 63 us (64 rows on mma.sync 239), 4096 of window 4096
// 695 (2912).  Not kept: a warp per
// half for its S and its PV MMAs (the same); S of 128 keys at once, one buffer
// per half (800 against 700, halves in turn 830); P handed over 32 keys at a
// time (153 us for 142); O stored without the exchange
// in 32-byte pieces or in 128-byte runs (2 - 3 % slower).
#pragma once

#include "pd_kernel.cuh"

namespace pd {

// the n lowest of 32 bits (none below 0, all from 32 on)
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : (1u << max(n, 0)) - 1u;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(wp_threads(D), 1)
    pd_window_prefill(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ Params p) {
  constexpr int KS = D / 16, TB = 4, SC = TB * kBlockKeys, NBOX = D / 64;
  constexpr int BLOCK_BYTES = kBlockKeys * D * 2, STAGE = wp_stage_bytes(D), BIDS = kTpBlockIds;
  constexpr int H = wp_halves(D), ROWS = H * kTpRows;  // halves of a tile, its rows
  constexpr int kHalf = kTpRows * D * 2;               // bytes of a half's Q
  constexpr int kCols = 512;  // tensor memory: S / P 2 H x 64 columns, O H x D
  static_assert(2 * TB * BLOCK_BYTES == STAGE, "K and V of 64 keys");
  static_assert(2 * H * SC + H * D <= kCols, "O beside S");
  using tag = std::integral_constant<bool, BF16>;
  using T = std::conditional_t<BF16, __nv_bfloat16, __half>;

  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem =
      smem_raw + ((kSmemAlign - (smem_u32(smem_raw) & (kSmemAlign - 1))) & (kSmemAlign - 1));
  const int NS = p.NS;
  unsigned char *ring = smem;
  unsigned char *qs = ring + NS * STAGE;
  uint64_t *full = reinterpret_cast<uint64_t *>(qs + H * kHalf);
  uint64_t *empty = full + NS;
  // [0..3] S full (2 x + b), [4..7] P written, [8..11] PV done, [12] every MMA
  // done, [13] Q landed, [14,15] item slot full, [16,17] item slot read
  uint64_t *bars = empty + NS;
  volatile int *flags = reinterpret_cast<volatile int *>(bars + kWpBarriers);  // [0] abort
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kWpBarriers) + 1;
  volatile int *items = flags + 4;                  // [2][8]: valid, s, h, first row, q0, ml, L
  int *pids = const_cast<int *>(items) + 16;        // [BIDS]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kSWarp = 4 * H, kLoadWarp = kSWarp + 1, kPvWarp = kSWarp + 2;
  constexpr int kReaders = 5 * H + 1;  // warps that read an item slot: all but the load warp
  if (warp == 0) {
    if (lane < NS) {
      mbar_init(smem_u32(full + lane), 1);
      mbar_init(smem_u32(empty + lane), H);  // the halves' PV commits
    }
    if (lane < kWpBarriers)
      mbar_init(smem_u32(bars + lane), lane >= 4 && lane <= 7 ? 4 : lane == 12 ? H + 1 : lane >= 16 ? kReaders : 1);
    if (lane == 31) flags[0] = 0;
    fence_mbar_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
    prefetch_tensormap(&tmQ);
  }
  if (warp == 0) tmem_alloc(smem_u32(tmem_slot), kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base =
      __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(tmem_slot), 0);
  const uint32_t tS = tmem_base, tO = tmem_base + 2 * H * SC;
  grid_dependency_wait();

  // A token's rows: its G q heads of a kv head, padded to a power of two with
  // the heads behind them (whose rows are not used), so that a half is a box of q
  const int lg_g = p.G > 1 ? 32 - __clz(p.G - 1) : 0;
  const int total = p.num_items * p.Hkv;
  auto give_up = [&]() {
    if (lane == 0) {
      flags[0] = 1;
      atomicOr(p.status, PD_DEV_WAIT_TIMEOUT);
    }
  };
  // a wait of the whole warp
  auto wait = [&](uint64_t *bar, int parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(bar), parity));
  };

  // A tile's keys: its rows' windows and the sinks as one run of nb blocks.
  struct Tile {
    int s, h, rr0, q0, ml, L;
    int rows;                    // padded rows of the request
    int u_lo, u_hi;              // union of the rows' windows
    int sk_nb, sk_gap, nb;
  };
  auto tile_of = [&](int s, int h, int rr0, int q0, int ml, int L) -> Tile {
    Tile t;
    t.s = s;
    t.h = h;
    t.rr0 = rr0;
    t.q0 = q0;
    t.ml = ml;
    t.L = L;
    t.rows = ml << lg_g;
    const int last = min(rr0 + ROWS, t.rows) - 1;
    t.u_lo = t.u_hi = 0;
    if (last >= rr0) {
      t.u_hi = row_keys(L, ml, last >> lg_g, p.window).hi;
      t.u_lo = row_keys(L, ml, rr0 >> lg_g, p.window).lo;
    }
    const int first = t.u_lo / kBlockKeys;
    t.sk_nb = (min(p.sinks, t.u_hi) + kBlockKeys - 1) / kBlockKeys;
    t.sk_gap = max(0, first - t.sk_nb);
    t.nb = t.u_hi > t.u_lo ? (t.u_hi + kBlockKeys - 1) / kBlockKeys - t.sk_gap : 0;
    return t;
  };
  // tile number n of this CTA, from its item slot; false at the list's end or
  // when a wait gave up
  auto take = [&](int n, Tile &t) -> bool {
    if (!wait(bars + 14 + (n & 1), (n >> 1) & 1)) {
      give_up();
      return false;
    }
    volatile int *it = items + 8 * (n & 1);
    const bool valid = it[0] != 0;
    t = tile_of(it[1], it[2], it[3], it[4], it[5], it[6]);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(bars + 16 + (n & 1)));
    return valid;
  };

  if (warp == kLoadWarp) {
    // ================= items, and K and V of their blocks ===================
    const uint64_t pol = policy_evict_first();
    const int bpp = p.P / kBlockKeys, lg_bpp = (bpp & (bpp - 1)) == 0 ? __ffs(bpp) - 1 : -1;
    const int cap = p.bt_width * p.P;
    int issued = 0, slot = 0, phase = 0;
    bool stop = false;
    // the item of list entry i: its words, then (dependent loads) its lengths
    auto words = [&](int i, int4 &w0, int4 &w1) {
      const int64_t at = 2 * (int64_t)(i / p.Hkv);
      w0 = __ldg(reinterpret_cast<const int4 *>(p.work) + at);
      w1 = __ldg(reinterpret_cast<const int4 *>(p.work) + at + 1);
    };
    auto good = [&](const int4 &w0) {
      // (this launch has no split tiles: one segment each)
      return w0.x >= 0 && w0.x < p.num_seqs && tile_in_range(w0.y, ROWS) &&
             w0.z == 0 && w0.w == 1;
    };
    auto lengths = [&](const int4 &w0, int &L, int &qa, int &qb) {
      const int s = good(w0) ? w0.x : 0;
      L = __ldg(p.seq_lens + s);
      qa = __ldg(p.query_start + s);
      qb = __ldg(p.query_start + s + 1);
    };
    int i = blockIdx.x, n = 0;
    int4 w0 = {}, w1 = {};
    int L = 0, qa = 0, qb = 0;
    if (i < total) {
      words(i, w0, w1);
      lengths(w0, L, qa, qb);
    }
    while (!stop) {
      // this entry into item slot n & 1, once tile n - 2 has been read from it
      const bool more = i < total;
      const bool ok = more && good(w0);
      if (more && !ok && lane == 0) atomicOr(p.status, PD_DEV_BAD_WORK);
      const int4 c0 = w0;
      const int cL = L, ca = qa, cb = qb, ch = i % p.Hkv;
      const int next = i + gridDim.x;
      if (more && next < total) words(next, w0, w1);  // on their way
      if (more && !ok) {
        if (next < total) lengths(w0, L, qa, qb);
        i = next;
        continue;
      }
      if (n >= 2 && !wait(bars + 16 + (n & 1), ((n >> 1) & 1) ^ 1)) {
        give_up();
        break;
      }
      const int a = min(max(ca, 0), p.num_tokens), b = min(max(cb, a), p.num_tokens);
      const int len = min(max(cL, 0), cap);
      if (lane == 0) {
        if (more && (a != ca || b != cb)) atomicOr(p.status, PD_DEV_BAD_QSTART);
        if (more && cL > cap) atomicOr(p.status, PD_DEV_BAD_SEQLEN);
        volatile int *it = items + 8 * (n & 1);
        it[0] = more;
        it[1] = c0.x;
        it[2] = ch;
        it[3] = c0.y * ROWS;
        it[4] = a;
        it[5] = b - a;
        it[6] = len;
        mbar_arrive(smem_u32(bars + 14 + (n & 1)));
      }
      __syncwarp();
      if (!more) break;
      ++n;
      const Tile t = tile_of(c0.x, ch, c0.y * ROWS, a, b - a, len);
      const int32_t *bt_row = p.block_table + (int64_t)t.s * p.bt_stride;
      auto seq_block = [&](int k) -> int { return k >= t.sk_nb ? k + t.sk_gap : k; };
      const int ntile = (t.nb + TB - 1) / TB;
      int pid_base = -BIDS;
      for (int j = 0; j < ntile; ++j) {
        if (j * TB >= pid_base + BIDS) {
          // physical pages of the next BIDS blocks
          pid_base = j * TB;
          __syncwarp();
          const int m = min(BIDS, t.nb - pid_base);
#pragma unroll 4
          for (int k = lane; k < m; k += 32) {
            const int blk = seq_block(pid_base + k);
            pids[k] = __ldg(bt_row + (lg_bpp >= 0 ? blk >> lg_bpp : blk / bpp));
          }
          __syncwarp();
        }
        if (issued >= NS && !wait(empty + slot, phase ^ 1)) {
          give_up();
          stop = true;
        }
        if (stop || flags[0]) {
          stop = true;
          break;
        }
        const int nbt = min(TB, t.nb - j * TB);
        if (lane == 0) mbar_arrive_expect_tx(smem_u32(full + slot), nbt * 2 * BLOCK_BYTES);
        __syncwarp();
        // K, one copy per (block, 64-dim box), box-major ([box][block][16
        // keys][128 B]) so that one box's keys are consecutive 128-byte rows;
        // V, one copy per block
        if (lane < nbt * (NBOX + 1)) {
          const bool k_copy = lane < nbt * NBOX;
          const int blk_i = k_copy ? lane / NBOX : lane - nbt * NBOX, box = k_copy ? lane % NBOX : 0;
          const int blk = seq_block(j * TB + blk_i);
          const int key_in_page = (lg_bpp >= 0 ? blk & (bpp - 1) : blk % bpp) * kBlockKeys;
          int phys = pids[j * TB + blk_i - pid_base];
          if ((unsigned)phys >= (unsigned)p.num_pool_blocks) {
            atomicOr(p.status, PD_DEV_BAD_PAGE);  // a page id outside the pool: report, read page 0
            phys = 0;
          }
          const uint32_t dst =
              smem_u32(ring + slot * STAGE) +
              (k_copy ? box * (TB * BLOCK_BYTES / NBOX) + blk_i * (BLOCK_BYTES / NBOX)
                      : TB * BLOCK_BYTES + blk_i * BLOCK_BYTES);
          tma_load_5d(dst, k_copy ? &tmK : &tmV, smem_u32(full + slot), 0, key_in_page, box, t.h, phys, pol);
        }
        ++issued;
        if (++slot == NS) {
          slot = 0;
          phase ^= 1;
        }
        if (j == 0 && next < total) lengths(w0, L, qa, qb);  // the next item's words are here
      }
      if (ntile == 0 && next < total) lengths(w0, L, qa, qb);
      i = next;
    }
    // leave no copy in flight: wait (bounded) for the last stages issued
    if (lane == 0) {
      for (int j = max(0, issued - NS); j < issued; ++j)
        if (!mbar_wait_bounded(smem_u32(full + j % NS), (j / NS) & 1))
          atomicOr(p.status, PD_DEV_WAIT_TIMEOUT);
    }
  } else if (warp == kSWarp) {
    // ================= Q, and the S MMAs of both halves =====================
    const uint32_t idS = umma_idesc_f16(kTpRows, SC, BF16, 0, 0);
    const uint32_t ring_u = smem_u32(ring), qb_u = smem_u32(qs);
    int g = 0, loads = 0;  // stages so far, tiles with keys so far
    bool ok = true;
    Tile t;
    for (int n = 0; ok && take(n, t); ++n) {
      const int ntile = (t.nb + TB - 1) / TB;
      if (ntile == 0) continue;
      // Q's buffer is free once the last S of the tile before is done
      for (int x = 0; x < H && ok && g > 0; ++x)
        ok = wait(bars + 2 * x + ((g - 1) & 1), ((g - 1) >> 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(bars + 13), H * kHalf);
        const int tok = t.q0 + (t.rr0 >> lg_g);
#pragma unroll
        for (int x = 0; x < H; ++x)
#pragma unroll
          for (int b = 0; b < NBOX; ++b)
            tma_load_4d(qb_u + x * kHalf + b * (kTpRows * 128), &tmQ, smem_u32(bars + 13), 0, t.h * p.G,
                        tok + x * (kTpRows >> lg_g), b);
      }
      __syncwarp();
      ok = wait(bars + 13, loads & 1);
      ++loads;
      for (int j = 0; j < ntile && ok; ++j, ++g) {
        const int slot = g % NS, sb = g & 1;
        ok = wait(full + slot, (g / NS) & 1);
        const uint32_t kst = ring_u + slot * STAGE;
#pragma unroll
        for (int x = 0; x < H; ++x) {
          // (S over the buffer once the PV MMAs of stage g - 2 have read its P)
          if (ok && g >= 2) ok = wait(bars + 8 + 2 * x + sb, ((g - 2) >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          // all 64 keys of the stage at once (keys of blocks a short stage did
          // not load give scores the softmax masks)
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
            umma_f16_warp(
                tS + (2 * x + sb) * SC,
                umma_desc_sw128(qb_u + x * kHalf + (ks >> 2) * (kTpRows * 128) + (ks & 3) * 32, 16, 1024),
                umma_desc_sw128(kst + (ks >> 2) * (TB * BLOCK_BYTES / NBOX) + (ks & 3) * 32, 16, 1024),
                idS, ks > 0 ? 1u : 0u);
          umma_commit_warp(smem_u32(bars + 2 * x + sb));  // S_x of stage g is ready
        }
      }
    }
    if (!ok) give_up();
    umma_commit_warp(smem_u32(bars + 12));  // this warp's MMAs have completed
  } else if (warp >= kPvWarp) {
    // ================= the PV MMAs of half x ================================
    const int x = warp - kPvWarp;
    const uint32_t idO = umma_idesc_f16(kTpRows, D, BF16, 0, 1);
    const uint32_t ring_u = smem_u32(ring);
    int g = 0;
    bool ok = true;
    Tile t;
    for (int n = 0; ok && take(n, t); ++n) {
      const int ntile = (t.nb + TB - 1) / TB;
      for (int j = 0; j < ntile; ++j, ++g) {
        const int pb = g & 1, slot = g % NS;
        // (P of a tile's first stage follows the softmax's last read of O)
        ok = wait(bars + 4 + 2 * x + pb, (g >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const int nbt = min(TB, t.nb - j * TB);
        const uint64_t dv = umma_desc_sw128(ring_u + slot * STAGE + TB * BLOCK_BYTES, 2048, 1024);
#pragma unroll
        for (int b = 0; b < TB; ++b)
          if (b < nbt)
            umma_f16_ts_warp(tO + x * D, tS + (2 * x + pb) * SC + 8 * b,
                             dv + (uint64_t)(b * BLOCK_BYTES / 16), idO, (j > 0 || b > 0) ? 1u : 0u);
        umma_commit_warp(smem_u32(bars + 8 + 2 * x + pb));  // P buffer pb free, O_x current
        umma_commit_warp(smem_u32(empty + slot));  // (with the other half's) the stage is free
      }
    }
    if (!ok) give_up();
    umma_commit_warp(smem_u32(bars + 12));  // this warp's MMAs have completed
  } else {
    // ================= softmax: one row per thread ==========================
    const int X = warp >> 2;  // this warp's half
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tOx = tO + X * D;
    const float sl2 = p.scale_log2;
    T *obase = static_cast<T *>(p.out);
    int g = 0;
    bool ok = true;
    Tile t;
    for (int n = 0; ok && take(n, t); ++n) {
      const int rr = t.rr0 + kTpRows * X + 32 * (warp & 3) + lane;
      const int rr_q = rr & ((1 << lg_g) - 1);  // q head of the kv head's
      const bool live = rr < t.rows && rr_q < p.G;
      const RowKeys keys = live ? row_keys(t.L, t.ml, rr >> lg_g, p.window) : RowKeys{0, 0};
      const int lo = keys.lo, hi = keys.hi;
      const int ntile = (t.nb + TB - 1) / TB;
      // The run of the tile's blocks leaves this many keys out, behind the
      // sinks: key k past them is the run's k - hole.  (No row sees keys of
      // the hole, nor a key of the sinks' blocks past the sinks.)
      const int hole = t.sk_gap * kBlockKeys;
      // Stages that may hold keys no row sees: those of the sinks' last block,
      // the window's first and the last one.
      const int j_hid0 = (t.sk_nb - 1) >> 2, j_hid2 = (t.nb - 1) >> 2;
      const int j_hid1 = (t.u_lo / kBlockKeys - t.sk_gap) >> 2;
      static_assert(TB == 4, "blocks of a stage");
      // Stages whose keys every row of the half sees: [0, j_sinks) and [j_lo, j_hi).
      int j_sinks, j_lo, j_hi;
      {
        // (a half without rows: any of these)
        const int last = min(t.rr0 + kTpRows * (X + 1), t.rows) - 1, first = min(t.rr0 + kTpRows * X, last);
        const int h_hi = row_keys(t.L, t.ml, first >> lg_g, p.window).hi;
        const int h_lo = row_keys(t.L, t.ml, last >> lg_g, p.window).lo;
        j_sinks = min(p.sinks, h_hi) / SC;
        const int b_lo = max((h_lo + kBlockKeys - 1) / kBlockKeys - t.sk_gap, t.sk_gap > 0 ? t.sk_nb : 0);
        j_lo = (b_lo + TB - 1) / TB;
        j_hi = min(h_hi / kBlockKeys - t.sk_gap, t.nb) / TB;
      }
      // (rows past the request's tokens or a token's heads hold other rows of q
      // or zeros and are never stored: an infinite reference makes their
      // weights 0)
      float m_used = live ? -INFINITY : INFINITY, lsum = 0.f;
      for (int j = 0; j < ntile; ++j, ++g) {
        const uint32_t tSx = tS + (2 * X + (g & 1)) * SC;  // S, then P, of the stage
        ok = wait(bars + 2 * X + (g & 1), (g >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        // the row's scores of the stage (fp32 bits), the second half's load
        // under way while the first half's exponentials are taken
        uint32_t sr[2][32];
        tmem_ld32(tSx + lane_base, sr[0]);
        tmem_wait_ld();
        tmem_ld32(tSx + lane_base + 32, sr[1]);
        const bool fast = j < j_sinks || (j >= j_lo && j < j_hi);
        // the keys of the stage that the row sees, as bits
        uint32_t vis[2] = {0xffffffffu, 0xffffffffu};
        if (!fast) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int at = SC * j + 32 * y;
            vis[y] = (low_bits(hi - hole - at) & ~low_bits(lo - hole - at)) | low_bits(min(p.sinks, hi) - at);
          }
        }
        // the row's largest scaled score of the stage, eight independent chains
        auto row_max = [&]() -> float {
          float a[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) a[u] = -INFINITY;
#pragma unroll
          for (int c = 0; c < SC; ++c)
            a[c & 7] = fmaxf(a[c & 7], (vis[c >> 5] & (1u << (c & 31)))
                                           ? __uint_as_float(sr[c >> 5][c & 31]) * sl2
                                           : -INFINITY);
#pragma unroll
          for (int u = 4; u >= 1; u >>= 1)
#pragma unroll
            for (int v = 0; v < u; ++v) a[v] = fmaxf(a[v], a[v + u]);
          return a[0];
        };
        // O_X *= alpha row by row in tensor memory (the whole warp), once the
        // PV MMAs of the stage before have completed
        auto rescale_o = [&](float alpha) -> bool {
          if (!wait(bars + 8 + 2 * X + ((g - 1) & 1), ((g - 1) >> 1) & 1)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tmem_ld32(tOx + lane_base + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(tOx + lane_base + c0, o);
          }
          tmem_wait_st();
          tc_fence_before();
          return true;
        };
        // P = 2^(x - m) against the row's reference m, rounded to the input
        // type; keys that the row does not see give 0.  Where every row has a
        // reference (with sinks, from the tile's first stage on) the max is
        // not taken: the largest P tells when a row's max grew more than 8
        // past its reference, and only then the row takes the max, O a
        // rescale and the stage its exponentials again.
        uint32_t w[2][16];
        auto exps = [&](int y, float mu) {
#pragma unroll
          for (int c = 0; c < 32; c += 2)
            w[y][c >> 1] = pack2(sfu_exp2(fmaf(__uint_as_float(sr[y][c]), sl2, -mu)),
                                 sfu_exp2(fmaf(__uint_as_float(sr[y][c + 1]), sl2, -mu)), tag{});
        };
        auto hide = [&]() {
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (!fast && __any_sync(0xffffffffu, vis[y] != 0xffffffffu)) {
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const uint32_t two = vis[y] >> (2 * c);
                w[y][c] &= ((two & 1u) | ((two << 15) & 0x10000u)) * 0xffffu;
              }
            }
        };
        // the reference raised to m_new where that is more than 8 past it
        auto raise = [&](float m_new) -> bool {
          const bool need = m_used != -INFINITY && m_new > m_used + 8.f;
          if (__any_sync(0xffffffffu, need)) {  // (implies j >= 1)
            const float alpha = need ? sfu_exp2(m_used - m_new) : 1.f;
            if (!rescale_o(alpha)) return false;
            if (need) {
              lsum *= alpha;
              m_used = m_new;
            }
          }
          return true;
        };
        const bool refs = __all_sync(0xffffffffu, m_used != -INFINITY);
        if (!refs) {
          wait_ld32(sr[1]);
          const float m_new = row_max();
          ok = raise(m_new);
          if (!ok) break;
          if (m_used == -INFINITY) m_used = m_new;
        }
        const float mu = m_used == -INFINITY ? 0.f : m_used;
        exps(0, mu);
        wait_ld32(sr[1]);
        exps(1, mu);
        hide();
        // (the largest as rounded; a NaN P is skipped, as by the max)
        if (refs && __any_sync(0xffffffffu, fmaxf(max2_of(w[0], tag{}), max2_of(w[1], tag{})) > 256.f)) {
          ok = raise(fmaxf(m_used, row_max()));
          if (!ok) break;
          exps(0, m_used);
          exps(1, m_used);
          hide();
        }
        tmem_st16(tSx + lane_base, w[0]);
        tmem_st16(tSx + lane_base + 16, w[1]);
        // zero V of keys no row of the tile sees (stale or NaN slots); each half
        // does it before its own PV MMAs (the other half's writes are the same
        // zeros)
        if (j == j_hid0 || j == j_hid1 || j == j_hid2) {
          constexpr int kV = D / 8;  // threads to a key's bytes
          const int v = lane % kV, c0 = (32 * (warp & 3) + lane) / kV;
          unsigned char *vb = ring + (g % NS) * STAGE + TB * BLOCK_BYTES + (v >> 3) * 2048 + (v & 7) * 16;
#pragma unroll 1
          for (int k = TB * j; k < min(TB * j + TB, t.nb); ++k) {
            const int k0 = (k >= t.sk_nb ? k + t.sk_gap : k) * kBlockKeys;
            if (k0 + kBlockKeys <= t.u_hi && (k0 >= t.u_lo || k0 + kBlockKeys <= p.sinks)) continue;
            for (int c = c0; c < kBlockKeys; c += 128 / kV)
              if (!(k0 + c < t.u_hi && (k0 + c >= t.u_lo || k0 + c < p.sinks)))
                *reinterpret_cast<uint4 *>(vb + (k - TB * j) * BLOCK_BYTES + c * 128) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();  // the zeros reach the tensor core
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(bars + 4 + 2 * X + (g & 1)));  // P of the stage written
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < SC / 2; ++c) ls[c & 3] = add2_f32(ls[c & 3], w[c >> 4][c & 15], tag{});
        lsum += (ls[0] + ls[1]) + (ls[2] + ls[3]);
      }
      if (!ok) break;

      // ---- O of the half: normalised and stored ------------------------------
      if (ntile > 0) {
        ok = wait(bars + 8 + 2 * X + ((g - 1) & 1), ((g - 1) >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
      }
      const float inv = (ntile > 0 && lsum > 0.f) ? sfu_rcp(lsum) : 0.f;
      unsigned long long row = 0;
      if (live) {
        const int i = rr >> lg_g;
        row = reinterpret_cast<unsigned long long>(obase + (int64_t)(t.q0 + i) * p.o_s0 +
                                                   (int64_t)(t.h * p.G + rr_q) * p.o_s1);
      }
      // Four lanes exchange their rows' 16-byte pieces, so that lane i of them
      // holds piece i of all four rows and they store 64-byte runs.
      const int i4 = lane & 3;
      unsigned long long rows4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) rows4[k] = __shfl_sync(0xffffffffu, row, (lane & ~3) + k);
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t w[4][4];  // [piece][word], 8 columns each
        {
          uint32_t o[32];
          if (ntile > 0) {
            tmem_ld32(tOx + lane_base + c0, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            w[i >> 3][(i >> 1) & 3] =
                pack2(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv, tag{});
        }
#pragma unroll
        for (int bit = 1; bit <= 2; bit <<= 1) {
          const bool up = i4 & bit;
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            if (a & bit) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[a][e] : w[a | bit][e], bit);
              if (up)
                w[a][e] = got;
              else
                w[a | bit][e] = got;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (rows4[k])
            *reinterpret_cast<uint4 *>(rows4[k] + 2 * c0 + 16 * i4) =
                make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
      }
      tc_fence_before();  // the next tile's P (and its PV MMAs over O) come after these reads
    }
    if (!ok) give_up();
  }

  // ---- the end: every MMA done, the tensor memory back -----------------------
  grid_dependents_launch();
  if (warp == 0 && !mbar_wait_bounded(smem_u32(bars + 12), 0) && lane == 0)
    atomicOr(p.status, PD_DEV_WAIT_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kCols);
  }
  if (blockIdx.x == 0) {
    // rows at and past the last request's end (padding) see no key: zeros
    const int t0 = min(max(__ldg(p.query_start + p.num_seqs), 0), p.num_tokens);
    const int per_row = p.Hq * (D / 8);
    for (int64_t i = tid; i < (int64_t)(p.num_tokens - t0) * per_row; i += blockDim.x) {
      const int tt = t0 + (int)(i / per_row), rem = (int)(i - (int64_t)(tt - t0) * per_row);
      const int hq = rem / (D / 8), c = rem - hq * (D / 8);
      *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (int64_t)tt * p.o_s0 + (int64_t)hq * p.o_s1 + c * 8) =
          make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

template <int D, bool BF16>
cudaError_t launch_window_prefill_t(const CUtensorMap &tk, const CUtensorMap &tv, const CUtensorMap &tq,
                                    const Params &p, const Launch &l, cudaStream_t stream) {
  auto kern = pd_window_prefill<D, BF16>;
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
  return cudaLaunchKernelEx(&cfg, kern, tk, tv, tq, p);
}

}  // namespace pd
