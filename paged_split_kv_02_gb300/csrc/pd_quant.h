// What the calls on an 8-bit cache share: the kernel parameters, the plan's
// constants and the host's argument checks.
#pragma once

#include "paged_quant.h"
#include "pd_internal.h"

namespace pd {

// An 8-bit pool and its scales: element strides of (page, token, kv head), and
// of the scales (page, block of 16 tokens, kv head).
struct QuantPool {
  unsigned char *codes;
  int64_t page, tok, head;
  float *scale;
  int64_t s_page, s_blk, s_head;
};

// Division of whole numbers from 0 to 2^31 - 1 by a number that the host knows.
struct FastDiv {
  uint32_t mul = 1u << 31;
  int shift = 31;
  FastDiv() = default;
  explicit FastDiv(uint32_t d) {
    int l = 0;
    while ((1ull << l) < d) ++l;
    // ceil(2^(31 + l) / d), at most d - 1 < 2^l over: n times that stays below 2^(31 + l)
    shift = 31 + l;
    mul = (uint32_t)(((1ull << shift) + d - 1) / d);
  }
#ifdef __CUDACC__
  __device__ __forceinline__
#endif
  uint32_t div(int n) const { return (uint32_t)(((uint64_t)(uint32_t)n * mul) >> shift); }
};

// Attention over an 8-bit cache (pd_quant_attn.cuh).
struct QuantAttnParams {
  const void *q;
  int64_t q_s0, q_s1;
  void *out;
  int64_t o_s0, o_s1;
  QuantPool k, v;
  const int32_t *block_table;
  int64_t bt_stride;
  int bt_width;
  const int32_t *seq_lens, *query_start;
  int num_seqs, num_tokens, num_pages;
  int Hq, Hkv, G, M, P, bpp, window, sinks;  // bpp: 16-key blocks of a page
  float scale_log2;  // scale x log2(e): the softmax runs on exp2
  int rg, rows_grp;  // row groups of a kv head's packed rows, rows of one
  int seqs_y;        // sequences of one blockIdx.y
  int whole;         // 1: no unit is cut
  int min_share;     // the least share of a CTA
  int min_part;      // the fewest blocks of a part of an aligned unit
  FastDiv by_units, by_groups, by_heads, by_page, by_ctas;  // Hkv rg, rg, G, bpp, gridDim.x
  float *part_acc, *part_ml;  // [2 x CTAs][8 NT][D], [..][8 NT][2]
  int *counters;              // [units][unit_counters]: parts published, of a unit and of its groups
  int unit_counters;
  int merge_bytes;            // of a unit's parts that one CTA merges at once
  unsigned int *status;
};

// What a unit counts in the line of blocks beside its blocks: its end, the last
// round of its steps, its first references take a CTA 4 us (32 requests of 1..4
// tokens, 32 / 8 heads at D = 128, 12 / 24 / 40 / 64: 76 / 74 / 66 / 69 us).
constexpr int quant_unit_cost(int D) { return D == 64 ? 80 : D == 128 ? 40 : D == 256 ? 28 : 16; }
// Sequences of one line at most (their lengths and places lie in shared memory).
constexpr int kQuantSeqs = 448;
constexpr int kQuantWarps = 8;
// 16-key blocks of a warp's step; slots of its ring, each K or V of a step; n-tiles of
// 8 packed rows with their sums in registers.  The slots take the shared memory that
// there is; 64 requests of 4,096 tokens, 8 kv heads (2 at D = 256), in us: at D = 64 steps
// of 1 / 2 / 4 blocks 85 / 70 / 60 (with 32 rows, 16 requests: 37 / 36 / 40), at 128 of 1 / 2 /
// 4 104 / 89 / 91, with 3 slots for 6 of 2 blocks 93, at 256 of 1 / 2 54 / 53.
constexpr int quant_step_blocks(int D, int NT) { return D == 64 ? (NT <= 2 ? 4 : 2) : D <= 256 ? 2 : 1; }
constexpr int quant_slots(int D, int NT) { return D >= 256 ? 3 : 6; }
constexpr int quant_max_tiles(int D) { return D == 64 ? 4 : 512 / D; }
constexpr int quant_slot_bytes(int D, int NT) { return quant_step_blocks(D, NT) * 16 * D + 32; }
// passes over the columns when a CTA's warps add their sums, each in one slot
constexpr int quant_passes(int D, int NT) {
  return 2 * NT > quant_step_blocks(D, NT) ? 2 * NT / quant_step_blocks(D, NT) : 1;
}
// pieces of a share whose place is known at a time (a power of two): a warp looks
// at most four runs of its own ahead, and one of eight pieces has one
constexpr int kQuantPieces = 64;
constexpr int kQuantRunBytes = 40, kQuantPieceBytes = 76;
// Dynamic shared memory: the warps' rings, two sets of Q fragments, row scales and
// row ends, the warps' (m, l) of the rows, the pieces, two runs of each warp, sums
// and flags, lengths, first rows, blocks, order and places.
constexpr int smem_bytes_quant(int D, int NT, int seqs) {
  return 128 + kQuantWarps * quant_slots(D, NT) * quant_slot_bytes(D, NT) + 2 * (NT * 16 * D + 8 * NT * 8) +
         8 * NT * kQuantWarps * 8 + (kQuantPieces + 2) * kQuantPieceBytes + kQuantWarps * 2 * kQuantRunBytes +
         4 * (2 * kQuantWarps + 8) + 4 * (5 * seqs + 1);
}

cudaError_t launch_quant_d64(bool bf16, int nt, const QuantAttnParams &p, const Launch &l, cudaStream_t stream);
cudaError_t launch_quant_d128(bool bf16, int nt, const QuantAttnParams &p, const Launch &l, cudaStream_t stream);
cudaError_t launch_quant_d256(bool bf16, int nt, const QuantAttnParams &p, const Launch &l, cudaStream_t stream);
cudaError_t launch_quant_d512(bool bf16, int nt, const QuantAttnParams &p, const Launch &l, cudaStream_t stream);

// An 8-bit pool's descriptors, checked, and its strides.
int quant_pool(const pd_tensor *cache, const pd_tensor *scale, int layout, int Hkv, int P, int D,
               QuantPool *out);

}  // namespace pd
