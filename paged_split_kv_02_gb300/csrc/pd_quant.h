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
  int Hq, Hkv, G, M, P, window, sinks;
  float scale_log2;  // scale x log2(e): the softmax runs on exp2
  int rg, rows_grp;  // row groups of a kv head's packed rows, rows of one
  int seqs_y;        // sequences of one blockIdx.y
  int whole;         // 1: no unit is cut
  int min_share;     // the least share of a CTA
  float *part_acc, *part_ml;  // [2 x CTAs][8 NT][D], [..][8 NT][2]
  int *counters;              // parts published of each unit
  unsigned int *status;
};

// Sequences of one line at most (their lengths and places lie in shared memory).
constexpr int kQuantSeqs = 1024;
// 16-key blocks of a warp's step, its steps in flight and the warps of a CTA;
// n-tiles of 8 packed rows with their sums in registers.
constexpr int quant_step_blocks(int D, int NT) { return D == 64 && NT <= 2 ? 2 : 1; }
constexpr int quant_stages(int D, int NT) { return D == 512 ? 2 : 3; }
constexpr int quant_max_tiles(int D) { return D == 64 ? 4 : 512 / D; }
constexpr int quant_max_warps(int D, int NT) { return NT * D >= 512 ? 8 : 12; }
// passes over the columns when a CTA's warps add their sums
constexpr int quant_passes(int D, int NT) { return NT * D > 128 ? NT * D / 128 : 1; }
constexpr int quant_stage_bytes(int D, int NT) { return quant_step_blocks(D, NT) * (32 * D + 16); }
// Dynamic shared memory: the warps' rings, the sums of one pass, (m, l) of every
// warp's rows, two sets of Q fragments, row scales and row ends, lengths, first
// rows and places.
constexpr int smem_bytes_quant(int D, int NT, int NW, int NS, int seqs) {
  return 128 + NW * NS * quant_stage_bytes(D, NT) + NW * 8 * NT * (D / quant_passes(D, NT)) * 4 +
         NW * 8 * NT * 8 + 2 * (NT * 16 * D + 8 * NT * 8) + 4 * (3 * seqs + 2) + 64 * 4;
}

cudaError_t launch_quant_d64(bool bf16, int nt, const QuantAttnParams &p, const Launch &l, cudaStream_t stream);
cudaError_t launch_quant_d128(bool bf16, int nt, const QuantAttnParams &p, const Launch &l, cudaStream_t stream);
cudaError_t launch_quant_d256(bool bf16, int nt, const QuantAttnParams &p, const Launch &l, cudaStream_t stream);
cudaError_t launch_quant_d512(bool bf16, int nt, const QuantAttnParams &p, const Launch &l, cudaStream_t stream);

// An 8-bit pool's descriptors, checked, and its strides.
int quant_pool(const pd_tensor *cache, const pd_tensor *scale, int layout, int Hkv, int P, int D,
               QuantPool *out);

}  // namespace pd
