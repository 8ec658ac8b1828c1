// Rotary position embedding with a position per axis (time, height, width of
// an image or video token) and the store of k and v into the paged cache:
// pd_rope.cu's call, where rotated pair i takes its angle at the position of
// the axis pair_axis[i].
//
// One CTA per token.  A thread keeps one 16-byte chunk of the rotated dims
// (NeoX: dims 8c.. and rot/2 + 8c..; GPT-J: dims 8c..8c+7) and walks the q and
// k heads with it, so the angles of its pairs, gathered from as many table
// rows as the chunk has axes, are read once and stay in registers.  Then come
// the pass-through chunks past rot_dim and the v chunks.  Rotated in fp32,
// rounded once.  Memory-bound: every byte is read or written once.
#include "paged_step.h"
#include "pd_rope.cuh"

namespace pd {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxPairs = 256;  // rot_dim / 2 at head size 512

struct RopeAxesParams {
  RopeParams r;
  int64_t pos_stride;  // int32 between the axes' rows of positions
  int axes;
  uint8_t axis[kMaxPairs];
};

template <bool BF16, bool NEOX>
__global__ void __launch_bounds__(kThreads) pd_rope_axes(const __grid_constant__ RopeAxesParams pa) {
  const RopeParams &p = pa.r;
  constexpr int kPairs = NEOX ? 8 : 4;  // pairs of a chunk
  constexpr int kU = 4;                 // heads in flight per thread
  const int t = blockIdx.x;
  const int half = p.rot >> 1, heads = p.Hq + p.Hkv;
  const int chunks = half / kPairs;               // per head, <= 64
  const int c = threadIdx.x % chunks, h0 = threadIdx.x / chunks, hs = kThreads / chunks;
  // the inputs may be the previous kernel's outputs
  grid_dependency_wait();
  grid_dependents_launch();
  if (threadIdx.x < pa.axes) {
    const int pos = __ldg(p.positions + threadIdx.x * pa.pos_stride + t);
    if (pos < 0 || pos >= p.max_pos) atomicOr(p.status, PD_DEV_BAD_POSITION);
  }
  const int slot = __ldg(p.slots + t);
  const bool write_kv = slot >= 0 && (int64_t)slot < p.num_slots;
  if (slot >= 0 && !write_kv && threadIdx.x == 0) atomicOr(p.status, PD_DEV_BAD_SLOT);
  const int page = write_kv ? slot / p.P : 0, off = write_kv ? slot - page * p.P : 0;

  float co[kPairs], si[kPairs];
#pragma unroll
  for (int e = 0; e < kPairs; ++e) {
    const int i = kPairs * c + e;
    const int pos = __ldg(p.positions + pa.axis[i] * pa.pos_stride + t);
    const float *row = p.cos_sin + (int64_t)min(max(pos, 0), p.max_pos - 1) * p.cs_s0;
    co[e] = __ldg(row + i);
    si[e] = __ldg(row + half + i);
  }

  // dims [d, d + 8) of head hh (q heads first, then k heads): source and
  // destination.  Coherent loads: q_out may be q itself, and each chunk is
  // read and then written by the same thread.
  auto src_ptr = [&](int hh, int d) -> const uint4 * {
    const unsigned short *b = hh < p.Hq
        ? static_cast<const unsigned short *>(p.q) + (int64_t)t * p.q_s0 + (int64_t)hh * p.q_s1
        : static_cast<const unsigned short *>(p.k) + (int64_t)t * p.k_s0 +
              (int64_t)(hh - p.Hq) * p.k_s1;
    return reinterpret_cast<const uint4 *>(b + d);
  };
  auto dst_ptr = [&](int hh, int d) -> uint4 * {
    unsigned short *b = hh < p.Hq
        ? static_cast<unsigned short *>(p.q_out) + (int64_t)t * p.qo_s0 + (int64_t)hh * p.qo_s1
        : static_cast<unsigned short *>(p.k_cache) + (int64_t)page * p.kc_page +
              (int64_t)off * p.kc_tok + (int64_t)(hh - p.Hq) * p.kc_head;
    return reinterpret_cast<uint4 *>(b + d);
  };

  if (h0 < hs) {
#pragma unroll 1
    for (int hh0 = h0; hh0 < heads; hh0 += kU * hs) {
      uint4 w1[kU], w2[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int hh = hh0 + u * hs;
        w1[u] = w2[u] = make_uint4(0u, 0u, 0u, 0u);
        if (hh >= heads) continue;
        w1[u] = *src_ptr(hh, 8 * c);
        if (NEOX) w2[u] = *src_ptr(hh, half + 8 * c);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int hh = hh0 + u * hs;
        if (hh >= heads || (hh >= p.Hq && !write_kv)) continue;
        float x1[8], y1[8];
        unpack8<BF16>(w1[u], x1);
        if constexpr (NEOX) {
          float x2[8], y2[8];
          unpack8<BF16>(w2[u], x2);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y1[e] = x1[e] * co[e] - x2[e] * si[e];
            y2[e] = x2[e] * co[e] + x1[e] * si[e];
          }
          *dst_ptr(hh, 8 * c) = pack8<BF16>(y1);
          *dst_ptr(hh, half + 8 * c) = pack8<BF16>(y2);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y1[2 * e] = x1[2 * e] * co[e] - x1[2 * e + 1] * si[e];
            y1[2 * e + 1] = x1[2 * e + 1] * co[e] + x1[2 * e] * si[e];
          }
          *dst_ptr(hh, 8 * c) = pack8<BF16>(y1);
        }
      }
    }
  }
  // the dims past rot_dim of q and k, and v
  const int pass = (p.D - p.rot) / 8, n_pass = heads * pass;
  const int per_v = p.D / 8, n_v = write_kv ? p.Hkv * per_v : 0;
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < n_pass + n_v; i0 += kU * kThreads) {
    uint4 w[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = i0 + u * kThreads;
      w[u] = make_uint4(0u, 0u, 0u, 0u);
      if (i < n_pass) {
        const int hh = i / pass;
        w[u] = *src_ptr(hh, p.rot + 8 * (i - hh * pass));
      } else if (i < n_pass + n_v) {
        const int h = (i - n_pass) / per_v, cc = (i - n_pass) - h * per_v;
        w[u] = *reinterpret_cast<const uint4 *>(static_cast<const unsigned short *>(p.v) +
                                                (int64_t)t * p.v_s0 + (int64_t)h * p.v_s1 + 8 * cc);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = i0 + u * kThreads;
      if (i < n_pass) {
        const int hh = i / pass;
        if (hh < p.Hq || write_kv) *dst_ptr(hh, p.rot + 8 * (i - hh * pass)) = w[u];
      } else if (i < n_pass + n_v) {
        const int h = (i - n_pass) / per_v, cc = (i - n_pass) - h * per_v;
        *reinterpret_cast<uint4 *>(static_cast<unsigned short *>(p.v_cache) +
                                   (int64_t)page * p.vc_page + (int64_t)off * p.vc_tok +
                                   (int64_t)h * p.vc_head + 8 * cc) = w[u];
      }
    }
  }
}

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" PD_API int paged_rope_axes_cache_write(
    const pd_tensor *q, const pd_tensor *k, const pd_tensor *v, const pd_tensor *positions,
    const pd_tensor *slot_mapping, const pd_tensor *cos_sin_cache, const uint8_t *pair_axis,
    pd_tensor *q_out, pd_tensor *k_cache, pd_tensor *v_cache, int num_q_heads, int num_kv_heads,
    int head_size, int rot_dim, int page_size, int layout, int is_neox, void *stream) {
  if (!positions || !pair_axis || positions->ndim != 2) return PD_EINVAL;
  const int64_t axes = positions->shape[0];
  if (axes < 1 || axes > PD_MAX_AXES) return PD_EINVAL;
  if (positions->shape[1] > 1 && positions->stride[1] != 1) return PD_EALIGN;
  if (positions->stride[0] < 0) return PD_EINVAL;
  // one axis's row: the vector that the one-axis checks take
  pd_tensor row = *positions;
  row.ndim = 1;
  row.shape[0] = positions->shape[1];
  row.stride[0] = 1;
  RopeAxesParams p{};
  int rc = rope_params(q, k, v, &row, slot_mapping, cos_sin_cache, q_out, k_cache, v_cache,
                       num_q_heads, num_kv_heads, head_size, rot_dim, page_size, layout, is_neox,
                       &p.r);
  if (rc != PD_OK) return rc;
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (pair_axis[i] >= axes) return PD_EINVAL;
    p.axis[i] = pair_axis[i];
  }
  if (p.r.T == 0) return PD_OK;
  if ((rc = device_check(nullptr, &p.r.status)) != PD_OK) return rc;
  p.axes = (int)axes;
  p.pos_stride = positions->stride[0];

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.r.T);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool bf16 = q->dtype == PD_BF16;
  cudaError_t e;
  if (bf16)
    e = is_neox ? cudaLaunchKernelEx(&cfg, pd_rope_axes<true, true>, p)
                : cudaLaunchKernelEx(&cfg, pd_rope_axes<true, false>, p);
  else
    e = is_neox ? cudaLaunchKernelEx(&cfg, pd_rope_axes<false, true>, p)
                : cudaLaunchKernelEx(&cfg, pd_rope_axes<false, false>, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return PD_ECUDA;
  }
  return PD_OK;
}
