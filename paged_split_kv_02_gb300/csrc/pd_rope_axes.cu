// Rotary position embedding with a position per axis (time, height, width of
// an image or video token) and the store of k and v into the paged cache:
// pd_rope.cu's call, where rotated pair i takes its angle at the position of
// the axis pair_axis[i].
//
// The token's angles, gathered from as many table rows as its pairs have axes,
// go to shared memory once.  A thread keeps one 16-byte chunk of the rotated
// dims (NeoX: dims 8c.. and rot/2 + 8c..; GPT-J: dims 8c..8c+7) and walks the
// q and k heads with it, the chunk's angles in registers; the first loads of q
// and k, then the dims past rot_dim and v, which need no angle, are under way
// before the angles arrive.  Rotated in fp32, rounded once.  Memory-bound:
// every byte is read or written once.
//
// A CTA per token: of 128 threads with four heads in flight each when few tokens
// leave the SMs empty (fewer than 8 per SM: 64 tokens of 32 / 8 heads at D = 128
// 3.4 us; with 64 threads and one head 4.3), else of 64 threads, one head and
// the next, and as many CTAs as registers allow: 16384 such tokens 69 us (89
// % of the measured copy rate; two tokens to a CTA 71, 128 threads 76 - 80, a
// warp per token 69 - 73, four heads in flight 110, angles gathered by every
// thread 122); 5001 tokens of 16 / 2 heads at D = 256 with 64 rotated dims 22
// us (71 %; two loads in flight past rot_dim 23, eight 25).
#include "paged_step.h"
#include "pd_rope.cuh"

namespace pd {
namespace {

constexpr int kFewGroup = 128;  // threads of a token when there are few
constexpr int kManyGroup = 64;  // and when there are many
constexpr int kMaxPairs = 256;  // rot_dim / 2 at head size 512

struct RopeAxesParams {
  RopeParams r;
  int64_t pos_stride;  // int32 between the axes' rows of positions
  int axes;
  uint8_t axis[kMaxPairs];
};

// kGroup: threads of a token; kU: heads whose loads a thread has in flight;
// the loads of the next kU are issued before the present ones are turned and
// stored.
template <bool BF16, bool NEOX, int kGroup, int kU>
__global__ void __launch_bounds__(kGroup, kGroup == kManyGroup ? (NEOX ? 16 : 20) : 1)
    pd_rope_axes(const __grid_constant__ RopeAxesParams pa) {
  const RopeParams &p = pa.r;
  constexpr int kPairs = NEOX ? 8 : 4;  // pairs of a chunk
  // the token's angles: cos, then sin
  __shared__ __align__(16) float cs[2 * kMaxPairs];
  const int me = threadIdx.x, t = blockIdx.x;
  const int half = p.rot >> 1, heads = p.Hq + p.Hkv;
  const int chunks = half / kPairs;            // per head, <= 64
  const int wide = min(chunks, kGroup);        // chunks taken at a time
  const int h0 = me / wide, c0 = me - h0 * wide, hs = kGroup / wide;

  // dims [d, d + 8) of head hh (q heads first, then k heads).  Coherent
  // loads: q_out may be q itself, and each chunk is read and then written by
  // the same thread.
  auto src_ptr = [&](int hh, int d) -> const uint4 * {
    const unsigned short *b = hh < p.Hq
        ? static_cast<const unsigned short *>(p.q) + (int64_t)t * p.q_s0 + (int64_t)hh * p.q_s1
        : static_cast<const unsigned short *>(p.k) + (int64_t)t * p.k_s0 +
              (int64_t)(hh - p.Hq) * p.k_s1;
    return reinterpret_cast<const uint4 *>(b + d);
  };
  uint4 w1[kU], w2[kU];
  auto load = [&](int hh0, int c) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int hh = hh0 + u * hs;
      w1[u] = w2[u] = make_uint4(0u, 0u, 0u, 0u);
      if (hh >= heads || c >= chunks) continue;
      w1[u] = *src_ptr(hh, 8 * c);
      if (NEOX) w2[u] = *src_ptr(hh, half + 8 * c);
    }
  };
  // the inputs may be the previous kernel's outputs
  grid_dependency_wait();
  grid_dependents_launch();
  const int first = h0 < hs ? h0 : heads;
  load(first, c0);
  const int slot = __ldg(p.slots + t);
  if (me < pa.axes) {
    const int pos = __ldg(p.positions + me * pa.pos_stride + t);
    if (pos < 0 || pos >= p.max_pos) atomicOr(p.status, PD_DEV_BAD_POSITION);
  }
  // the angles of the token's pairs, once
  for (int i = me; i < half; i += kGroup) {
    const int pos = __ldg(p.positions + pa.axis[i] * pa.pos_stride + t);
    const float *row = p.cos_sin + (int64_t)min(max(pos, 0), p.max_pos - 1) * p.cs_s0;
    cs[i] = __ldg(row + i);
    cs[half + i] = __ldg(row + half + i);
  }
  const bool write_kv = slot >= 0 && (int64_t)slot < p.num_slots;
  if (slot >= 0 && !write_kv && me == 0) atomicOr(p.status, PD_DEV_BAD_SLOT);
  const int page = write_kv ? slot / p.P : 0, off = write_kv ? slot - page * p.P : 0;
  auto dst_ptr = [&](int hh, int d) -> uint4 * {
    unsigned short *b = hh < p.Hq
        ? static_cast<unsigned short *>(p.q_out) + (int64_t)t * p.qo_s0 + (int64_t)hh * p.qo_s1
        : static_cast<unsigned short *>(p.k_cache) + (int64_t)page * p.kc_page +
              (int64_t)off * p.kc_tok + (int64_t)(hh - p.Hq) * p.kc_head;
    return reinterpret_cast<uint4 *>(b + d);
  };
  // the dims past rot_dim of q and k, and v
  constexpr int kW = 4;
  const int pass = (p.D - p.rot) / 8, n_pass = heads * pass;
  const int per_v = p.D / 8, n_v = write_kv ? p.Hkv * per_v : 0;
#pragma unroll 1
  for (int i0 = me; i0 < n_pass + n_v; i0 += kW * kGroup) {
    uint4 w[kW];
#pragma unroll
    for (int u = 0; u < kW; ++u) {
      const int i = i0 + u * kGroup;
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
    for (int u = 0; u < kW; ++u) {
      const int i = i0 + u * kGroup;
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
  __syncthreads();
#pragma unroll 1
  for (int c = c0; c < chunks; c += wide) {
    if (c != c0) load(first, c);
    float co[kPairs], si[kPairs];
#pragma unroll
    for (int e = 0; e < kPairs; e += 4) {
      const float4 a = *reinterpret_cast<const float4 *>(cs + kPairs * c + e);
      const float4 b = *reinterpret_cast<const float4 *>(cs + half + kPairs * c + e);
      co[e] = a.x; co[e + 1] = a.y; co[e + 2] = a.z; co[e + 3] = a.w;
      si[e] = b.x; si[e + 1] = b.y; si[e + 2] = b.z; si[e + 3] = b.w;
    }
#pragma unroll 1
    for (int hh0 = first; hh0 < heads; hh0 += kU * hs) {
      uint4 v1[kU], v2[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        v1[u] = w1[u];
        v2[u] = w2[u];
      }
      if (hh0 + kU * hs < heads) load(hh0 + kU * hs, c);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int hh = hh0 + u * hs;
        if (hh >= heads || (hh >= p.Hq && !write_kv)) continue;
        float x1[8], y1[8];
        unpack8<BF16>(v1[u], x1);
        if constexpr (NEOX) {
          float x2[8], y2[8];
          unpack8<BF16>(v2[u], x2);
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
  int num_sms = 0;
  if ((rc = device_check(&num_sms, &p.r.status)) != PD_OK) return rc;
  p.axes = (int)axes;
  p.pos_stride = positions->stride[0];

  cudaLaunchConfig_t cfg = {};
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool bf16 = q->dtype == PD_BF16, few = (int64_t)p.r.T * 4 < (int64_t)num_sms * 32;
  cfg.gridDim = dim3((unsigned)p.r.T);
  cfg.blockDim = dim3(few ? kFewGroup : kManyGroup);
  auto launch = [&](auto kern) { return cudaLaunchKernelEx(&cfg, kern, p); };
  cudaError_t e;
  if (few)
    e = bf16 ? (is_neox ? launch(pd_rope_axes<true, true, kFewGroup, 4>) : launch(pd_rope_axes<true, false, kFewGroup, 4>))
             : (is_neox ? launch(pd_rope_axes<false, true, kFewGroup, 4>) : launch(pd_rope_axes<false, false, kFewGroup, 4>));
  else
    e = bf16 ? (is_neox ? launch(pd_rope_axes<true, true, kManyGroup, 1>) : launch(pd_rope_axes<true, false, kManyGroup, 1>))
             : (is_neox ? launch(pd_rope_axes<false, true, kManyGroup, 1>) : launch(pd_rope_axes<false, false, kManyGroup, 1>));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return PD_ECUDA;
  }
  return PD_OK;
}
