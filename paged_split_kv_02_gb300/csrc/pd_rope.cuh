// What the two rotary + cache-write kernels share: 16-bit pairs to and from
// fp32, and the host side of a call.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_decode.h"
#include "pd_internal.h"
#include "pd_ptx.cuh"

namespace pd {
namespace {

template <bool BF16>
struct Elem;
template <>
struct Elem<true> {
  using T2 = __nv_bfloat162;
  static __device__ __forceinline__ float2 to2(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<const T2 *>(&w));
  }
  static __device__ __forceinline__ uint32_t from2(float a, float b) {
    T2 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
  }
};
template <>
struct Elem<false> {
  using T2 = __half2;
  static __device__ __forceinline__ float2 to2(uint32_t w) {
    return __half22float2(*reinterpret_cast<const T2 *>(&w));
  }
  static __device__ __forceinline__ uint32_t from2(float a, float b) {
    T2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
  }
};

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  using E = Elem<BF16>;
  const float2 a = E::to2(w.x), b = E::to2(w.y), c = E::to2(w.z), d = E::to2(w.w);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
  uint4 w;
  w.x = Elem<BF16>::from2(y[0], y[1]);
  w.y = Elem<BF16>::from2(y[2], y[3]);
  w.z = Elem<BF16>::from2(y[4], y[5]);
  w.w = Elem<BF16>::from2(y[6], y[7]);
  return w;
}

inline bool aligned16(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

// [T, H, D] fp16/bf16 token rows: 16-byte aligned rows, innermost stride 1
inline int check_token_rows(const pd_tensor *t, int64_t T, int H, int D) {
  if (!t || t->ndim != 3 || (!t->data && T != 0)) return PD_EINVAL;  // (empty: any pointer)
  if (t->shape[0] != T || t->shape[1] != H || t->shape[2] != D) return PD_EINVAL;
  if (t->dtype != PD_F16 && t->dtype != PD_BF16) return PD_EDTYPE;
  if (t->stride[2] != 1) return PD_EALIGN;
  if (t->stride[0] < 0 || t->stride[1] < 0) return PD_EINVAL;
  if (t->stride[0] % 8 != 0 || t->stride[1] % 8 != 0 || !aligned16(t->data)) return PD_EALIGN;
  return PD_OK;
}

inline int check_i32_vector(const pd_tensor *t, int64_t n) {
  if (!t || (!t->data && n != 0) || t->ndim != 1 || t->shape[0] != n || t->stride[0] != 1)
    return PD_EINVAL;
  if (t->dtype != PD_I32) return PD_EDTYPE;
  return PD_OK;
}

// (page, token, kv head) element strides of a pool in its layout
inline void pool_strides(const pd_tensor *t, int layout, int64_t *page, int64_t *tok, int64_t *head) {
  *page = t->stride[0];
  *tok = layout == PD_NHD ? t->stride[1] : t->stride[2];
  *head = layout == PD_NHD ? t->stride[2] : t->stride[1];
}

// The checks of a call's tensors (the sizes, types and alignments that the
// public header gives) and its kernel parameters, all but the status word.
inline int rope_params(const pd_tensor *q, const pd_tensor *k, const pd_tensor *v,
                       const pd_tensor *positions, const pd_tensor *slot_mapping,
                       const pd_tensor *cos_sin_cache, pd_tensor *q_out, pd_tensor *k_cache,
                       pd_tensor *v_cache, int num_q_heads, int num_kv_heads, int head_size,
                       int rot_dim, int page_size, int layout, int is_neox, RopeParams *out) {
  if (!q || !k || !v || !positions || !slot_mapping || !cos_sin_cache || !q_out || !k_cache ||
      !v_cache)
    return PD_EINVAL;
  if (num_q_heads <= 0 || num_kv_heads <= 0) return PD_EINVAL;
  if (head_size != 64 && head_size != 128 && head_size != 256 && head_size != 512) return PD_EHEAD;
  if (page_size <= 0 || (layout != PD_NHD && layout != PD_HND)) return PD_EINVAL;
  if (rot_dim <= 0 || rot_dim > head_size || rot_dim % (is_neox ? 16 : 8) != 0) return PD_EINVAL;
  if (q->ndim != 3 || q->shape[0] < 0 || q->shape[0] > INT32_MAX) return PD_EINVAL;
  const int64_t T = q->shape[0];
  int rc;
  if ((rc = check_token_rows(q, T, num_q_heads, head_size)) != PD_OK) return rc;
  if ((rc = check_token_rows(q_out, T, num_q_heads, head_size)) != PD_OK) return rc;
  if ((rc = check_token_rows(k, T, num_kv_heads, head_size)) != PD_OK) return rc;
  if ((rc = check_token_rows(v, T, num_kv_heads, head_size)) != PD_OK) return rc;
  if ((rc = check_i32_vector(positions, T)) != PD_OK) return rc;
  if ((rc = check_i32_vector(slot_mapping, T)) != PD_OK) return rc;
  if ((rc = check_cache_tensor(k_cache, layout, num_kv_heads, page_size, head_size)) != PD_OK)
    return rc;
  if ((rc = check_cache_tensor(v_cache, layout, num_kv_heads, page_size, head_size)) != PD_OK)
    return rc;
  for (int i = 0; i < 4; ++i)
    if (k_cache->shape[i] != v_cache->shape[i]) return PD_EINVAL;
  const int dt = q->dtype;
  if (q_out->dtype != dt || k->dtype != dt || v->dtype != dt || k_cache->dtype != dt ||
      v_cache->dtype != dt)
    return PD_EDTYPE;
  const pd_tensor *cs = cos_sin_cache;
  if (!cs->data || cs->ndim != 2 || cs->shape[0] < 1 || cs->shape[0] > INT32_MAX ||
      cs->shape[1] < rot_dim || cs->stride[1] != 1 || cs->stride[0] < rot_dim)
    return PD_EINVAL;
  if (cs->dtype != PD_F32) return PD_EDTYPE;
  if (cs->stride[0] % 4 != 0 || !aligned16(cs->data)) return PD_EALIGN;
  out->q = q->data;
  out->q_s0 = q->stride[0];
  out->q_s1 = q->stride[1];
  out->k = k->data;
  out->k_s0 = k->stride[0];
  out->k_s1 = k->stride[1];
  out->v = v->data;
  out->v_s0 = v->stride[0];
  out->v_s1 = v->stride[1];
  out->q_out = q_out->data;
  out->qo_s0 = q_out->stride[0];
  out->qo_s1 = q_out->stride[1];
  out->k_cache = k_cache->data;
  out->v_cache = v_cache->data;
  pool_strides(k_cache, layout, &out->kc_page, &out->kc_tok, &out->kc_head);
  pool_strides(v_cache, layout, &out->vc_page, &out->vc_tok, &out->vc_head);
  out->positions = static_cast<const int32_t *>(positions->data);
  out->slots = static_cast<const int32_t *>(slot_mapping->data);
  out->cos_sin = static_cast<const float *>(cs->data);
  out->cs_s0 = cs->stride[0];
  out->max_pos = (int)cs->shape[0];
  out->T = (int)T;
  out->Hq = num_q_heads;
  out->Hkv = num_kv_heads;
  out->D = head_size;
  out->rot = rot_dim;
  out->P = page_size;
  out->num_slots = k_cache->shape[0] * (int64_t)page_size;
  return PD_OK;
}

}  // namespace
}  // namespace pd
