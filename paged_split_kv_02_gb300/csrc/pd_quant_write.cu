// The rotary embedding of q and k and the store of k and v into an 8-bit cache.
//
// Two kinds of CTAs.  Of q: some tokens, rotated as in pd_rope_axes.cu (a token's angles in
// shared memory once, a thread keeps one 16-byte chunk of dims and walks the heads).
// Of k and v: the runs of tokens that begin in a few neighbouring tokens; a run
// is the new tokens of one 16-token block, and a unit of work is a run's K or V
// of one kv head, 16 rows at most, held in fp32 in the registers of one warp (two at
// head size 256, four at 512) from the load to the codes: read once, the largest
// magnitude by shuffles, then scaled and stored, 8 codes a lane.  An appended
// block's other codes are read and written again where its scale grows.
//
// The rotation rounds each product and the sum (no fused multiply-add), so that a
// code, which sits on a rounding, does not depend on how a compiler pairs them.
//
// Memory-bound: every byte is read or written once but for the rescaled codes.  A
// prompt of 16,384 tokens, 32 / 8 heads of 128: 71 us, 5.3 TB/s, 78 % of a copy's rate;
// k and v alone take 29 (angles one float at a time, read with two-way bank conflicts:
// 34), 23 without a rotation.  64 tokens, one a request: 4.4 us, 2.5 of them a launch.
//
// No two units may have a block at once.  A unit therefore looks through the kLook
// tokens before its run for another slot of the block, while its rows are loaded, and
// leaves its run out if there is one (900 appends 18.8 -> 19.0 us; done before the loads
// 19.4).
#include "pd_e4m3.cuh"
#include "pd_quant.h"
#include "pd_rope.cuh"

#include <algorithm>

namespace pd {
namespace {

constexpr int kLgThreads = 7, kThreads = 1 << kLgThreads;
constexpr int kCtas = 5;        // of an SM where tokens are many (k and v of the prompt above with 5 / 6: 29 / 33 us)
constexpr int kWindow = 64;     // tokens of a k/v CTA at most: 16 a warp
constexpr int kLook = PD_RUN_DISTANCE;  // tokens before a run among which its block may not be
constexpr int kAngleBytes = 40 << 10;  // of their angles
constexpr int kMaxPairs = 256;  // rot_dim / 2 at head size 512
constexpr int kLeast = -64;     // the exponent of the least scale

struct QuantWriteParams {
  const void *q, *k, *v;
  int64_t q_s0, q_s1, k_s0, k_s1, v_s0, v_s1;
  void *q_out;
  int64_t qo_s0, qo_s1;
  QuantPool kc, vc;
  const int32_t *positions, *slots;
  int64_t pos_stride;
  const float *cos_sin;
  int64_t cs_s0;
  int max_pos, T, Hq, Hkv, rot, P, axes;
  int64_t num_slots;
  int window, slices, units;  // tokens of a k/v CTA, CTAs of a window, units of one
  int kv_ctas;                // k/v CTAs come first
  int lg_group;               // log2 of the threads of a token of q
  unsigned int *status;
  alignas(4) uint8_t axis[kMaxPairs];
};

__device__ __forceinline__ void turn(float a, float b, float c, float s, float &x, float &y) {
  x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// The angles of token t's pairs to cs (cos, then sin), by n threads.
__device__ __forceinline__ void load_angles(const QuantWriteParams &p, int t, float *cs, int me, int n) {
  const int half = p.rot >> 1;
  if (me < p.axes) {
    const int pos = __ldg(p.positions + me * p.pos_stride + t);
    if (pos < 0 || pos >= p.max_pos) atomicOr(p.status, PD_DEV_BAD_POSITION);
  }
  for (int i = me; i < half; i += n) {
    const int pos = __ldg(p.positions + p.axis[i] * p.pos_stride + t);
    const float *row = p.cos_sin + (int64_t)min(max(pos, 0), p.max_pos - 1) * p.cs_s0;
    cs[i] = __ldg(row + i);
    cs[half + i] = __ldg(row + half + i);
  }
}

// q of some tokens, 2^lg threads each, kU heads in flight.
template <int D, bool BF16, bool NEOX, int kU>
__device__ __forceinline__ void q_tokens(const QuantWriteParams &p, int t0, int lg, float *smem) {
  constexpr int kPairs = NEOX ? 8 : 4;  // pairs of a chunk
  const int group = 1 << lg, me = threadIdx.x & (group - 1), t = t0 + (threadIdx.x >> lg);
  float *cs = smem + (threadIdx.x >> lg) * p.rot;
  const int half = p.rot >> 1, chunks = half / kPairs;
  const bool live = t < p.T;
  // (coherent loads: q_out may be q, and a thread reads what it writes, before)
  auto src = [&](int h, int d) -> const uint4 * {
    return reinterpret_cast<const uint4 *>(static_cast<const unsigned short *>(p.q) + (int64_t)t * p.q_s0 +
                                           (int64_t)h * p.q_s1 + d);
  };
  auto dst = [&](int h, int d) -> uint4 * {
    return reinterpret_cast<uint4 *>(static_cast<unsigned short *>(p.q_out) + (int64_t)t * p.qo_s0 +
                                     (int64_t)h * p.qo_s1 + d);
  };
  const int wide = max(min(chunks, group), 1);  // chunks taken at a time
  const int h0 = me / wide, c0 = me - h0 * wide, hs = group / wide;
  const int first = live && chunks > 0 && h0 < hs ? h0 : p.Hq;
  uint4 w1[kU], w2[kU];
  auto load = [&](int hh, int c) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = hh + u * hs;
      w1[u] = w2[u] = make_uint4(0u, 0u, 0u, 0u);
      if (h >= p.Hq || c >= chunks) continue;
      w1[u] = *src(h, 8 * c);
      if (NEOX) w2[u] = *src(h, half + 8 * c);
    }
  };
  load(first, c0);
  if (live && p.rot > 0) load_angles(p, t, cs, me, group);
  if (live) {
    // dims past rot_dim
    constexpr int kW = 4;
    const int pass = (D - p.rot) / 8, n = p.Hq * pass;
#pragma unroll 1
    for (int i0 = me; i0 < n; i0 += kW * group) {
      uint4 w[kW];
#pragma unroll
      for (int u = 0; u < kW; ++u) {
        const int i = i0 + u * group;
        w[u] = make_uint4(0u, 0u, 0u, 0u);
        if (i < n) w[u] = *src(i / pass, p.rot + 8 * (i % pass));
      }
#pragma unroll
      for (int u = 0; u < kW; ++u) {
        const int i = i0 + u * group;
        if (i < n) *dst(i / pass, p.rot + 8 * (i % pass)) = w[u];
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
    for (int hh = first; hh < p.Hq; hh += kU * hs) {
      uint4 v1[kU], v2[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        v1[u] = w1[u];
        v2[u] = w2[u];
      }
      if (hh + kU * hs < p.Hq) load(hh + kU * hs, c);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = hh + u * hs;
        if (h >= p.Hq) continue;
        float x1[8], y1[8];
        unpack8<BF16>(v1[u], x1);
        if constexpr (NEOX) {
          float x2[8], y2[8];
          unpack8<BF16>(v2[u], x2);
#pragma unroll
          for (int e = 0; e < 8; ++e) turn(x1[e], x2[e], co[e], si[e], y1[e], y2[e]);
          *dst(h, 8 * c) = pack8<BF16>(y1);
          *dst(h, half + 8 * c) = pack8<BF16>(y2);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) turn(x1[2 * e], x1[2 * e + 1], co[e], si[e], y1[2 * e], y1[2 * e + 1]);
          *dst(h, 8 * c) = pack8<BF16>(y1);
        }
      }
    }
  }
}

// The smallest power of two, 2^kLeast at least, under which a is at most 448 =
// 1.75 x 2^8.
__device__ __forceinline__ float least_scale(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int e = (int)(bits >> 23) - 127 - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return __uint_as_float((uint32_t)(max(e, kLeast) + 127) << 23);
}

// (FEW: its runs stay in registers, of 16 tokens at most; 0.2 us of a small call)
template <int D, bool BF16, bool NEOX, bool FEW>
__device__ __forceinline__ void kv_runs(const QuantWriteParams &p, int cta, float *smem) {
  constexpr int WU = D > 128 ? D / 128 : 1;  // warps of a unit
  constexpr int SLOTS = kThreads / 32 / WU;  // units at a time
  // a thread has two 16-byte chunks of a row: of K under NeoX's rotation those that
  // are rotated together, else neighbours
  constexpr int LPR = D / 16;                // threads of a row
  constexpr int RPP = 32 * WU / LPR;         // rows that a unit's threads have at once
  constexpr int NP = PD_SCALE_TOKENS / RPP;  // rows of a thread
  constexpr int kTokens = kWindow + PD_SCALE_TOKENS - 1;  // of a CTA at most
  // (a CTA of 16 tokens, or 1, loads its slots and those before them in one go)
  static_assert(kLook + 2 * PD_SCALE_TOKENS <= kThreads, "slots a thread each");
  __shared__ int slots_at[kLook + kTokens];                // of tokens t0 - kLook ..
  const int *const slot_of = slots_at + kLook;             // of tokens t0 ..
  __shared__ int row_of[PD_MAX_AXES * kTokens];            // the angles' rows of tokens t0 .., axis by axis
  // the runs, in order: a warp's at 16 times its number; first token, tokens and the slots of
  // the block that are written
  __shared__ int run_count[kThreads / 32], run_lead[kWindow], run_n[kWindow];
  __shared__ uint32_t run_mask[kWindow];
  __shared__ float top[kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wi = cta / p.slices, slice = cta - wi * p.slices;
  const int t0 = wi * p.window;
  const int u0 = slice * p.units, nu = min(p.units, 2 * p.Hkv - u0);
  for (int i = tid; i < kLook + p.window + PD_SCALE_TOKENS - 1; i += kThreads) {
    const int t = t0 - kLook + i;
    int s = t >= 0 && t < p.T ? __ldg(p.slots + t) : -1;
    if (s >= 0 && s >= p.num_slots) {
      if (slice == 0) atomicOr(p.status, PD_DEV_BAD_SLOT);
      s = -1;
    }
    slots_at[i] = s;
  }
  const bool angles = u0 < p.Hkv && p.rot > 0;
  if (angles) {
    const int lg = p.window > PD_SCALE_TOKENS ? 7 : 5, near = p.window + PD_SCALE_TOKENS - 1;
    for (int i = tid; i < p.axes << lg; i += kThreads) {
      const int axis = i >> lg, j = i & ((1 << lg) - 1), t = t0 + j;
      if (j >= near) continue;
      const int pos = t < p.T ? __ldg(p.positions + axis * p.pos_stride + t) : 0, row = min(max(pos, 0), p.max_pos - 1);
      row_of[axis * kTokens + j] = row;
      // (of q's tokens q's CTAs report)
      if (p.q == nullptr && j < p.window && row != pos) atomicOr(p.status, PD_DEV_BAD_POSITION);
    }
  }
  __syncthreads();
  // the runs that begin here: warp w has those of tokens 16 w .. (up to 16 tokens every warp has
  // them all, and waits for none), a lane token 16 w - 1 + lane: 31 of them and the one before
  const bool wide = !FEW && p.window > PD_SCALE_TOKENS;
  int n = 0;              // of the run that begins with token first16 + lane
  uint32_t written = 0, begins;
  int n_runs = 0, lead0 = 0, t_end = 0;
  {
    const int first16 = wide ? warp * PD_SCALE_TOKENS : 0, own = min(p.window - first16, PD_SCALE_TOKENS);
    if (own > 0) {
      const int s = lane < own + 16 ? slot_of[first16 - 1 + lane] : -1, before = __shfl_up_sync(0xffffffffu, s, 1);
      const bool same = s >= 0 && before >= 0 && s / PD_SCALE_TOKENS == before / PD_SCALE_TOKENS;
      const uint32_t on = __ballot_sync(0xffffffffu, same && s > before);    // goes on with the token before
      const uint32_t bad = __ballot_sync(0xffffffffu, same && s <= before);  // should
      const uint32_t first = __ballot_sync(0xffffffffu, s >= 0 && !same) & ~1u;
      // token first16 + lane is lane + 1 of the masks
      if (lane < own && first >> (lane + 1) & 1u) {
        const uint32_t after = lane < 30 ? on >> (lane + 2) : 0u;
        n = min(__ffs(~after), PD_SCALE_TOKENS);  // (ones from there on, and itself)
        for (int j = 0; j < n; ++j) written |= 1u << (slot_of[first16 + lane + j] & 15);
      }
      // (each token by the CTA, or the warp, that it is one of, whichever has the run before it)
      if (lane < own && bad >> (lane + 1) & 1u && slice == 0) atomicOr(p.status, PD_DEV_BAD_SLOT);
    }
    begins = __ballot_sync(0xffffffffu, n > 0);
    if (!FEW && n > 0) {
      const int at = first16 + __popc(begins & ((1u << lane) - 1));
      run_lead[at] = first16 + lane;
      run_n[at] = n;
      run_mask[at] = written;
    }
    if (!FEW && lane == 0) run_count[first16 / PD_SCALE_TOKENS] = __popc(begins);
  }
  if constexpr (FEW) {
    if (begins == 0) return;  // (every warp alike)
    n_runs = __popc(begins);
    lead0 = __ffs(begins) - 1;
    const int last = 31 - __clz(begins);
    t_end = last + __shfl_sync(0xffffffffu, n, last);
  } else {
    if (wide) __syncthreads();
    else __syncwarp();
    for (int w = 0; w < (wide ? kThreads / 32 : 1); ++w) {
      const int c = run_count[w], at = w * PD_SCALE_TOKENS;
      if (c > 0) {
        if (n_runs == 0) lead0 = run_lead[at];
        t_end = run_lead[at + c - 1] + run_n[at + c - 1];
      }
      n_runs += c;
    }
    if (n_runs == 0) return;
  }
  const int half = p.rot >> 1;
  // where pairs e .. e + 3 lie among a token's cosines (and sines): first the even fours, then the odd
  // ones, so that the lanes of a row read side by side
  auto angle_at = [&](int e) { return (e & 4 ? (half + 4) / 8 * 4 : 0) + (e >> 3) * 4; };
  if (angles) {
    // four pairs of a token at a time, four of those of a thread (half is a multiple of 4)
    const int quads = half / 4, n = (t_end - lead0) * quads;
#pragma unroll 1
    for (int i0 = tid; i0 < n; i0 += 4 * kThreads) {
      float4 c[4], s[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kThreads, j = i / quads, e = 4 * (i - j * quads);
        if (i >= n) continue;
        const uint32_t axes = *reinterpret_cast<const uint32_t *>(p.axis + e), a0 = axes & 0xffu;
        auto row = [&](uint32_t axis) { return p.cos_sin + (int64_t)row_of[axis * kTokens + lead0 + j] * p.cs_s0; };
        const float *r = row(a0);
        if (axes == a0 * 0x01010101u) {
          c[u] = __ldg(reinterpret_cast<const float4 *>(r + e));
          s[u] = __ldg(reinterpret_cast<const float4 *>(r + half + e));
        } else {
          const float *r1 = row(axes >> 8 & 0xffu), *r2 = row(axes >> 16 & 0xffu), *r3 = row(axes >> 24);
          c[u] = make_float4(__ldg(r + e), __ldg(r1 + e + 1), __ldg(r2 + e + 2), __ldg(r3 + e + 3));
          s[u] = make_float4(__ldg(r + half + e), __ldg(r1 + half + e + 1), __ldg(r2 + half + e + 2),
                             __ldg(r3 + half + e + 3));
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kThreads, j = i / quads, e = 4 * (i - j * quads);
        if (i >= n) continue;
        float *to = smem + j * p.rot + angle_at(e);
        *reinterpret_cast<float4 *>(to) = c[u];
        *reinterpret_cast<float4 *>(to + half) = s[u];
      }
    }
    __syncthreads();
  }
  const int slot = warp / WU, ut = tid - slot * (32 * WU), ch = ut % LPR, r0 = ut / LPR;
  const int work = n_runs * nu, rounds = (work + SLOTS - 1) / SLOTS;
#pragma unroll 1
  for (int it = 0; it < rounds; ++it) {
    const int e = it * SLOTS + slot;
    const bool on = e < work;
    int run = on ? e / nu : 0;
    const int u = u0 + (on ? e - run * nu : 0);
    int lead, rn;
    uint32_t mask;
    if constexpr (FEW) {
      uint32_t later = begins;
      for (int i = 0; i < run; ++i) later &= later - 1;
      lead = __ffs(later) - 1;
      rn = __shfl_sync(0xffffffffu, n, lead);
      mask = __shfl_sync(0xffffffffu, written, lead);
    } else {
      // (its place: its warp's 16 and its number among them)
      int at = 0;
      while (run >= run_count[at]) run -= run_count[at++];
      at = at * PD_SCALE_TOKENS + run;
      lead = run_lead[at];
      rn = run_n[at];
      mask = run_mask[at];
    }
    const bool is_k = u < p.Hkv;
    const int h = is_k ? u : u - p.Hkv;
    const QuantPool &pool = is_k ? p.kc : p.vc;
    const int first_slot = slot_of[lead];
    const int page = first_slot / p.P, sub = (first_slot - page * p.P) / PD_SCALE_TOKENS;
    float *scale_at = pool.scale + page * pool.s_page + sub * pool.s_blk + h * pool.s_head;
    unsigned char *codes = pool.codes + page * pool.page + (int64_t)(sub * PD_SCALE_TOKENS) * pool.tok + h * pool.head;
    const int64_t row = is_k ? p.k_s0 : p.v_s0;
    const unsigned short *src = is_k ? static_cast<const unsigned short *>(p.k) + (int64_t)h * p.k_s1
                                     : static_cast<const unsigned short *>(p.v) + (int64_t)h * p.v_s1;
    src += (int64_t)(t0 + lead) * row;
    // the chunks' first dims
    const bool pair = NEOX && is_k && 16 * ch < p.rot;
    const int da = pair ? 8 * ch : 16 * ch, db = pair ? 8 * ch + half : 16 * ch + 8;
    // its values in fp32, K's rotated
    float x[NP][2][8];
    float old = 0.f, a = 0.f;
    bool again = false;
    if (on) {
      old = *scale_at;
      uint4 wa[NP], wb[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int j = r0 + RPP * i;
        wa[i] = wb[i] = make_uint4(0u, 0u, 0u, 0u);
        if (j < rn) {
          wa[i] = __ldg(reinterpret_cast<const uint4 *>(src + j * row + da));
          wb[i] = __ldg(reinterpret_cast<const uint4 *>(src + j * row + db));
        }
      }
      // a run whose block one of the tokens before it has is left out: two units would write the block at
      // once (looked at here, while the rows are on their way)
      const uint32_t block = (uint32_t)first_slot & ~(uint32_t)(PD_SCALE_TOKENS - 1);
#pragma unroll
      for (int i = 0; i < kLook; i += 32) again |= (uint32_t)slot_of[lead - 1 - lane - i] - block < PD_SCALE_TOKENS;
      again = __any_sync(0xffffffffu, again);
      if (again && u == 0 && lane == 0) atomicOr(p.status, PD_DEV_BAD_SLOT);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        unpack8<BF16>(wa[i], x[i][0]);
        unpack8<BF16>(wb[i], x[i][1]);
      }
      if (is_k && p.rot > 0) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          if (r0 + RPP * i >= rn) continue;
          const float *cs = smem + (lead - lead0 + r0 + RPP * i) * p.rot + 4 * ch;
          float(&y)[8] = x[i][0], (&z)[8] = x[i][1];
          if constexpr (NEOX) {
            if (!pair) continue;
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
              const float4 co = *reinterpret_cast<const float4 *>(cs + angle_at(e));
              const float4 si = *reinterpret_cast<const float4 *>(cs + half + angle_at(e));
              turn(y[e], z[e], co.x, si.x, y[e], z[e]);
              turn(y[e + 1], z[e + 1], co.y, si.y, y[e + 1], z[e + 1]);
              turn(y[e + 2], z[e + 2], co.z, si.z, y[e + 2], z[e + 2]);
              turn(y[e + 3], z[e + 3], co.w, si.w, y[e + 3], z[e + 3]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (16 * ch + 8 * k >= p.rot) break;
              float(&v)[8] = x[i][k];
              const float4 co = *reinterpret_cast<const float4 *>(cs + angle_at(4 * k));
              const float4 si = *reinterpret_cast<const float4 *>(cs + half + angle_at(4 * k));
              turn(v[0], v[1], co.x, si.x, v[0], v[1]);
              turn(v[2], v[3], co.y, si.y, v[2], v[3]);
              turn(v[4], v[5], co.z, si.z, v[4], v[5]);
              turn(v[6], v[7], co.w, si.w, v[6], v[7]);
            }
          }
        }
      }
      // (fmaxf leaves NaN out)
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) a = fmaxf(a, fmaxf(fabsf(x[i][0][e]), fabsf(x[i][1][e])));
      if (a == INFINITY) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float m = fabsf(x[i][e >> 3][e & 7]);
            a = fmaxf(a, m < INFINITY ? m : 0.f);  // (of finite values)
          }
      }
    }
    uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(a));  // (>= 0: ordered as integers)
    if constexpr (WU > 1) {
      if (lane == 0) top[warp] = __uint_as_float(bits);
      __syncthreads();  // (and every lane has the old scale)
      a = top[slot * WU];
#pragma unroll
      for (int i = 1; i < WU; ++i) a = fmaxf(a, top[slot * WU + i]);
      __syncthreads();
    } else {
      a = __uint_as_float(bits);
    }
    if (!on || again) continue;  // (whole units)
    const float need = least_scale(a);
    const bool had = old > 0.f && old < INFINITY && !(mask & 1u);
    const bool grown = had && need > old;
    const float now = had && !grown ? old : need;
    const bool pow2 = power_of_two(now);
    const float inv = 1.f / now;
    if (!pow2) {
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[i][e >> 3][e & 7] = over_marked(x[i][e >> 3][e & 7], now);
    }
    const float by = pow2 ? inv : 1.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int j = r0 + RPP * i;
      if (j >= rn) continue;
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float *v = &x[i][k >> 1][(k & 1) * 4];
        c[k] = codes4(v[0] * by, v[1] * by, v[2] * by, v[3] * by);
      }
      unsigned char *to = codes + (slot_of[lead + j] & 15) * pool.tok;
      if (pair) {
        *reinterpret_cast<uint2 *>(to + da) = make_uint2(c[0], c[1]);
        *reinterpret_cast<uint2 *>(to + db) = make_uint2(c[2], c[3]);
      } else {
        *reinterpret_cast<uint4 *>(to + da) = make_uint4(c[0], c[1], c[2], c[3]);
      }
    }
    if (grown) {
      // the block's other codes, to the new scale (a power of two: the ratio is exact, or too small to count)
      const float ratio = __fdiv_rn(old, now);
#pragma unroll 1
      for (int i = 0; i < NP; ++i) {
        const int off = r0 + RPP * i;
        if (mask >> off & 1u) continue;
        uint4 *at = reinterpret_cast<uint4 *>(codes + off * pool.tok + 16 * ch);
        uint4 w = *at;
        uint32_t *words[4] = {&w.x, &w.y, &w.z, &w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float y[4];
          floats4(*words[k], y);
          *words[k] = codes4(times_marked(y[0], ratio), times_marked(y[1], ratio), times_marked(y[2], ratio),
                             times_marked(y[3], ratio));
        }
        *at = w;
      }
    }
    __syncwarp();  // (every lane has the old scale)
    if (ut == 0 && now != old) *scale_at = now;
  }
}

template <int D, bool BF16, bool NEOX, bool FEW>
__global__ void __launch_bounds__(kThreads, FEW ? 1 : kCtas) pd_quant_write(const __grid_constant__ QuantWriteParams p) {
  extern __shared__ __align__(16) float smem_f[];
  grid_dependency_wait();
  grid_dependents_launch();
  const int b = blockIdx.x;
  if (b < p.kv_ctas)
    kv_runs<D, BF16, NEOX, FEW>(p, b, smem_f);
  else
    q_tokens<D, BF16, NEOX, FEW ? 4 : 2>(p, (b - p.kv_ctas) << (kLgThreads - p.lg_group), p.lg_group, smem_f);
}

template <int D>
cudaError_t launch_write(const QuantWriteParams &p, bool bf16, bool neox, bool few, int ctas, int smem,
                         cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  auto go = [&](auto kern, SmemLimit &limit) {
    const cudaError_t e = allow_smem(limit, kern, smem);
    return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kern, p) : e;
  };
  static SmemLimit limits[8];
  const int which = (bf16 ? 4 : 0) + (neox ? 2 : 0) + (few ? 1 : 0);
  switch (which) {
    case 0: return go(pd_quant_write<D, false, false, false>, limits[0]);
    case 1: return go(pd_quant_write<D, false, false, true>, limits[1]);
    case 2: return go(pd_quant_write<D, false, true, false>, limits[2]);
    case 3: return go(pd_quant_write<D, false, true, true>, limits[3]);
    case 4: return go(pd_quant_write<D, true, false, false>, limits[4]);
    case 5: return go(pd_quant_write<D, true, false, true>, limits[5]);
    case 6: return go(pd_quant_write<D, true, true, false>, limits[6]);
    default: return go(pd_quant_write<D, true, true, true>, limits[7]);
  }
}

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" PD_API int paged_rope_quant_cache_write(
    const pd_tensor *q, const pd_tensor *k, const pd_tensor *v, const pd_tensor *positions,
    const pd_tensor *slot_mapping, const pd_tensor *cos_sin_cache, const uint8_t *pair_axis,
    pd_tensor *q_out, pd_tensor *k_cache, pd_tensor *v_cache, pd_tensor *k_scale, pd_tensor *v_scale,
    int num_q_heads, int num_kv_heads, int head_size, int rot_dim, int page_size, int layout,
    int is_neox, void *stream) {
  if (!k || !v || !slot_mapping || !k_cache || !v_cache || !k_scale || !v_scale || !q != !q_out)
    return PD_EINVAL;
  if (num_kv_heads <= 0 || (q && num_q_heads <= 0)) return PD_EINVAL;
  if (head_size != 64 && head_size != 128 && head_size != 256 && head_size != 512) return PD_EHEAD;
  if (page_size <= 0 || page_size % PD_SCALE_TOKENS != 0 || (layout != PD_NHD && layout != PD_HND))
    return PD_EINVAL;
  if (rot_dim < 0 || rot_dim > head_size || rot_dim % (is_neox ? 16 : 8) != 0) return PD_EINVAL;
  if ((rot_dim > 0) != (positions != nullptr) || (rot_dim > 0) != (cos_sin_cache != nullptr))
    return PD_EINVAL;
  if (k->ndim != 3 || k->shape[0] < 0 || k->shape[0] > INT32_MAX / 2) return PD_EINVAL;
  const int64_t T = k->shape[0];
  int rc;
  if ((rc = check_token_rows(k, T, num_kv_heads, head_size)) != PD_OK) return rc;
  if ((rc = check_token_rows(v, T, num_kv_heads, head_size)) != PD_OK) return rc;
  if (k->dtype != v->dtype) return PD_EDTYPE;
  QuantWriteParams p{};
  if (q) {
    if ((rc = check_token_rows(q, T, num_q_heads, head_size)) != PD_OK) return rc;
    if ((rc = check_token_rows(q_out, T, num_q_heads, head_size)) != PD_OK) return rc;
    if (q->dtype != k->dtype || q_out->dtype != k->dtype) return PD_EDTYPE;
    p.q = q->data;
    p.q_s0 = q->stride[0];
    p.q_s1 = q->stride[1];
    p.q_out = q_out->data;
    p.qo_s0 = q_out->stride[0];
    p.qo_s1 = q_out->stride[1];
    p.Hq = num_q_heads;
  }
  if ((rc = check_i32_vector(slot_mapping, T)) != PD_OK) return rc;
  if (rot_dim > 0) {
    const pd_tensor *ps = positions, *cs = cos_sin_cache;
    if (ps->ndim != 1 && ps->ndim != 2) return PD_EINVAL;
    const int at = ps->ndim - 1;
    const int64_t axes = at ? ps->shape[0] : 1;
    if (axes < 1 || axes > PD_MAX_AXES || ps->shape[at] != T || (!ps->data && T != 0)) return PD_EINVAL;
    if (ps->dtype != PD_I32) return PD_EDTYPE;
    if (T > 1 && ps->stride[at] != 1) return PD_EALIGN;
    if (at && ps->stride[0] < 0) return PD_EINVAL;
    if (!cs->data || cs->ndim != 2 || cs->shape[0] < 1 || cs->shape[0] > INT32_MAX ||
        cs->shape[1] < rot_dim || cs->stride[1] != 1 || cs->stride[0] < rot_dim)
      return PD_EINVAL;
    if (cs->dtype != PD_F32) return PD_EDTYPE;
    if (cs->stride[0] % 4 != 0 || !aligned16(cs->data)) return PD_EALIGN;
    for (int i = 0; i < rot_dim / 2; ++i) {
      if (pair_axis && pair_axis[i] >= axes) return PD_EINVAL;
      p.axis[i] = pair_axis ? pair_axis[i] : 0;
    }
    p.positions = static_cast<const int32_t *>(ps->data);
    p.pos_stride = at ? ps->stride[0] : 0;
    p.axes = (int)axes;
    p.cos_sin = static_cast<const float *>(cs->data);
    p.cs_s0 = cs->stride[0];
    p.max_pos = (int)cs->shape[0];
  }
  if ((rc = quant_pool(k_cache, k_scale, layout, num_kv_heads, page_size, head_size, &p.kc)) != PD_OK)
    return rc;
  if ((rc = quant_pool(v_cache, v_scale, layout, num_kv_heads, page_size, head_size, &p.vc)) != PD_OK)
    return rc;
  if (k_cache->shape[0] != v_cache->shape[0]) return PD_EINVAL;
  if (T == 0) return PD_OK;
  int num_sms = 0;
  if ((rc = device_check(&num_sms, &p.status)) != PD_OK) return rc;
  p.k = k->data;
  p.k_s0 = k->stride[0];
  p.k_s1 = k->stride[1];
  p.v = v->data;
  p.v_s0 = v->stride[0];
  p.v_s1 = v->stride[1];
  p.slots = static_cast<const int32_t *>(slot_mapping->data);
  p.T = (int)T;
  p.Hkv = num_kv_heads;
  p.rot = rot_dim;
  p.P = page_size;
  p.num_slots = k_cache->shape[0] * (int64_t)page_size;
  const bool few = T * 4 < (int64_t)num_sms * 32;
  // Tokens of a k/v CTA, and units: one round of units, and as few tokens as leave at most 10 CTAs
  // an SM, up to a block's 16, or with few heads as many as make two rounds of units, and up to what
  // the angles (of them and 15 more) find room for, five CTAs an SM.  Where those are still more CTAs,
  // K (or V) of all heads, whose slots and angles are read once.  (110,000 tokens of prompts, 8 / 1
  // heads of 128: 122 us with 16 tokens, 112 with 64; 900 of prompts, 32 / 8 heads of 512: 34 us with 2
  // tokens and 8 units, 23 with 16 and one.)
  const int slots = head_size > 256 ? 1 : head_size > 128 ? 2 : 4;  // units of a CTA at a time
  const int64_t ctas_most = 10LL * num_sms;
  p.units = slots;
  auto slices = [&] { return (2 * num_kv_heads + p.units - 1) / p.units; };
  auto windows = [&] { return (T + p.window - 1) / p.window; };
  for (p.window = 1; p.window < (few ? PD_SCALE_TOKENS : kWindow) && windows() * slices() > ctas_most; p.window *= 2) {
    if (p.window >= PD_SCALE_TOKENS && p.window / PD_SCALE_TOKENS * num_kv_heads >= slots) break;
    if ((2 * p.window + PD_SCALE_TOKENS - 1) * rot_dim * 4 > kAngleBytes) break;
  }
  if (windows() * slices() > ctas_most) p.units = (num_kv_heads + slots - 1) / slots * slots;
  p.slices = slices();
  // Threads of a token of q: all while tokens are few, else as many as have 8 chunks of 16 bytes
  // each, from 8 to 64, and 4 CTAs an SM (131,072 tokens, 8 / 1 heads of 128: 224 us with 64, 147
  // with 16).
  p.lg_group = kLgThreads;
  while (!few && p.lg_group > 3 && (p.lg_group == kLgThreads || (int64_t)num_q_heads * head_size < 64 << p.lg_group) &&
         T << p.lg_group > (int64_t)num_sms * 4 * kThreads)
    --p.lg_group;
  const int64_t q_ctas = q ? ((T << p.lg_group) + kThreads - 1) >> kLgThreads : 0;
  if (windows() * p.slices + q_ctas > INT32_MAX) return PD_EINVAL;
  p.kv_ctas = (int)(windows() * p.slices);
  const int ctas = p.kv_ctas + (int)q_ctas;
  const int smem = (p.window + PD_SCALE_TOKENS - 1) * rot_dim * 4;
  const bool bf16 = k->dtype == PD_BF16;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  switch (head_size) {
    case 64: e = launch_write<64>(p, bf16, is_neox, few, ctas, smem, st); break;
    case 128: e = launch_write<128>(p, bf16, is_neox, few, ctas, smem, st); break;
    case 256: e = launch_write<256>(p, bf16, is_neox, few, ctas, smem, st); break;
    case 512: e = launch_write<512>(p, bf16, is_neox, few, ctas, smem, st); break;
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return PD_ECUDA;
  }
  return PD_OK;
}
