// 8-bit floats: codes to and from 32- and 16-bit floats.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace pd {

// Four e4m3 codes of fp32 values: the nearest, ties to even, 448 at most.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Four e4m3 codes as halves: bytes 0, 1 and bytes 2, 3.
__device__ __forceinline__ void halves_of(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Four e4m3 codes as fp32.
__device__ __forceinline__ void floats4(uint32_t w, float (&x)[4]) {
  uint32_t lo, hi;
  halves_of(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

// Products and quotients that are rounded again, to 16 or 8 bits: towards zero, and the last bit set
// where something was cut off.  A value so marked lies on the exact one's side of every number of two
// bits less, so that the second rounding gives what the exact value would (of results that are
// normal in fp32, and of infinities and NaN).
__device__ __forceinline__ float marked(float x, float cut) {
  return cut != 0.f && fabsf(x) < INFINITY ? __uint_as_float(__float_as_uint(x) | 1u) : x;
}
__device__ __forceinline__ float times_marked(float a, float b) {
  const float x = __fmul_rz(a, b);
  return marked(x, fmaf(a, b, -x));  // (what was cut off is a float)
}
__device__ __forceinline__ float over_marked(float a, float b) {
  const float x = __fdiv_rz(a, b);
  return marked(x, fmaf(-x, b, a));  // (so is the remainder)
}

__device__ __forceinline__ bool power_of_two(float x) { return (__float_as_uint(x) & 0x7fffffu) == 0; }

}  // namespace pd
