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

}  // namespace pd
