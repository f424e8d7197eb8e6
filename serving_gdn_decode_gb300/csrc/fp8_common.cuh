// e4m3 codes on the device: pairs of codes from and to f16 and f32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

// Codes i and i + 1 of a word (i = 0 or 2) as two f16, exactly (e4m3 is a part of f16; NaN stays NaN).
__device__ __forceinline__ unsigned codes_f16x2(unsigned word, int i) {
  unsigned y;
  const unsigned short pair = static_cast<unsigned short>(i ? word >> 16 : word);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(y) : "h"(pair));
  return y;
}

__device__ __forceinline__ float2 codes_f32x2(unsigned word, int i) {
  const unsigned y = codes_f16x2(word, i);
  return __half22float2(*reinterpret_cast<const __half2 *>(&y));
}

// Four values as codes, each rounded to nearest, ties to even; above 448 they are 448, NaN is NaN.
__device__ __forceinline__ unsigned codes_of(float a, float b, float c, float d) {
  unsigned short lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(d), "f"(c));
  return lo | static_cast<unsigned>(hi) << 16;
}

}  // namespace gdn
