// q8_device.cuh -- device pieces of the 8-bit cache: codes to numbers and back.
//
// A code is an int8 or an e4m3 float (PKV_Q8_*).  Both are exact in fp16, so the attention
// kernel's products take them as fp16 with an fp32 accumulator and the scales apply outside.
#pragma once

#include "pkv_internal.h"

namespace pkv {
namespace q8 {

template <int KIND>
__host__ __device__ constexpr float top() { return KIND == PKV_Q8_INT8 ? 127.f : 448.f; }

// What `prep` makes of four codes, `pair` turns into fp16 two at a time: bytes 0, 1 (HI = 0) or
// 2, 3 (HI = 1).  int8: with the sign bit flipped a code is u = c + 128; behind the byte 0x64 it
// is the fp16 1024 + u, and 1024 + u - 1152 = c, exactly.
template <int KIND>
__device__ __forceinline__ uint32_t prep(uint32_t w) {
  return KIND == PKV_Q8_INT8 ? w ^ 0x80808080u : w;
}
template <int KIND, int HI>
__device__ __forceinline__ uint32_t pair(uint32_t w) {
  uint32_t r;
  if constexpr (KIND == PKV_Q8_INT8) {
    const uint32_t x = __byte_perm(w, 0x64646464u, HI ? 0x4342 : 0x4140);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x64806480u));
  } else {
    const uint16_t h = (uint16_t)(HI ? w >> 16 : w & 0xffffu);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  }
  return r;
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Four values in units of the scale, rounded to the nearest code (halves to even, larger ones to
// the largest code).  NaN: e4m3's NaN, int8's 0.
template <int KIND>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if constexpr (KIND == PKV_Q8_INT8) {
    auto one = [](float x) { return (uint32_t)(__float2int_rn(fminf(fmaxf(x, -127.f), 127.f)) & 0xff); };
    return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | (uint32_t)hi << 16;
  }
}

}  // namespace q8
}  // namespace pkv
