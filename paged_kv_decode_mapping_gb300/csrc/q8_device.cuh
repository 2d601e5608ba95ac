// q8_device.cuh -- device pieces of the 8-bit cache: codes to numbers and back.
//
// A code is an int8 or an e4m3 float (PKV_Q8_*).  Both are exact in fp16, so the attention
// kernel's products take them as fp16 with an fp32 accumulator and the scales apply outside.
#pragma once

#include "pkv_internal.h"

namespace pkv {
namespace q8 {

// The 8-bit cache's kernels are launched while the one ahead of them in the stream may still run,
// and begin by waiting for its end: their launch and its end overlap (calls one after another, 16
// contexts of 2048 keys: a decode every 13.1 us instead of 14.8; 256 contexts 41.1 instead of 43.3).
__device__ __forceinline__ void await_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// So what earlier kernels write may change in this one's lifetime, before the wait: plain loads, not the
// ones for memory that is read-only (which may be moved up).
template <typename T>
__device__ __forceinline__ T ld(const T *p) { return *p; }
// From here on the kernel behind this one may be launched; await_stream() first, unless what that one
// reads before its own await_stream() is older than both.
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) (void)cudaGetLastError();  // (handed on, not left behind)
  return e;
}

// n / d for n >= 0, d > 0, by 32 bits where that is enough (a 64-bit division takes 0.2 us).
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  if (((n | d) >> 32) == 0) return (uint32_t)n / (uint32_t)d;
  return n / d;
}

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

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
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
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
  }
}

// Two products rounded once each (a packed instruction), and with an addend.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(uint64_t x) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(x));
  return f;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The codes of x / s for bf16 x, as fp32 division gives them, mostly without one.  x times either
// bound of 1 / s brackets the quotient (below 2^-21 of it apart either way, its own rounding
// included); where both round to one code, that is its code, since rounding is monotone.  Only
// quotients next to a border between two codes are divided.  (Eight divisions a vector were most
// of the write's 57 million instructions: 34000 tokens of 8 heads of 128 took 69 us.)
struct Inverse {
  float s;
  uint64_t lo, hi;  // twice each
};
__device__ __forceinline__ Inverse inverse_of(float s) {
  const float inv = __fdiv_rn(1.f, s);
  // (an infinite one, of a scale that is no normal number, leaves every quotient to the division)
  const float lo = isinf(inv) ? 0.f : inv * (1.f - 4.76837158e-7f), hi = inv * (1.f + 4.76837158e-7f);
  return {s, f32x2(lo, lo), f32x2(hi, hi)};
}
template <int KIND>
__device__ __forceinline__ uint2 divided8(const uint4 &v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float q[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    q[2 * k] = __fdiv_rn(dev::bf16lo_to_f32(w[k]), s);
    q[2 * k + 1] = __fdiv_rn(dev::bf16hi_to_f32(w[k]), s);
  }
  return make_uint2(encode4<KIND>(q[0], q[1], q[2], q[3]), encode4<KIND>(q[4], q[5], q[6], q[7]));
}
// *sure: whether both bounds give these codes; else divided8 is wanted.
template <int KIND>
__device__ __forceinline__ uint2 encode8(const uint4 &v, const Inverse &s, bool *sure) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[2], differ = 0u;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint64_t x = f32x2(dev::bf16lo_to_f32(w[2 * k]), dev::bf16hi_to_f32(w[2 * k]));
    const uint64_t y = f32x2(dev::bf16lo_to_f32(w[2 * k + 1]), dev::bf16hi_to_f32(w[2 * k + 1]));
    if constexpr (KIND == PKV_Q8_INT8) {
      // 2^23 + 2^22 + x / s, whose last bits are the rounded whole number (of at most 127)
      const uint64_t magic = f32x2(12582912.f, 12582912.f);
      const float2 a = split(fma2(x, s.lo, magic)), b = split(fma2(x, s.hi, magic));
      const float2 d = split(fma2(y, s.lo, magic)), e = split(fma2(y, s.hi, magic));
      differ |= __float_as_uint(a.x) ^ __float_as_uint(b.x);
      differ |= __float_as_uint(a.y) ^ __float_as_uint(b.y);
      differ |= __float_as_uint(d.x) ^ __float_as_uint(e.x);
      differ |= __float_as_uint(d.y) ^ __float_as_uint(e.y);
      c[k] = __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),  // low bytes
                         __byte_perm(__float_as_uint(d.x), __float_as_uint(d.y), 0x0040), 0x5410);
    } else {
      const float2 a = split(mul2(x, s.lo)), b = split(mul2(x, s.hi));
      const float2 d = split(mul2(y, s.lo)), e = split(mul2(y, s.hi));
      c[k] = encode4<KIND>(a.x, a.y, d.x, d.y);
      differ |= c[k] ^ encode4<KIND>(b.x, b.y, e.x, e.y);
    }
  }
  *sure = differ == 0u;
  return make_uint2(c[0], c[1]);
}

}  // namespace q8
}  // namespace pkv
