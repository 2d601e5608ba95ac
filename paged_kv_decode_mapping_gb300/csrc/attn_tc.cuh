// attn_tc.cuh -- device pieces of the attention kernels on the 5th-generation tensor cores
// (paged prefill, packed prompts, shared prefixes): the softmax threads' work on one
// 128-key block of a score row in TMEM, and the straight-line issue of the MMAs.
#pragma once

#include "attn_device.cuh"
#include "pkv_exp2.cuh"

// Of the 16 column pairs of each 32-column chunk of a score row, how many take their
// exponentials on the FMA pipe (exp2_fma) rather than the special-function unit, in
// row_block_exp and in the one-pass weights.  0: every fraction tried measured slower
// (2 pairs: -4 to -6%, 4 pairs: -8 to -15% on the four prefill workloads): the softmax
// waits on latency and issue, not on the special-function unit.
#ifndef PKV_PREFILL_POLY_PAIRS
#define PKV_PREFILL_POLY_PAIRS 0
#endif
// Row maxima with three-input max instructions (1) or two-input ones (0).
#ifndef PKV_PREFILL_MAX3
#define PKV_PREFILL_MAX3 1
#endif
// Scaled, max-subtracted scores two at a time with packed fp32 FMAs (1) or one at a time (0).
#ifndef PKV_PREFILL_FMA2
#define PKV_PREFILL_FMA2 1
#endif
// Row sums of the bf16 weights with mixed-precision adds (1) or widen-then-add (0).
#ifndef PKV_PREFILL_SUM_MIXED
#define PKV_PREFILL_SUM_MIXED 1
#endif

namespace pkv {

constexpr int kTcRows = kTileRows;
constexpr int kTcKeys = kTileKeys;
// A row's reference max moves only when a block raises it by more than this (base 2).
constexpr float kTcRescale = 8.f;

// ---------------------------------------------------------------------------
// The softmax warps' work on one 128-column block of a score row in TMEM (one thread =
// one row = one TMEM lane).  TMEM is read in 32-column chunks with the next chunk's load
// in flight while the current one is processed.

// Waits for this thread's TMEM loads; the 32 registers the last one fills are tied to
// the wait, so that nothing reads them before it.
__device__ __forceinline__ void tmem_wait_ld_regs(uint32_t (&x)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]),
                 "+r"(x[6]), "+r"(x[7]), "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]),
                 "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15]), "+r"(x[16]), "+r"(x[17]),
                 "+r"(x[18]), "+r"(x[19]), "+r"(x[20]), "+r"(x[21]), "+r"(x[22]), "+r"(x[23]),
                 "+r"(x[24]), "+r"(x[25]), "+r"(x[26]), "+r"(x[27]), "+r"(x[28]), "+r"(x[29]),
                 "+r"(x[30]), "+r"(x[31])
               :
               : "memory");
}

// c + lo(x) + hi(x) for a bf16 pair x: two mixed-precision adds (bf16 + fp32).
__device__ __forceinline__ float add_bf16x2(uint32_t x, float c) {
  float d;
  asm("{\n\t.reg .b16 lo, hi;\n\t.reg .f32 t;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "add.rn.f32.bf16 t, lo, %2;\n\tadd.rn.f32.bf16 %0, hi, t;\n\t}"
      : "=f"(d)
      : "r"(x), "f"(c));
  return d;
}

// (x0, x1) * s + c, both lanes rounded once (fused), in one packed instruction.
__device__ __forceinline__ void fma_f32x2(float x0, float x1, float s, float c, float &d0,
                                          float &d1) {
  asm("{\n\t.reg .b64 x, sc, cc, d;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 sc, {%4, %4};\n\tmov.b64 cc, {%5, %5};\n\t"
      "fma.rn.f32x2 d, x, sc, cc;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(x0), "f"(x1), "f"(s), "f"(c));
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One 32-bit TMEM column of this thread's lane (load: complete with a wait).
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t x;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(taddr));
  return x;
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(x) : "memory");
}

// Pass 1: the row's maximum scaled score over the columns c <= lim (all of them when
// `whole`) of NCH 32-column chunks starting at chunk ch0.  With a positive scale, the
// max of the raw scores scaled once equals the max of the scaled scores (rounding is
// monotonic).
template <int NCH>
__device__ __forceinline__ float row_block_max(uint32_t sb, int ch0, int lim, bool whole,
                                               bool pos_scale, float scale_log2) {
  float mx[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) mx[u] = -INFINITY;
  const float sc = pos_scale ? 1.f : scale_log2;
  uint32_t xa[32], xb[32];
  dev::tmem_ld32(sb + ch0 * 32, xa);
  tmem_wait_ld_regs(xa);
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    uint32_t(&cur)[32] = (ch & 1) ? xb : xa;
    uint32_t(&nxt)[32] = (ch & 1) ? xa : xb;
    if (ch + 1 < NCH) dev::tmem_ld32(sb + (ch0 + ch + 1) * 32, nxt);
    const int lc = lim - (ch0 + ch) * 32;
    if (whole && pos_scale) {
#if PKV_PREFILL_MAX3
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        mx[(i >> 1) & 7] = fmax3(mx[(i >> 1) & 7], __uint_as_float(cur[i]), __uint_as_float(cur[i + 1]));
#else
#pragma unroll
      for (int i = 0; i < 32; ++i) mx[i & 7] = fmaxf(mx[i & 7], __uint_as_float(cur[i]));
#endif
    } else if (whole) {
#pragma unroll
      for (int i = 0; i < 32; ++i) mx[i & 7] = fmaxf(mx[i & 7], __uint_as_float(cur[i]) * sc);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        mx[i & 7] = fmaxf(mx[i & 7], i <= lc ? __uint_as_float(cur[i]) * sc : -INFINITY);
    }
    if (ch + 1 < NCH) tmem_wait_ld_regs(nxt);
  }
  float bmax = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                     fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
  return pos_scale ? bmax * scale_log2 : bmax;
}

// Pass 2: P = exp2(S * scale - m_ref) for the columns c <= lim (0 past it) of NCH
// 32-column chunks starting at chunk ch0, rounded to bf16 and stored into row r of the
// P buffer at shared offset `prow` (K-major, 128-byte swizzle: two 64-column sub-tiles
// `sub` bytes apart); returns the sum of the rounded values, which is what the tensor
// cores multiply.  The first PKV_PREFILL_POLY_PAIRS column pairs of each chunk take
// exp2_fma.
template <int NCH, bool kSum = true>
__device__ __forceinline__ float row_block_exp(uint32_t sb, int ch0, uint8_t *bp, uint32_t prow,
                                               uint32_t sub, int r, int lim, bool whole,
                                               float scale_log2, float m_ref) {
  float ls[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) ls[u] = 0.f;
  uint32_t xa[32], xb[32];
  dev::tmem_ld32(sb + ch0 * 32, xa);
  tmem_wait_ld_regs(xa);
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    uint32_t(&cur)[32] = (ch & 1) ? xb : xa;
    uint32_t(&nxt)[32] = (ch & 1) ? xa : xb;
    if (ch + 1 < NCH) dev::tmem_ld32(sb + (ch0 + ch + 1) * 32, nxt);
    const int cha = ch0 + ch;  // absolute chunk
    const int lc = whole ? 32 : lim - cha * 32;
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#if PKV_PREFILL_FMA2
      float a0, a1;
      fma_f32x2(__uint_as_float(cur[2 * e]), __uint_as_float(cur[2 * e + 1]), scale_log2, -m_ref,
                a0, a1);
#else
      const float a0 = fmaf(__uint_as_float(cur[2 * e]), scale_log2, -m_ref);
      const float a1 = fmaf(__uint_as_float(cur[2 * e + 1]), scale_log2, -m_ref);
#endif
      float p0, p1;
      if (e < PKV_PREFILL_POLY_PAIRS) {
        p0 = dev::exp2_fma(a0);
        p1 = dev::exp2_fma(a1);
      } else {
        p0 = dev::ex2(a0);
        p1 = dev::ex2(a1);
      }
      if (!whole) {
        p0 = 2 * e <= lc ? p0 : 0.f;
        p1 = 2 * e + 1 <= lc ? p1 : 0.f;
      }
      pk[e] = dev::pack_bf16x2(p0, p1);
      // sum what the tensor cores multiply: with a stale reference max the largest P is
      // not a power of two, and only this keeps the weights a convex combination
      if constexpr (kSum) {
#if PKV_PREFILL_SUM_MIXED
        ls[e & 7] = add_bf16x2(pk[e], ls[e & 7]);
#else
        ls[(2 * e) & 7] += dev::bf16lo_to_f32(pk[e]);
        ls[(2 * e + 1) & 7] += dev::bf16hi_to_f32(pk[e]);
#endif
      }
    }
    const uint32_t dst = prow + (cha >> 1) * sub;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c16 = (cha & 1) * 4 + u;
      *reinterpret_cast<uint4 *>(bp + dst + ((c16 ^ (r & 7)) << 4)) =
          make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
    }
    if (ch + 1 < NCH) tmem_wait_ld_regs(nxt);
  }
  return ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
}

// The same two passes from one read of the row's chunks into registers (TMEM is read
// once per block instead of twice).
template <int NCH>
__device__ __forceinline__ void row_block_load(uint32_t sb, int ch0, uint32_t (&x)[NCH * 32]) {
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    uint32_t(&c)[32] = *reinterpret_cast<uint32_t(*)[32]>(&x[ch * 32]);
    dev::tmem_ld32(sb + (ch0 + ch) * 32, c);
  }
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    uint32_t(&c)[32] = *reinterpret_cast<uint32_t(*)[32]>(&x[ch * 32]);
    if (ch == 0)
      tmem_wait_ld_regs(c);  // one wait covers every load above
    else
      asm volatile("" : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]), "+r"(c[4]), "+r"(c[5]),
                   "+r"(c[6]), "+r"(c[7]), "+r"(c[8]), "+r"(c[9]), "+r"(c[10]), "+r"(c[11]),
                   "+r"(c[12]), "+r"(c[13]), "+r"(c[14]), "+r"(c[15]), "+r"(c[16]), "+r"(c[17]),
                   "+r"(c[18]), "+r"(c[19]), "+r"(c[20]), "+r"(c[21]), "+r"(c[22]), "+r"(c[23]),
                   "+r"(c[24]), "+r"(c[25]), "+r"(c[26]), "+r"(c[27]), "+r"(c[28]), "+r"(c[29]),
                   "+r"(c[30]), "+r"(c[31]));
  }
}

template <int NCH>
__device__ __forceinline__ float row_regs_max(const uint32_t (&x)[NCH * 32], int ch0, int lim,
                                              bool whole, bool pos_scale, float scale_log2) {
  float mx[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) mx[u] = -INFINITY;
  const float sc = pos_scale ? 1.f : scale_log2;
  if (whole && pos_scale) {
#pragma unroll
    for (int i = 0; i < NCH * 32; i += 2)
      mx[(i >> 1) & 7] = fmax3(mx[(i >> 1) & 7], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
  } else if (whole) {
#pragma unroll
    for (int i = 0; i < NCH * 32; ++i) mx[i & 7] = fmaxf(mx[i & 7], __uint_as_float(x[i]) * sc);
  } else {
    const int lc = lim - ch0 * 32;
#pragma unroll
    for (int i = 0; i < NCH * 32; ++i)
      mx[i & 7] = fmaxf(mx[i & 7], i <= lc ? __uint_as_float(x[i]) * sc : -INFINITY);
  }
  const float bmax = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                           fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
  return pos_scale ? bmax * scale_log2 : bmax;
}

template <int NCH>
__device__ __forceinline__ float row_regs_exp(const uint32_t (&x)[NCH * 32], int ch0, uint8_t *bp,
                                              uint32_t prow, uint32_t sub, int r, int lim,
                                              bool whole, float scale_log2, float m_ref) {
  float ls[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) ls[u] = 0.f;
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    const int cha = ch0 + ch;
    const int lc = whole ? 32 : lim - cha * 32;
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float a0, a1;
      fma_f32x2(__uint_as_float(x[ch * 32 + 2 * e]), __uint_as_float(x[ch * 32 + 2 * e + 1]),
                scale_log2, -m_ref, a0, a1);
      float p0 = dev::ex2(a0), p1 = dev::ex2(a1);
      if (!whole) {
        p0 = 2 * e <= lc ? p0 : 0.f;
        p1 = 2 * e + 1 <= lc ? p1 : 0.f;
      }
      pk[e] = dev::pack_bf16x2(p0, p1);
      ls[e & 7] = add_bf16x2(pk[e], ls[e & 7]);
    }
    const uint32_t dst = prow + (cha >> 1) * sub;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c16 = (cha & 1) * 4 + u;
      *reinterpret_cast<uint4 *>(bp + dst + ((c16 ^ (r & 7)) << 4)) =
          make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
    }
  }
  return ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
}

// Pass 2 from registers, without the stores: the rounded weights stay packed in `pk`
// (column pair e of chunk ch at pk[16 ch + e]) until the P buffer is free; returns their
// sum, as row_regs_exp.
template <int NCH, bool kSum = true>
__device__ __forceinline__ float row_regs_exp_pk(const uint32_t (&x)[NCH * 32], int ch0, int lim,
                                                 bool whole, float scale_log2, float m_ref,
                                                 uint32_t (&pk)[NCH * 16]) {
  float ls[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) ls[u] = 0.f;
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    const int lc = whole ? 32 : lim - (ch0 + ch) * 32;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float a0, a1;
      fma_f32x2(__uint_as_float(x[ch * 32 + 2 * e]), __uint_as_float(x[ch * 32 + 2 * e + 1]),
                scale_log2, -m_ref, a0, a1);
      float p0 = dev::ex2(a0), p1 = dev::ex2(a1);
      if (!whole) {
        p0 = 2 * e <= lc ? p0 : 0.f;
        p1 = 2 * e + 1 <= lc ? p1 : 0.f;
      }
      pk[ch * 16 + e] = dev::pack_bf16x2(p0, p1);
      if constexpr (kSum) ls[e & 7] = add_bf16x2(pk[ch * 16 + e], ls[e & 7]);
    }
  }
  return ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
}

// The body of row_regs_exp_pk_max for one masking mode, the running maxima in mx.
template <int NCH, bool kSum, int kMode>  // kMode 0: whole, positive scale; 1: whole; 2: masked
__device__ __forceinline__ float row_regs_exp_pk_max_impl(const uint32_t (&x)[NCH * 32], int ch0,
                                                          int lim, float sc, float scale_log2,
                                                          float m_ref, uint32_t (&pk)[NCH * 16],
                                                          float (&mx)[8]) {
  float ls[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) ls[u] = 0.f;
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    const int lc = kMode == 2 ? lim - (ch0 + ch) * 32 : 32;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float x0 = __uint_as_float(x[ch * 32 + 2 * e]), x1 = __uint_as_float(x[ch * 32 + 2 * e + 1]);
      if constexpr (kMode == 0)
        mx[e & 7] = fmax3(mx[e & 7], x0, x1);
      else if constexpr (kMode == 1)
        mx[e & 7] = fmax3(mx[e & 7], x0 * sc, x1 * sc);
      else
        mx[e & 7] = fmax3(mx[e & 7], 2 * e <= lc ? x0 * sc : -INFINITY,
                          2 * e + 1 <= lc ? x1 * sc : -INFINITY);
      float a0, a1;
      fma_f32x2(x0, x1, scale_log2, -m_ref, a0, a1);
      float p0, p1;
      if (e < PKV_PREFILL_POLY_PAIRS) {
        p0 = dev::exp2_fma(a0);
        p1 = dev::exp2_fma(a1);
      } else {
        p0 = dev::ex2(a0);
        p1 = dev::ex2(a1);
      }
      if constexpr (kMode == 2) {
        p0 = 2 * e <= lc ? p0 : 0.f;
        p1 = 2 * e + 1 <= lc ? p1 : 0.f;
      }
      pk[ch * 16 + e] = dev::pack_bf16x2(p0, p1);
      if constexpr (kSum) ls[e & 7] = add_bf16x2(pk[ch * 16 + e], ls[e & 7]);
    }
  }
  return ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
}

// row_regs_exp_pk and row_regs_max in one pass: the weights against a reference m_ref
// taken before the block's max is known, and that max (as row_regs_max returns it) in
// *bmax.  Weights of columns far above m_ref may overflow; the caller recomputes them
// once the max says the reference must move.
template <int NCH, bool kSum = true>
__device__ __forceinline__ float row_regs_exp_pk_max(const uint32_t (&x)[NCH * 32], int ch0, int lim,
                                                     bool whole, bool pos_scale, float scale_log2,
                                                     float m_ref, uint32_t (&pk)[NCH * 16],
                                                     float *bmax) {
  float mx[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) mx[u] = -INFINITY;
  const float sc = pos_scale ? 1.f : scale_log2;
  float ls;
  if (whole && pos_scale)
    ls = row_regs_exp_pk_max_impl<NCH, kSum, 0>(x, ch0, lim, sc, scale_log2, m_ref, pk, mx);
  else if (whole)
    ls = row_regs_exp_pk_max_impl<NCH, kSum, 1>(x, ch0, lim, sc, scale_log2, m_ref, pk, mx);
  else
    ls = row_regs_exp_pk_max_impl<NCH, kSum, 2>(x, ch0, lim, sc, scale_log2, m_ref, pk, mx);
  const float m = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                        fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
  *bmax = pos_scale ? m * scale_log2 : m;
  return ls;
}

// Stores the packed weights of row_regs_exp_pk into row r of the P buffer (K-major,
// 128-byte swizzle, two 64-column sub-tiles `sub` bytes apart).
template <int NCH>
__device__ __forceinline__ void row_store_p(const uint32_t (&pk)[NCH * 16], int ch0, uint8_t *bp,
                                            uint32_t prow, uint32_t sub, int r) {
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    const int cha = ch0 + ch;
    const uint32_t dst = prow + (cha >> 1) * sub;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c16 = (cha & 1) * 4 + u;
      *reinterpret_cast<uint4 *>(bp + dst + ((c16 ^ (r & 7)) << 4)) =
          make_uint4(pk[ch * 16 + 4 * u], pk[ch * 16 + 4 * u + 1], pk[ch * 16 + 4 * u + 2],
                     pk[ch * 16 + 4 * u + 3]);
    }
  }
}

// ---------------------------------------------------------------------------
// Tensor-core issue.  A tcgen05.mma returns to the issuing thread only once the tensor
// core has taken it, about as long as it then runs (~65 cycles for M=128, N<=128, K=16),
// so any work the thread does between two of them leaves the tensor core idle.  The MMA
// thread therefore builds every descriptor before a sequence and issues four at a time
// from one straight-line block: the first accumulates per `acc_first`, the others always.

// Adds a byte offset (a multiple of 16) to a shared-memory descriptor's start address.
__device__ __forceinline__ uint64_t desc_add(uint64_t desc, uint32_t bytes) {
  return desc + (uint64_t)(bytes >> 4);
}

__device__ __forceinline__ void umma4(uint32_t d_tmem, uint64_t a0, uint64_t a1, uint64_t a2,
                                      uint64_t a3, uint64_t b0, uint64_t b1, uint64_t b2,
                                      uint64_t b3, uint32_t idesc, uint32_t acc_first) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %10, 0;\n\tsetp.eq.u32 q, 1, 1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %5, %9, p;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %6, %9, q;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %7, %9, q;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %8, %9, q;\n\t}" ::"r"(d_tmem),
      "l"(a0), "l"(a1), "l"(a2), "l"(a3), "l"(b0), "l"(b1), "l"(b2), "l"(b3), "r"(idesc),
      "r"(acc_first)
      : "memory");
}

// S = Q . K^T over D: D/16 MMAs of K = 16.  q, k: descriptors of the K-major, 128-byte
// swizzled tiles (64-dim sub-tiles `sub` bytes apart).
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint64_t q, uint64_t k, uint32_t sub,
                                         uint32_t idesc) {
#pragma unroll
  for (int g4 = 0; g4 < D / 64; ++g4) {
    const uint32_t o = g4 * sub;
    umma4(d_tmem, desc_add(q, o), desc_add(q, o + 32), desc_add(q, o + 64), desc_add(q, o + 96),
          desc_add(k, o), desc_add(k, o + 32), desc_add(k, o + 64), desc_add(k, o + 96), idesc,
          g4 > 0 ? 1u : 0u);
  }
}

// O (+)= P . V over a block of kTcKeys keys: kTcKeys/16 MMAs of K = 16.  p: descriptor of
// the K-major P buffer (64-key sub-tiles `sub` bytes apart); v: descriptor of the
// MN-major V tile (16 keys = 2048 bytes apart).
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint64_t p, uint64_t v, uint32_t sub,
                                         uint32_t idesc, uint32_t acc_first) {
#pragma unroll
  for (int g4 = 0; g4 < kTcKeys / 64; ++g4) {
    const uint32_t o = g4 * sub, vo = g4 * 4 * 2048u;
    umma4(d_tmem, desc_add(p, o), desc_add(p, o + 32), desc_add(p, o + 64), desc_add(p, o + 96),
          desc_add(v, vo), desc_add(v, vo + 2048), desc_add(v, vo + 4096), desc_add(v, vo + 6144),
          idesc, g4 > 0 ? 1u : acc_first);
  }
}

// The same with P read from TMEM (the A operand in TMEM: row i in lane i, column c
// holding keys 2c and 2c+1): p_tmem is P's first column; K slice kk is 8 columns on.
__device__ __forceinline__ void umma4_ts(uint32_t d_tmem, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint64_t b0, uint64_t b1, uint64_t b2,
                                         uint64_t b3, uint32_t idesc, uint32_t acc_first) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %10, 0;\n\tsetp.eq.u32 q, 1, 1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %5, %9, p;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %6, %9, q;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %7, %9, q;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], %8, %9, q;\n\t}" ::"r"(d_tmem),
      "r"(a0), "r"(a1), "r"(a2), "r"(a3), "l"(b0), "l"(b1), "l"(b2), "l"(b3), "r"(idesc),
      "r"(acc_first)
      : "memory");
}
__device__ __forceinline__ void issue_pv_ts(uint32_t d_tmem, uint32_t p_tmem, uint64_t v,
                                            uint32_t idesc, uint32_t acc_first,
                                            uint32_t group_cols = 32u) {
#pragma unroll
  for (int g4 = 0; g4 < kTcKeys / 64; ++g4) {
    const uint32_t a = p_tmem + group_cols * g4, vo = g4 * 4 * 2048u;
    umma4_ts(d_tmem, a, a + 8, a + 16, a + 24, desc_add(v, vo), desc_add(v, vo + 2048),
             desc_add(v, vo + 4096), desc_add(v, vo + 6144), idesc, g4 > 0 ? 1u : acc_first);
  }
}

}  // namespace pkv
