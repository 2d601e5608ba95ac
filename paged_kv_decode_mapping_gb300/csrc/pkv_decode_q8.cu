// pkv_decode_q8.cu -- single-token attention over the 8-bit paged cache, and the whole step.
//
//   s_t = scale * ks[n] * <q, ck_t>,   out = sum_t softmax(s)_t * vs[n] * cv_t,   n = t's page
//
// HBM-bound: 2 bytes of K and V per (key, dim) feed G = Hq / Hkv query heads.  What differs from
// the bf16 decode:
//  * Codes are exact in fp16, so the products are mma.sync m16n8k16 fp16 tiles (16 keys x 8 heads)
//    with fp32 accumulators.  q, scaled by a power of two for its largest value to be in
//    [2^14, 2^15), is fp16 without loss down to 2^-29 of that value; the weights are fp16 with
//    their largest at 2^15, times the page's V scale over the largest so far.  Scales of K apply
//    to the scores.  (bf16 weights, without those two scalings, want a second product for their
//    low halves.)
//  * No ldmatrix: the fragments' element order along dims (K) and along keys (V) is free, as long
//    as both operands agree, so each lane loads 16 bytes in a row and widens them in registers:
//    K rows' dims 2 bytes at a time, V rows by interleaving the bytes of two keys (prmt).
//  * The batch's keys, in 128-key chunks, are one list (sequence, kv head, chunk), and every CTA
//    of a single wave takes an even share of it.  A (sequence, kv head) that several CTAs share
//    is merged by the last of them, in the order of the keys whoever that is.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "decode_device.cuh"
#include "q8_device.cuh"

namespace pkv {
namespace {

constexpr int kQ8Keys = 128;           // keys of a stage: 32 for each consumer warp
constexpr int kQ8MinChunks = 2;        // chunks a CTA takes at least (fewer CTAs run otherwise)
constexpr int kQ8MaxCtas = 1024;       // CTAs of a launch, at most
constexpr float kWeightLog2 = 15.f;    // the largest weight is 2^15 (fp16 ends at 65504)

constexpr int q8_stages(int d) { return d == 64 ? 4 : 3; }
constexpr int q8_occupancy(int d) { return d == 64 ? 3 : 2; }

struct Q8Desc {                 // one stage's chunk
  int32_t b, g, key0, len;      // its first key, and the context's length
  int32_t first, last;          // of this CTA's share of the (sequence, kv head)
  int32_t slot;                 // partial row its result goes to; -1: the whole context is here
  int32_t cta0, parts;          // CTAs that share it: cta0 .. cta0 + parts - 1
};

template <int D>
struct Q8Smem {  // offsets from the 1024-byte aligned base
  static constexpr int kStages = q8_stages(D);
  static constexpr uint32_t kTile = kQ8Keys * D;
  static constexpr uint32_t kStage = 2 * kTile;
  static constexpr uint32_t kQ = kMaxGroup * D * 2;
  static constexpr uint32_t q = kStages * kStage;
  static constexpr uint32_t scales = q + kStages * kQ;             // ks[16], vs[16] of a stage
  static constexpr uint32_t desc = scales + kStages * 128;
  static constexpr uint32_t bars = (desc + kStages * (uint32_t)sizeof(Q8Desc) + 15) / 16 * 16;
  static constexpr uint32_t misc = bars + kStages * 16;            // flag, last, issued, start b
  static constexpr uint32_t sums = misc + 32;                      // the prefix scan's warps
  static constexpr uint32_t total = sums + 64;
};
constexpr size_t q8_smem(int d) { return 1024 + (d == 64 ? Q8Smem<64>::total : Q8Smem<128>::total); }
static_assert(3 * (q8_smem(64) + 1024) <= 228 * 1024 && 2 * (q8_smem(128) + 1024) <= 228 * 1024,
              "8-bit decode CTAs per SM");
static_assert(kConsumerWarps * kMaxGroup * (128 + 2) * 4 <= (int)Q8Smem<128>::kStage &&
                  kConsumerWarps * kMaxGroup * (64 + 2) * 4 <= (int)Q8Smem<64>::kStage,
              "the warps' merge fits a stage");

struct Q8Args {
  const uint16_t *q;            // [B][Hq][D]
  uint16_t *out;
  const int32_t *tables, *lens;
  const float *k_scale, *v_scale;
  float *o_part;                // [2 * CTAs][G][D]: a CTA's first share's row, then its last's
  float *lse_part;              // [2 * CTAs][G], base 2
  uint32_t *counters;           // [kQ8MaxCtas] by first sharing CTA; zero between calls
  int64_t num_blocks;
  int32_t max_blocks, max_len, num_seqs, num_q_heads, num_kv_heads, group;
  int32_t block_size, log2_bs, box_rows, log2_box;
  float scale_log2;
};

// Which key of a 16-key tile row r of the products' fragments is.  Lanes read K rows key_of(2j),
// key_of(2j + 1) together, and V rows key_of(2t + i), t = 0 .. 3: with 64-byte rows this order puts
// each such set into different banks; with 128-byte rows the swizzle does it alone.
template <int D>
__device__ __forceinline__ int key_of(int r) {
  return D == 128 ? r : (r & 8) | (int)((0x65742130u >> (4 * (r & 7))) & 7u);
}
// Byte offset of 16-byte chunk `c` of key row `key` in a tile filled by swizzled boxes.
template <int D>
__device__ __forceinline__ uint32_t chunk_off(int key, int c) {
  return (uint32_t)(key * D + ((c ^ (D == 128 ? key & 7 : (key >> 1) & 3)) << 4));
}

__device__ __forceinline__ void lds(uint32_t (&w)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr));
}
__device__ __forceinline__ void lds(uint32_t (&w)[2], uint32_t addr) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}

// D(16x8, f32) += A(16x16, fp16, row) * B(16x8, fp16, col)
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A consumer warp's state.  Lane (gid, tig): O^T fragments, row gid of m-tile mt being dim
// D/8 * gid + 2 mt and row gid + 8 the dim after it, for heads 2 tig and 2 tig + 1.
template <int D>
struct Q8Acc {
  float o[D / 16][4];
  float m0, m1, l0, l1;
  float vref, vinv;         // the largest V scale so far, and 1 over it: o is in units of vref
  uint32_t q[D / 16][2];    // fragments of q, fp16
  float f0, f1;             // scores' factors of the two heads, without K's scale
};

// The (sequence, kv head)'s query rows at qs ([G][D] bf16, shared) as fragments: head gid, the
// dims that this lane's K bytes hold (D/4 tig ..).
template <int D>
__device__ __forceinline__ void load_q(Q8Acc<D> &a, uint32_t qs, int group, int lane, float scale_log2) {
  const int gid = lane >> 2, tig = lane & 3;
  uint32_t w[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) w[i] = 0u;
  if (gid < group) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t v[4];
      lds(v, qs + (uint32_t)(gid * D + (D / 4) * tig + 8 * i) * 2u);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[4 * i + k] = v[k];
    }
  }
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
    mx = fmaxf(mx, fmaxf(fabsf(dev::bf16lo_to_f32(w[i])), fabsf(dev::bf16hi_to_f32(w[i]))));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  // 2^(14 - exponent of mx), as far as that and its inverse are normal numbers
  const int e = min(max(14 - ((int)(__float_as_uint(mx) >> 23) - 127), -126), 126);
  const float up = __uint_as_float((uint32_t)(e + 127) << 23);
  const float down = __uint_as_float((uint32_t)(127 - e) << 23) * scale_log2;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      a.q[ks][k] = pack_f16x2(dev::bf16lo_to_f32(w[2 * ks + k]) * up, dev::bf16hi_to_f32(w[2 * ks + k]) * up);
  a.f0 = __shfl_sync(0xffffffffu, down, 8 * tig);  // lanes of heads 2 tig and 2 tig + 1
  a.f1 = __shfl_sync(0xffffffffu, down, 8 * tig + 4);
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) a.o[mt][0] = a.o[mt][1] = a.o[mt][2] = a.o[mt][3] = 0.f;
  a.m0 = a.m1 = -INFINITY;
  a.l0 = a.l1 = a.vref = a.vinv = 0.f;
}

// Scores, softmax and weighted sum of the warp's 32 keys (the first nvalid of them in range) of a
// stage: K tile at kb, V tile at vb, the boxes' scales at sc (ks[16], vs[16]).
template <int D, int KIND>
__device__ __forceinline__ void q8_tiles(Q8Acc<D> &a, uint32_t kb, uint32_t vb, const float *sc, int log2_box,
                                         int warp, int lane, int nvalid) {
  constexpr int KS = D / 16;
  const int gid = lane >> 2, tig = lane & 3;
  float s[2][4], vs[4];
  float mx0 = -INFINITY, mx1 = -INFINITY, vmax = 0.f;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int nv = nvalid - 16 * t;  // uniform over the warp
    vs[2 * t] = vs[2 * t + 1] = 0.f;
    s[t][0] = s[t][1] = s[t][2] = s[t][3] = -INFINITY;
    if (nv <= 0) continue;
    float c[4] = {0.f, 0.f, 0.f, 0.f};
    const int r0 = 32 * warp + 16 * t + key_of<D>(gid);
    uint32_t w0[D / 16], w1[D / 16];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      uint32_t x[4], y[4];
      lds(x, kb + chunk_off<D>(r0, (D / 64) * tig + i));
      lds(y, kb + chunk_off<D>(r0 + 8, (D / 64) * tig + i));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w0[4 * i + k] = q8::prep<KIND>(x[k]);
        w1[4 * i + k] = q8::prep<KIND>(y[k]);
      }
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      mma_f16_16816(c, q8::pair<KIND, 0>(w0[ks]), q8::pair<KIND, 0>(w1[ks]), q8::pair<KIND, 1>(w0[ks]),
                    q8::pair<KIND, 1>(w1[ks]), a.q[ks][0], a.q[ks][1]);
    // a half of 8 keys lies in one box; a half past the range has no scale
    const int b0 = (32 * warp + 16 * t) >> log2_box, b1 = (32 * warp + 16 * t + 8) >> log2_box;
    const float ks0 = sc[b0], ks1 = nv > 8 ? sc[b1] : 0.f;
    vs[2 * t] = sc[16 + b0];
    vs[2 * t + 1] = nv > 8 ? sc[16 + b1] : 0.f;
    if (key_of<D>(gid) < nv) {
      s[t][0] = c[0] * (a.f0 * ks0);
      s[t][1] = c[1] * (a.f1 * ks0);
    }
    if (key_of<D>(gid) + 8 < nv) {
      s[t][2] = c[2] * (a.f0 * ks1);
      s[t][3] = c[3] * (a.f1 * ks1);
    }
    mx0 = fmaxf(mx0, fmaxf(s[t][0], s[t][2]));
    mx1 = fmaxf(mx1, fmaxf(s[t][1], s[t][3]));
    vmax = fmaxf(vmax, fmaxf(vs[2 * t], vs[2 * t + 1]));
  }
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) {
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, x));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, x));
  }
  const float mn0 = fmaxf(a.m0, mx0), mn1 = fmaxf(a.m1, mx1);
  const float ref0 = softmax_ref(mn0), ref1 = softmax_ref(mn1);
  // The running maxima and the largest V scale move rarely once a few keys are seen.
  if (vmax > a.vref || __any_sync(0xffffffffu, mn0 > a.m0 || mn1 > a.m1)) {
    float al0 = dev::ex2(a.m0 - ref0), al1 = dev::ex2(a.m1 - ref1);
    a.l0 *= al0;
    a.l1 *= al1;
    if (vmax > a.vref) {
      a.vinv = 1.f / vmax;
      al0 *= a.vref * a.vinv;
      al1 *= a.vref * a.vinv;
      a.vref = vmax;
    }
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      a.o[mt][0] *= al0;
      a.o[mt][1] *= al1;
      a.o[mt][2] *= al0;
      a.o[mt][3] *= al1;
    }
    a.m0 = mn0;
    a.m1 = mn1;
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int nv = nvalid - 16 * t;
    if (nv <= 0) continue;
    const float p0 = dev::ex2(s[t][0] - ref0 + kWeightLog2), p1 = dev::ex2(s[t][1] - ref1 + kWeightLog2);
    const float p2 = dev::ex2(s[t][2] - ref0 + kWeightLog2), p3 = dev::ex2(s[t][3] - ref1 + kWeightLog2);
    a.l0 += p0 + p2;
    a.l1 += p1 + p3;
    const float r0 = vs[2 * t] * a.vinv, r1 = vs[2 * t + 1] * a.vinv;
    const uint32_t b0 = dev::movmatrix_trans(pack_f16x2(p0 * r0, p1 * r0));
    const uint32_t b1 = dev::movmatrix_trans(pack_f16x2(p2 * r1, p3 * r1));
    // V bytes of 4 keys, D/8 dims from D/8 gid on; a row past the range may hold anything (e4m3
    // has NaN codes): zeroed
    uint32_t w[4][D / 32];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int key = key_of<D>(2 * tig + (k & 1) + 8 * (k >> 1));
      const int row = 32 * warp + 16 * t + key;
      if constexpr (D == 128)
        lds(w[k], vb + chunk_off<D>(row, gid));
      else
        lds(w[k], vb + chunk_off<D>(row, gid >> 1) + 8u * (gid & 1));
      const uint32_t keep = key < nv ? 0xffffffffu : 0u;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) w[k][i] = q8::prep<KIND>(KIND == PKV_Q8_E4M3 ? w[k][i] & keep : w[k][i]);
    }
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      const uint32_t sel = mt & 1 ? 0x7362 : 0x5140;  // bytes (key, key', key, key') of dims 2mt, 2mt + 1
      const uint32_t lo = __byte_perm(w[0][mt / 2], w[1][mt / 2], sel);
      const uint32_t hi = __byte_perm(w[2][mt / 2], w[3][mt / 2], sel);
      mma_f16_16816(a.o[mt], q8::pair<KIND, 0>(lo), q8::pair<KIND, 1>(lo), q8::pair<KIND, 0>(hi),
                    q8::pair<KIND, 1>(hi), b0, b1);
    }
  }
}

// Reduces l over the warp and writes the warp's (m, l, O) for heads < G.
template <int D>
__device__ __forceinline__ void q8_stash(Q8Acc<D> &a, const MergeArea &r, int G, int warp, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
  float l0 = a.l0, l1 = a.l1;
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, x);
    l1 += __shfl_xor_sync(0xffffffffu, l1, x);
  }
  const int h0 = 2 * tig, h1 = h0 + 1;
  if (gid == 0) {
    r.m[warp * kMaxGroup + h0] = a.m0;
    r.m[warp * kMaxGroup + h1] = a.m1;
    r.l[warp * kMaxGroup + h0] = l0;
    r.l[warp * kMaxGroup + h1] = l1;
  }
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) {
    const int d = (D / 8) * gid + 2 * mt;
    if (h0 < G)
      *reinterpret_cast<float2 *>(r.o + (warp * G + h0) * D + d) =
          make_float2(a.o[mt][0] * a.vref, a.o[mt][2] * a.vref);
    if (h1 < G)
      *reinterpret_cast<float2 *>(r.o + (warp * G + h1) * D + d) =
          make_float2(a.o[mt][1] * a.vref, a.o[mt][3] * a.vref);
  }
}

// One head's partial results -- rows row_of(0 .. n-1): normalised output and base-2 log-sum --
// merged into bf16.  One warp; as merge_rows, but for where the rows are.
template <int D>
__device__ __forceinline__ void q8_merge_head(uint16_t *dst, const Q8Args &a, int cta0, int n, int h, int lane) {
  constexpr int VPL = D / 32;
  float M = -INFINITY, den = 0.f, acc[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) acc[v] = 0.f;
  for (int k0 = 0; k0 < n; k0 += 8) {
    float lk[8], ov[8][VPL];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int k = k0 + u;
      lk[u] = -INFINITY;
#pragma unroll
      for (int v = 0; v < VPL; ++v) ov[u][v] = 0.f;
      if (k < n) {
        const int64_t row = (int64_t)(k == 0 ? 2 * cta0 + 1 : 2 * (cta0 + k)) * a.group + h;
        lk[u] = __ldcg(a.lse_part + row);
        const float *src = a.o_part + row * D + lane * VPL;
        if constexpr (VPL == 2) {
          const float2 t2 = __ldcg(reinterpret_cast<const float2 *>(src));
          ov[u][0] = t2.x;
          ov[u][1] = t2.y;
        } else {
          const float4 t4 = __ldcg(reinterpret_cast<const float4 *>(src));
          ov[u][0] = t4.x;
          ov[u][1] = t4.y;
          ov[u][2] = t4.z;
          ov[u][3] = t4.w;
        }
      }
    }
    float mb = lk[0];
#pragma unroll
    for (int u = 1; u < 8; ++u) mb = fmaxf(mb, lk[u]);
    const float Mn = fmaxf(M, mb), ref = softmax_ref(Mn);
    const float sc = dev::ex2(M - ref);
    den *= sc;
#pragma unroll
    for (int v = 0; v < VPL; ++v) acc[v] *= sc;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float wt = dev::ex2(lk[u] - ref);
      den += wt;
#pragma unroll
      for (int v = 0; v < VPL; ++v) acc[v] += wt * ov[u][v];
    }
    M = Mn;
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  uint16_t *d = dst + lane * VPL;
  if constexpr (VPL == 2)
    *reinterpret_cast<uint32_t *>(d) = dev::pack_bf16x2(acc[0] * inv, acc[1] * inv);
  else
    *reinterpret_cast<uint2 *>(d) = make_uint2(dev::pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                              dev::pack_bf16x2(acc[2] * inv, acc[3] * inv));
}

// The end of a share, on the consumer warps after q8_stash (cf. finish_partition).
template <int D>
__device__ __forceinline__ void q8_finish(const Q8Args &a, const MergeArea &r, const Q8Desc &d, int tid, int warp,
                                          int lane, volatile int *s_flag, volatile int *s_last) {
  const int64_t head0 = (int64_t)d.b * a.num_q_heads + d.g * a.group;
  for (int i = tid; i < a.group * D; i += kConsumers) {
    const int h = i / D, c = i - h * D;
    float M2, den;
    const float val = cta_merge<D>(r, a.group, h, c, &M2, &den);
    if (d.slot < 0) {
      a.out[head0 * D + i] = to_bf16(val);
    } else {
      const int64_t row = (int64_t)d.slot * a.group + h;
      a.o_part[row * D + c] = val;
      if (c == 0) a.lse_part[row] = M2 + log2f(den);
    }
  }
  if (d.slot < 0) return;
  consumer_bar();
  if (tid == 0) {
    int last = 0;
    if (!*s_flag) last = dev::atomic_add_acq_rel(a.counters + d.cta0, 1u) + 1 == (unsigned)d.parts;
    *s_last = last;
  }
  consumer_bar();
  if (*s_last) {
    for (int h = warp; h < a.group; h += kConsumerWarps)
      q8_merge_head<D>(a.out + (head0 + h) * D, a, d.cta0, d.parts, h, lane);
    if (tid == 0) a.counters[d.cta0] = 0u;  // ready for the next call
  }
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const float *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival on `bar` when this thread's cp.asyncs so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads, q8_occupancy(D))
    decode_q8_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                     const __grid_constant__ Q8Args a) {
  using SL = Q8Smem<D>;
  constexpr int STAGES = SL::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = dev::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *const base_ptr = smem_raw + (base - raw);
  const uint32_t bar_full = base + SL::bars, bar_empty = bar_full + STAGES * 8;
  volatile int *const s_flag = reinterpret_cast<volatile int *>(base_ptr + SL::misc);
  volatile int *const s_last = s_flag + 1;
  volatile int *const s_issued = s_flag + 2;
  volatile int *const s_b = s_flag + 3;
  volatile int64_t *const s_base = reinterpret_cast<volatile int64_t *>(base_ptr + SL::misc + 16);
  volatile int64_t *const s_sums = reinterpret_cast<volatile int64_t *>(base_ptr + SL::sums);
  Q8Desc *const s_desc = reinterpret_cast<Q8Desc *>(base_ptr + SL::desc);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hkv = a.num_kv_heads;
  const int cap = (int)min((int64_t)a.max_blocks * a.block_size, (int64_t)a.max_len);
  auto length = [&](int b) { return min(max(__ldg(a.lens + b), 0), cap); };
  auto chunks_of = [](int L) { return (int)(((int64_t)L + kQ8Keys - 1) / kQ8Keys); };

  // ---- this CTA's share of the list: the prefix of the sequences' chunks, a run of sequences
  // per thread
  const int run = (a.num_seqs + kThreads - 1) / kThreads;
  const int b_lo = min(tid * run, a.num_seqs), b_hi = min(b_lo + run, a.num_seqs);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const int L0 = __ldg(a.lens + b), L = min(max(L0, 0), cap);
    if (L != L0 && blockIdx.x == 0) raise_error(PKV_DEVERR_CONTEXT_LEN);
    mine += chunks_of(L);
    if (L == 0 && b % (int)gridDim.x == (int)blockIdx.x) {  // empty context: zero output
      uint2 *o = reinterpret_cast<uint2 *>(a.out + (int64_t)b * a.num_q_heads * D);
      for (int i = 0; i < a.num_q_heads * D / 4; ++i) o[i] = make_uint2(0u, 0u);
    }
  }
  if (tid == 0) {
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      dev::mbar_init(bar_full + 8 * s, 33);  // lane 0's bytes, and every producer lane's scales
      dev::mbar_init(bar_empty + 8 * s, kConsumerWarps);
    }
    *s_flag = 0;
    *s_issued = 0;
    dev::fence_mbar_init();
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_sums[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += s_sums[w];
    total += s_sums[w];
  }
  const int64_t W = total * Hkv;
  const int64_t N = min((int64_t)gridDim.x, max((int64_t)1, (W + kQ8MinChunks - 1) / kQ8MinChunks));
  if ((int64_t)blockIdx.x >= N || W == 0) return;
  const int64_t lo = W * blockIdx.x / N, hi = W * (blockIdx.x + 1) / N;
  if (before * Hkv <= lo && lo < (before + mine) * Hkv) {  // one thread
    int b = b_lo;
    int64_t at = before;
    for (;; ++b) {
      const int n = chunks_of(length(b));
      if (lo < (at + n) * Hkv) break;
      at += n;
    }
    *s_b = b;
    *s_base = at * Hkv;
  }
  __syncthreads();
  const int n_chunks = (int)(hi - lo);

  if (warp == kConsumerWarps) {
    // ------------------------------------------------------------- producer warp
    const uint64_t policy = dev::policy_evict_first();
    const int rb = a.box_rows;
    const uint32_t box_bytes = (uint32_t)(rb * D);
    const uint32_t q_bytes = (uint32_t)a.group * D * 2u;
    int b = *s_b;
    int64_t seq0 = *s_base;  // where the sequence begins in the list
    int L = length(b), nch = chunks_of(L);
    int g = (int)((lo - seq0) / nch), c = (int)((lo - seq0) - (int64_t)g * nch);
    const int32_t *trow = a.tables + (int64_t)b * a.max_blocks;
    int win = -1, tb = 0;  // lanes hold the table's entries [win, win + 32)
    Q8Desc dsc;
    bool first = true;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the step's write is done
    int i = 0;
    for (; i < n_chunks; ++i) {
      const int s = i % STAGES;
      if (first) {
        const int64_t u0 = seq0 + (int64_t)g * nch, u1 = u0 + nch;
        dsc.b = b;
        dsc.g = g;
        dsc.len = L;
        dsc.slot = -1;
        dsc.cta0 = (int)blockIdx.x;
        dsc.parts = 1;
        if (u0 < lo || u1 > hi) {  // shared: place x is CTA floor(((x + 1) N - 1) / W)'s
          dsc.cta0 = (int)(((u0 + 1) * N - 1) / W);
          dsc.parts = (int)((u1 * N - 1) / W) - dsc.cta0 + 1;
          dsc.slot = 2 * (int)blockIdx.x + (dsc.cta0 == (int)blockIdx.x ? 1 : 0);
        }
      }
      if (i >= STAGES &&
          !__all_sync(0xffffffffu, dev::mbar_wait(bar_empty + 8 * s, ((i / STAGES) - 1) & 1))) {
        if (lane == 0) {
          raise_error(PKV_DEVERR_TIMEOUT);
          *s_flag = 1;
        }
        break;
      }
      const int k0 = c * kQ8Keys;
      const int nk = min(kQ8Keys, L - k0);
      const int nbox = (nk + rb - 1) >> a.log2_box;
      const int lb_hi = (k0 + (nbox - 1) * rb) >> a.log2_bs;
      if (win < 0 || (k0 >> a.log2_bs) < win || lb_hi >= win + 32) {
        win = k0 >> a.log2_bs;
        tb = win + lane <= ((L - 1) >> a.log2_bs) ? __ldg(trow + win + lane) : 0;
      }
      const int key = k0 + lane * rb;
      const int64_t phys_raw = __shfl_sync(0xffffffffu, tb, min(max((key >> a.log2_bs) - win, 0), 31));
      if (lane == 0) {
        dsc.key0 = k0;
        dsc.first = first ? 1 : 0;
        dsc.last = c + 1 == nch || i + 1 == n_chunks ? 1 : 0;
        s_desc[s] = dsc;
        dev::mbar_arrive_expect_tx(bar_full + 8 * s, 2u * nbox * box_bytes + (first ? q_bytes : 0u));
        if (first)
          dev::bulk_load(base + SL::q + s * SL::kQ, a.q + ((int64_t)b * a.num_q_heads + g * a.group) * D, q_bytes,
                         bar_full + 8 * s);
      }
      __syncwarp();
      if (lane < nbox) {
        int64_t phys = phys_raw;
        if (phys < 0 || phys >= a.num_blocks) {
          raise_error(PKV_DEVERR_BLOCK_ID);
          phys = 0;
        }
        const int64_t unit = phys * Hkv + g;
        const int32_t row = (int32_t)(unit * a.block_size + (key & (a.block_size - 1)));
        const uint32_t dk = base + s * SL::kStage + lane * box_bytes;
        dev::tma_load_2d(dk, &tmk, 0, row, bar_full + 8 * s, policy);
        dev::tma_load_2d(dk + SL::kTile, &tmv, 0, row, bar_full + 8 * s, policy);
        const uint32_t ds = base + SL::scales + s * 128 + lane * 4;
        cp_async4(ds, a.k_scale + unit);
        cp_async4(ds + 64, a.v_scale + unit);
      }
      cp_async_arrive(bar_full + 8 * s);
      __syncwarp();
      first = false;
      if (++c == nch) {  // the next kv head, or the next sequence that has keys
        c = 0;
        first = true;
        if (++g == Hkv && i + 1 < n_chunks) {
          g = 0;
          seq0 += (int64_t)nch * Hkv;
          do {  // i + 1 < n_chunks: there is one
            L = length(++b);
          } while (L == 0 && b + 1 < a.num_seqs);
          nch = chunks_of(L);
          trow = a.tables + (int64_t)b * a.max_blocks;
          win = -1;
        }
      }
    }
    if (lane == 0) *s_issued = i;
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ----------------------------------------------------------- consumer warps
    Q8Acc<D> acc;
    for (int i = 0; i < n_chunks; ++i) {
      const int s = i % STAGES;
      if (!__all_sync(0xffffffffu, dev::mbar_wait(bar_full + 8 * s, (i / STAGES) & 1))) {
        if (lane == 0) {
          raise_error(PKV_DEVERR_TIMEOUT);
          *s_flag = 1;
        }
        break;
      }
      const int key0 = s_desc[s].key0, len = s_desc[s].len;
      if (s_desc[s].first) load_q<D>(acc, base + SL::q + s * SL::kQ, a.group, lane, a.scale_log2);
      const uint32_t kb = base + s * SL::kStage;
      const int nvalid = min(32, len - key0 - 32 * warp);
      if (nvalid > 0)
        q8_tiles<D, KIND>(acc, kb, kb + SL::kTile, reinterpret_cast<const float *>(base_ptr + SL::scales + s * 128),
                          a.log2_box, warp, lane, nvalid);
      if (s_desc[s].last) {
        const Q8Desc d = s_desc[s];
        consumer_bar();  // every warp is done with this stage's tiles: reuse them to merge
        MergeArea r;
        r.o = reinterpret_cast<float *>(base_ptr + s * SL::kStage);
        r.m = r.o + kConsumerWarps * a.group * D;
        r.l = r.m + kConsumerWarps * kMaxGroup;
        q8_stash<D>(acc, r, a.group, warp, lane);
        consumer_bar();
        q8_finish<D>(a, r, d, tid, warp, lane, s_flag, s_last);
        dev::fence_proxy_async_smem();  // what was written here, ahead of the next boxes
      }
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(bar_empty + 8 * s);
    }
  }

  // ---- a timed-out wait leaves copies possibly in flight: wait for them (bounded)
  __syncthreads();
  if (tid == 0 && *s_flag) {
    const int issued = *s_issued;
    for (int s = 0; s < STAGES; ++s) {
      const int last = s + ((issued - 1 - s) / STAGES) * STAGES;  // last chunk on stage s
      if (last >= 0 && last < issued) (void)dev::mbar_wait(bar_full + 8 * s, (last / STAGES) & 1);
    }
  }
}

bool g_q8_attr[kMaxDevices][2][2];  // kernel attributes set [head_dim][kind]

struct Q8Layout {
  size_t o_part, lse_part, total;
};

// Counters first, at the same place for every call; then the partial rows of as many CTAs as the
// GPU holds.
Q8Layout q8_layout(int group, int d, int sms) {
  const size_t rows = (size_t)2 * std::min(sms * q8_occupancy(d), kQ8MaxCtas) * group;
  Q8Layout l;
  l.o_part = kQ8MaxCtas * sizeof(uint32_t);
  l.lse_part = l.o_part + rows * d * sizeof(float);
  l.total = (l.lse_part + rows * sizeof(float) + 255) & ~size_t(255);
  return l;
}

struct DecodeQ8 {
  pkv_bf16 *out;
  const pkv_bf16 *q;
  const pkv_q8_cache *cache;
  const int32_t *tables;
  int32_t max_blocks;
  const int32_t *lens;
  int32_t max_len, num_seqs, hq;
  const pkv_cache_desc *desc;
  float scale;
  void *workspace;
  size_t workspace_bytes;
};

int sms_now(int *sms) {
  std::lock_guard<std::mutex> lk(attn_mutex());
  return device_sms(sms);
}

int check_decode_q8(const DecodeQ8 &x, const char *fn) {
  int rc = check_q8(x.cache, x.desc, x.num_seqs, fn);
  if (!rc)
    rc = check_decode(x.q, x.cache->k_cache, x.cache->v_cache, x.tables, x.max_blocks, x.lens, x.max_len,
                      x.num_seqs, x.hq, x.desc, fn);
  if (rc || x.num_seqs == 0) return rc;
  if (!x.out) return set_error(PKV_ERR_NULL, "%s: out is NULL", fn);
  if (reinterpret_cast<uintptr_t>(x.out) & 7u) return set_error(PKV_ERR_ALIGN, "%s: out must be 8-byte aligned", fn);
  int sms = 0;
  if (sms_now(&sms) != PKV_OK) sms = 152;  // no device: the checks that need none still stand
  const Q8Layout l = q8_layout(x.hq / x.desc->num_kv_heads, x.desc->head_dim, sms);
  if (!x.workspace || x.workspace_bytes < l.total)
    return set_error(PKV_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, x.workspace_bytes, l.total);
  if (!aligned16(x.workspace)) return set_error(PKV_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
  return PKV_OK;
}

template <int D, int KIND>
int launch_decode_q8(const DecodeQ8 &x, cudaStream_t stream, bool programmatic) {
  const pkv_cache_desc &c = *x.desc;
  CUtensorMap tmk, tmv;
  int sms = 0;
  auto *const kern = decode_q8_kernel<D, KIND>;
  const int box = std::min(c.block_size, kQ8Keys);
  {
    std::lock_guard<std::mutex> lk(attn_mutex());
    int dev = 0, rc;
    if ((rc = current_device(&dev)) || (rc = device_sms(&sms)) || (rc = codes_map(x.cache->k_cache, c, box, &tmk)) ||
        (rc = codes_map(x.cache->v_cache, c, box, &tmv)))
      return rc;
    bool *const attr = &g_q8_attr[dev][D == 64 ? 0 : 1][KIND];
    if (!*attr) {
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)q8_smem(D));
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
      if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute");
      *attr = true;
    }
  }
  const Q8Layout l = q8_layout(x.hq / c.num_kv_heads, D, sms);
  char *const ws = static_cast<char *>(x.workspace);
  Q8Args a;
  a.q = x.q;
  a.out = x.out;
  a.tables = x.tables;
  a.lens = x.lens;
  a.k_scale = x.cache->k_scale;
  a.v_scale = x.cache->v_scale;
  a.counters = reinterpret_cast<uint32_t *>(ws);
  a.o_part = reinterpret_cast<float *>(ws + l.o_part);
  a.lse_part = reinterpret_cast<float *>(ws + l.lse_part);
  a.num_blocks = c.num_blocks;
  a.max_blocks = x.max_blocks;
  a.max_len = x.max_len;
  a.num_seqs = x.num_seqs;
  a.num_q_heads = x.hq;
  a.num_kv_heads = c.num_kv_heads;
  a.group = x.hq / c.num_kv_heads;
  a.block_size = c.block_size;
  a.log2_bs = ilog2(c.block_size);
  a.box_rows = box;
  a.log2_box = ilog2(box);
  a.scale_log2 = x.scale * kLog2e;
  // one wave; fewer CTAs where the batch cannot have that many shares of kQ8MinChunks
  const int64_t most = ((int64_t)x.max_len + kQ8Keys - 1) / kQ8Keys * x.num_seqs * c.num_kv_heads;
  const int64_t wave = std::min(sms * q8_occupancy(D), kQ8MaxCtas);
  const int64_t grid = std::max<int64_t>(1, std::min(wave, (most + kQ8MinChunks - 1) / kQ8MinChunks));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = q8_smem(D);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = programmatic ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmk, tmv, a);
  if (e != cudaSuccess) return cuda_error(e, "decode_q8_kernel launch");
  return PKV_OK;
}

int launch_decode_q8(const DecodeQ8 &x, cudaStream_t s, bool programmatic) {
  if (x.num_seqs == 0) return PKV_OK;
  const bool i8 = x.cache->kind == PKV_Q8_INT8;
  if (x.desc->head_dim == 64)
    return i8 ? launch_decode_q8<64, PKV_Q8_INT8>(x, s, programmatic)
              : launch_decode_q8<64, PKV_Q8_E4M3>(x, s, programmatic);
  return i8 ? launch_decode_q8<128, PKV_Q8_INT8>(x, s, programmatic)
            : launch_decode_q8<128, PKV_Q8_E4M3>(x, s, programmatic);
}

// Both halves of a step checked, then both enqueued.
int step_q8(const WriteQ8 &w, const DecodeQ8 &x, cudaStream_t s, const char *fn) {
  int rc = check_write_q8(w, fn);
  if (!rc) rc = check_decode_q8(x, fn);
  if (!rc) rc = launch_write_q8(w, s);
  if (!rc) rc = launch_decode_q8(x, s, w.num_seqs > 0);
  if (!rc) clear_error();
  return rc;
}

}  // namespace

cudaError_t read_decode_q8_errors(uint32_t *flags, int clear) { return read_tu_errors(flags, clear); }

}  // namespace pkv

using namespace pkv;

PKV_API size_t paged_decode_q8_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                              int32_t head_dim, int32_t max_context_len) {
  if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
      num_q_heads / num_kv_heads > kMaxGroup || (head_dim != 64 && head_dim != 128) || max_context_len < 0)
    return 0;
  int sms = 0;
  if (sms_now(&sms) != PKV_OK) sms = 152;
  return q8_layout(num_q_heads / num_kv_heads, head_dim, sms).total;
}

PKV_API int paged_decode_attention_q8(pkv_bf16 *out, const pkv_bf16 *q, const pkv_q8_cache *cache,
                                      const int32_t *block_tables, int32_t max_blocks_per_seq,
                                      const int32_t *context_lens, int32_t max_context_len, int32_t num_seqs,
                                      int32_t num_q_heads, const pkv_cache_desc *desc, float scale, void *workspace,
                                      size_t workspace_bytes, void *stream) {
  const DecodeQ8 x = {out, q, cache, block_tables, max_blocks_per_seq, context_lens, max_context_len,
                      num_seqs, num_q_heads, desc, scale, workspace, workspace_bytes};
  int rc = check_decode_q8(x, "paged_decode_attention_q8");
  if (!rc) rc = launch_decode_q8(x, static_cast<cudaStream_t>(stream), false);
  if (!rc) clear_error();
  return rc;
}

PKV_API int paged_decode_step_q8(pkv_bf16 *out, const pkv_bf16 *q, const pkv_bf16 *k, const pkv_bf16 *v,
                                 int64_t k_stride, int64_t v_stride, const pkv_q8_cache *cache,
                                 const int32_t *block_tables, int32_t max_blocks_per_seq,
                                 const int32_t *context_lens, int32_t max_context_len, int32_t num_seqs,
                                 int32_t num_q_heads, const pkv_cache_desc *desc, float scale, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  WriteQ8 w = {};
  w.k = k, w.v = v, w.k_stride = k_stride, w.v_stride = v_stride, w.num_tokens = num_seqs, w.max_query_len = 1;
  w.block_tables = block_tables, w.max_blocks = max_blocks_per_seq, w.context_lens = context_lens;
  w.num_seqs = num_seqs, w.cache = cache, w.desc = desc;
  const DecodeQ8 x = {out, q, cache, block_tables, max_blocks_per_seq, context_lens, max_context_len,
                      num_seqs, num_q_heads, desc, scale, workspace, workspace_bytes};
  return step_q8(w, x, static_cast<cudaStream_t>(stream), "paged_decode_step_q8");
}

PKV_API int paged_decode_step_rope_q8(pkv_bf16 *out, const pkv_bf16 *q, int64_t q_stride, pkv_bf16 *q_out,
                                      const pkv_bf16 *k, const pkv_bf16 *v, int64_t k_stride, int64_t v_stride,
                                      const int64_t *positions, const float *cos_sin, int64_t max_position,
                                      int32_t rotary_dim, int32_t neox_style, const pkv_q8_cache *cache,
                                      const int32_t *block_tables, int32_t max_blocks_per_seq,
                                      const int32_t *context_lens, int32_t max_context_len, int32_t num_seqs,
                                      int32_t num_q_heads, const pkv_cache_desc *desc, float scale, void *workspace,
                                      size_t workspace_bytes, void *stream) {
  const char *const fn = "paged_decode_step_rope_q8";
  if (num_seqs > 0 && (!q || !q_out)) return set_error(PKV_ERR_NULL, "%s: NULL q/q_out", fn);
  if (!desc) return set_error(PKV_ERR_NULL, "%s: cache descriptor is NULL", fn);
  WriteQ8 w = {};
  w.k = k, w.v = v, w.k_stride = k_stride, w.v_stride = v_stride, w.num_tokens = num_seqs, w.max_query_len = 1;
  w.block_tables = block_tables, w.max_blocks = max_blocks_per_seq, w.context_lens = context_lens;
  w.num_seqs = num_seqs, w.cache = cache, w.desc = desc;
  w.rope = true;
  w.q = q, w.q_out = q_out, w.q_stride = q_stride, w.q_out_stride = (int64_t)num_q_heads * desc->head_dim;
  w.num_q_heads = num_q_heads;
  w.positions = positions, w.cos_sin = cos_sin, w.max_position = max_position;
  w.rotary_dim = rotary_dim, w.neox_style = neox_style;
  const DecodeQ8 x = {out, q_out, cache, block_tables, max_blocks_per_seq, context_lens, max_context_len,
                      num_seqs, num_q_heads, desc, scale, workspace, workspace_bytes};
  return step_q8(w, x, static_cast<cudaStream_t>(stream), fn);
}
