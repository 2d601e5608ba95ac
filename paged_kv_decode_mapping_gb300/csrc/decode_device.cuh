// decode_device.cuh -- device pieces of the decode kernels: a consumer warp's softmax state
// and its work on one 64-key stage, the merge of a CTA's four warps, and the merge of
// partition results in global memory.
#pragma once

#include "attn_device.cuh"

namespace pkv {

// ---------------------------------------------------------------------------
// Per-warp state and the per-stage work of a consumer warp.

template <int D>
struct WarpAcc {
  float o[D / 16][4];  // O^T fragment: dims (16*mt + gid, +8) x heads (2*tig, 2*tig+1)
  float m0, m1, l0, l1;  // running max (base 2) and partial sum for heads 2*tig, 2*tig+1
};

template <int D>
__device__ __forceinline__ void acc_reset(WarpAcc<D> &a) {
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) a.o[mt][0] = a.o[mt][1] = a.o[mt][2] = a.o[mt][3] = 0.f;
  a.m0 = a.m1 = -INFINITY;
  a.l0 = a.l1 = 0.f;
}

// What exponents are taken against where the largest score so far is m: m, or, where no score
// was over -inf yet, 0, so that scores of -inf weigh 0 and a sum that is NaN tells of a NaN.
__device__ __forceinline__ float softmax_ref(float m) { return m == -INFINITY ? 0.f : m; }

// QK, online softmax and PV for this warp's 16 keys (nvalid of them in range) of the
// stage whose K tile is at kb and V tile at vb.
template <int D>
__device__ __forceinline__ void warp_tile(WarpAcc<D> &acc, const uint32_t (&qb)[D / 16][2],
                                          uint32_t kb, uint32_t vb, int warp, int lane, int nvalid,
                                          float scale_log2) {
  constexpr int KS = D / 16;
  const int gid = lane >> 2, tig = lane & 3;
  const int lj = lane >> 3, lr = lane & 7;  // ldmatrix: matrix index / row within it
  // QK operand A = K rows: matrices (keys 0-7 | 8-15) x (dims lo | hi) of a k step.
  const int qk_key = 16 * warp + lr + ((lj & 1) << 3), qk_dsel = lj >> 1;
  // PV operand A = V^T: matrices (keys 0-7, dims lo), (keys 0-7, dims hi), (keys 8-15, ...).
  const int pv_key = 16 * warp + lr + ((lj >> 1) << 3), pv_dsel = lj & 1;

  // S^T (16 keys x 8 heads) = K_tile . Q^T
  float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    uint32_t ak[4];
    dev::ldsm_x4(ak, kb + tile_off(qk_key, 2 * ks + qk_dsel));
    dev::mma_bf16_16816(sc, ak, qb[ks][0], qb[ks][1]);
  }
  // scale to base 2, mask keys past the range
  const bool v0 = gid < nvalid, v1 = gid + 8 < nvalid;
  const float s0 = v0 ? sc[0] * scale_log2 : -INFINITY;
  const float s1 = v0 ? sc[1] * scale_log2 : -INFINITY;
  const float s2 = v1 ? sc[2] * scale_log2 : -INFINITY;
  const float s3 = v1 ? sc[3] * scale_log2 : -INFINITY;
  float mx0 = fmaxf(s0, s2), mx1 = fmaxf(s1, s3);
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) {
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, x));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, x));
  }
  const float mn0 = fmaxf(acc.m0, mx0), mn1 = fmaxf(acc.m1, mx1);
  const float ref0 = softmax_ref(mn0), ref1 = softmax_ref(mn1);
  const float al0 = dev::ex2(acc.m0 - ref0), al1 = dev::ex2(acc.m1 - ref1);
  const float p0 = dev::ex2(s0 - ref0), p1 = dev::ex2(s1 - ref1);
  const float p2 = dev::ex2(s2 - ref0), p3 = dev::ex2(s3 - ref1);
  acc.l0 = acc.l0 * al0 + (p0 + p2);
  acc.l1 = acc.l1 * al1 + (p1 + p3);
  acc.m0 = mn0;
  acc.m1 = mn1;
#pragma unroll
  for (int mt = 0; mt < KS; ++mt) {
    acc.o[mt][0] *= al0;
    acc.o[mt][1] *= al1;
    acc.o[mt][2] *= al0;
    acc.o[mt][3] *= al1;
  }
  // P^T as the B operand: bf16 hi part and the bf16 residual, transposed
  const uint32_t h01 = dev::pack_bf16x2(p0, p1), h23 = dev::pack_bf16x2(p2, p3);
  const uint32_t r01 = dev::pack_bf16x2(p0 - dev::bf16lo_to_f32(h01), p1 - dev::bf16hi_to_f32(h01));
  const uint32_t r23 = dev::pack_bf16x2(p2 - dev::bf16lo_to_f32(h23), p3 - dev::bf16hi_to_f32(h23));
  const uint32_t bh0 = dev::movmatrix_trans(h01), bh1 = dev::movmatrix_trans(h23);
  const uint32_t bl0 = dev::movmatrix_trans(r01), bl1 = dev::movmatrix_trans(r23);
  // O^T (D x 8 heads) += V^T . P^T; rows of V past the range are zeroed in registers
  // (never multiply an unloaded row: 0 * NaN would poison O)
  uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
  if (nvalid < 16) {
    const int kk = 2 * tig;
    mlo = (kk < nvalid ? 0x0000ffffu : 0u) | (kk + 1 < nvalid ? 0xffff0000u : 0u);
    mhi = (kk + 8 < nvalid ? 0x0000ffffu : 0u) | (kk + 9 < nvalid ? 0xffff0000u : 0u);
  }
#pragma unroll
  for (int mt = 0; mt < KS; ++mt) {
    uint32_t av[4];
    dev::ldsm_x4_trans(av, vb + tile_off(pv_key, 2 * mt + pv_dsel));
    av[0] &= mlo;
    av[1] &= mlo;
    av[2] &= mhi;
    av[3] &= mhi;
    dev::mma_bf16_16816(acc.o[mt], av, bh0, bh1);
    dev::mma_bf16_16816(acc.o[mt], av, bl0, bl1);
  }
}

// Merge area of the four warps: red_o [warps][G][D], red_m / red_l [warps][8].
struct MergeArea {
  float *o, *m, *l;
};

// Reduces l over the warp and writes the warp's (m, l, O) for heads < G.
template <int D>
__device__ __forceinline__ void warp_stash(WarpAcc<D> &acc, const MergeArea &r, int G, int warp,
                                           int lane) {
  const int gid = lane >> 2, tig = lane & 3;
  float l0 = acc.l0, l1 = acc.l1;
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, x);
    l1 += __shfl_xor_sync(0xffffffffu, l1, x);
  }
  const int h0 = 2 * tig, h1 = h0 + 1;
  if (gid == 0) {
    r.m[warp * kMaxGroup + h0] = acc.m0;
    r.m[warp * kMaxGroup + h1] = acc.m1;
    r.l[warp * kMaxGroup + h0] = l0;
    r.l[warp * kMaxGroup + h1] = l1;
  }
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) {
    const int d = 16 * mt + gid;
    if (h0 < G) {
      r.o[(warp * G + h0) * D + d] = acc.o[mt][0];
      r.o[(warp * G + h0) * D + d + 8] = acc.o[mt][2];
    }
    if (h1 < G) {
      r.o[(warp * G + h1) * D + d] = acc.o[mt][1];
      r.o[(warp * G + h1) * D + d + 8] = acc.o[mt][3];
    }
  }
}

// The four warps' softmax states merged for head h, dim d: the normalised output;
// *M2 gets the base-2 max and *den the sum, so lse2 = *M2 + log2(*den).  A warp that
// saw no key, or scores of -inf alone, has m = -inf and weighs nothing; if all are such, *den
// is 0 and so is the output (unless a v that weighs 0 is not finite).
template <int D>
__device__ __forceinline__ float cta_merge(const MergeArea &r, int G, int h, int d, float *M2,
                                           float *den) {
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kConsumerWarps; ++w) M = fmaxf(M, r.m[w * kMaxGroup + h]);
  float num = 0.f, dn = 0.f;
#pragma unroll
  for (int w = 0; w < kConsumerWarps; ++w) {
    const float wt = dev::ex2(r.m[w * kMaxGroup + h] - softmax_ref(M));
    num += wt * r.o[(w * G + h) * D + d];
    dn += wt * r.l[w * kMaxGroup + h];
  }
  *M2 = M;
  *den = dn;
  return dn == 0.f ? num : num / dn;
}

__device__ __forceinline__ uint16_t to_bf16(float x) {
  return (uint16_t)(dev::pack_bf16x2(x, 0.f) & 0xffffu);
}

// Merges the n partition results of one query head -- row p: normalised output
// o_rows[p*D .. p*D+D) and natural-log lse_rows[p] -- into bf16 dst[0 .. D).  One warp:
// each lane owns D/32 dims; partitions are read 8 at a time with all loads in flight
// and folded in with the online-softmax rule.  Loads bypass L1 (__ldcg): the rows were
// written by other CTAs.
template <int D>
__device__ __forceinline__ void merge_rows(uint16_t *dst, const float *o_rows,
                                           const float *lse_rows, int n, int lane) {
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
        lk[u] = __ldcg(lse_rows + k) * kLog2e;
        const float *src = o_rows + (int64_t)k * D + lane * VPL;
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
  if constexpr (VPL == 2) {
    *reinterpret_cast<uint32_t *>(d) = dev::pack_bf16x2(acc[0] * inv, acc[1] * inv);
  } else {
    *reinterpret_cast<uint2 *>(d) = make_uint2(dev::pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                              dev::pack_bf16x2(acc[2] * inv, acc[3] * inv));
  }
}

}  // namespace pkv
