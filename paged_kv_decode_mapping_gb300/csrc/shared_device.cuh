// shared_device.cuh -- device pieces of the shared-prefix decode, used by its two kernels: who
// belongs to which group, how a sequence is cut, and the merge of its partial results.
#pragma once

#include "decode_device.cuh"

namespace pkv {

// One group of `a`'s list per lane, `c` the first: where it begins and how long it is, made
// disjoint and in range whatever the list holds (a group begins no earlier than every group
// before it ended), so that both kernels see the same groups.  `carry`: the furthest end so
// far, over all groups before c (0 at first).  A group that had to be moved or cut is flagged.
__device__ __forceinline__ void disjoint_group(const int32_t *start, int num, int total, int max_len,
                                               int c, int lane, int &carry, int &s, int &len) {
  const int i = c + lane;
  int s0 = 0, e0 = 0, e = 0;
  if (i < num) {
    s0 = __ldg(start + i);
    e0 = __ldg(start + i + 1);
    e = min(max(e0, 0), total);
  }
  int far = e;  // the furthest end up to this lane
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, far, x);
    if (lane >= x) far = max(far, y);
  }
  int before = __shfl_up_sync(0xffffffffu, far, 1);
  before = max(lane > 0 ? before : 0, carry);
  carry = max(carry, __shfl_sync(0xffffffffu, far, 31));
  s = min(max(max(s0, 0), before), total);
  len = min(max(e - s, 0), max_len);
  if (i < num && (s != s0 || s + len != e0)) raise_error(PKV_DEVERR_CONTEXT_LEN);
}

// How a call cuts its sequences (kernel arguments of both kernels).
struct SharedCut {
  int32_t max_blocks, block_size, log2_bs, max_prefix, max_suffix;
  int32_t split_keys;        // prefix keys behind one partial row
  int32_t partition_tokens;  // own tokens behind one
  int32_t n_rows;            // partial rows of a (sequence, head): the prefix's, then its own
};

// The whole pages of a prefix length, clamped.
__device__ __forceinline__ int shared_pages(const SharedCut &c, int prefix) {
  const int cap = (int)min((int64_t)c.max_blocks * c.block_size, (int64_t)c.max_prefix);
  return min(max(prefix, 0), cap) >> c.log2_bs << c.log2_bs;
}
// A context length, clamped to the table and to max_suffix tokens past the prefix.
__device__ __forceinline__ int shared_len(const SharedCut &c, int L, int skip) {
  const int64_t cap = min((int64_t)c.max_blocks * c.block_size, (int64_t)skip + c.max_suffix);
  return (int)min((int64_t)max(L, 0), cap);
}
__device__ __forceinline__ int prefix_rows(const SharedCut &c, int skip) {
  return (skip + c.split_keys - 1) / c.split_keys;
}
__device__ __forceinline__ int own_rows(const SharedCut &c, int L, int skip) {
  return (max(L - skip, 0) + c.partition_tokens - 1) / c.partition_tokens;
}

// Merges n partial rows of one query head (as merge_rows, 16 in flight) into bf16 dst[0 .. D).
// Rows without keys hold lse = -inf, and nothing at all gives zeros.  One warp.
template <int D>
__device__ __forceinline__ void merge_partials(uint16_t *dst, const float *o_rows,
                                               const float *lse_rows, int n, int lane) {
  constexpr int VPL = D / 32, kFly = 16;
  float M = -INFINITY, den = 0.f, acc[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) acc[v] = 0.f;
  for (int k0 = 0; k0 < n; k0 += kFly) {
    float lk[kFly], ov[kFly][VPL];
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      const int k = k0 + u;
      lk[u] = -INFINITY;
#pragma unroll
      for (int v = 0; v < VPL; ++v) ov[u][v] = 0.f;
      if (k < n) {
        lk[u] = __ldcg(lse_rows + k) * kLog2e;
        const float *src = o_rows + (int64_t)k * D + lane * VPL;
        if constexpr (VPL == 2) {
          const float2 t = __ldcg(reinterpret_cast<const float2 *>(src));
          ov[u][0] = t.x;
          ov[u][1] = t.y;
        } else {
          const float4 t = __ldcg(reinterpret_cast<const float4 *>(src));
          ov[u][0] = t.x;
          ov[u][1] = t.y;
          ov[u][2] = t.z;
          ov[u][3] = t.w;
        }
      }
    }
    float mb = lk[0];
#pragma unroll
    for (int u = 1; u < kFly; ++u) mb = fmaxf(mb, lk[u]);
    const float Mn = fmaxf(M, mb);
    if (Mn == -INFINITY) {  // no keys so far (a NaN among the rows is kept)
#pragma unroll
      for (int u = 0; u < kFly; ++u)
        if (lk[u] != -INFINITY) den = lk[u];
      continue;
    }
    const float sc = dev::ex2(M - Mn);
    den *= sc;
#pragma unroll
    for (int v = 0; v < VPL; ++v) acc[v] *= sc;
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      const float wt = dev::ex2(lk[u] - Mn);
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

// The same for the `heads` consecutive heads of one (sequence, kv head), each with n <= 32
// partial rows `stride` rows apart: a few heads at a time, their rows in flight under the
// weights (a part's weight in the lane of its number).
template <int D>
__device__ __forceinline__ void merge_heads(uint16_t *dst, const float *o_rows, const float *lse_rows,
                                            int heads, int stride, int n, int lane) {
  constexpr int VPL = D / 32, kHeads = D == 64 ? 4 : 2, kFly = 4;
  for (int h0 = 0; h0 < heads; h0 += kHeads) {
    float l[kHeads], w[kHeads], ov[kHeads][kFly][VPL], acc[kHeads][VPL];
    auto load = [&](int k0) {
#pragma unroll
      for (int j = 0; j < kHeads; ++j)
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
#pragma unroll
          for (int v = 0; v < VPL; ++v) ov[j][u][v] = 0.f;
          if (h0 + j < heads && k0 + u < n) {
            const float *src = o_rows + ((int64_t)(h0 + j) * stride + k0 + u) * D + lane * VPL;
            if constexpr (VPL == 2) {
              const float2 t = __ldcg(reinterpret_cast<const float2 *>(src));
              ov[j][u][0] = t.x;
              ov[j][u][1] = t.y;
            } else {
              const float4 t = __ldcg(reinterpret_cast<const float4 *>(src));
              ov[j][u][0] = t.x;
              ov[j][u][1] = t.y;
              ov[j][u][2] = t.z;
              ov[j][u][3] = t.w;
            }
          }
        }
    };
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      l[j] = -INFINITY;
      if (h0 + j < heads && lane < n) l[j] = __ldcg(lse_rows + (int64_t)(h0 + j) * stride + lane) * kLog2e;
#pragma unroll
      for (int v = 0; v < VPL; ++v) acc[j][v] = 0.f;
    }
    load(0);
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      float m = l[j];
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
      if (m == -INFINITY) m = 0.f;  // no key at all: weights of 0
      const float p = dev::ex2(l[j] - m);
      float den = p;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) den += __shfl_xor_sync(0xffffffffu, den, x);
      w[j] = den == 0.f ? 0.f : p / den;
    }
    for (int k0 = 0; k0 < n; k0 += kFly) {
      if (k0 > 0) load(k0);
#pragma unroll
      for (int j = 0; j < kHeads; ++j)
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
          const float wk = __shfl_sync(0xffffffffu, w[j], (k0 + u) & 31);
#pragma unroll
          for (int v = 0; v < VPL; ++v)
            if (k0 + u < n) acc[j][v] = fmaf(wk, ov[j][u][v], acc[j][v]);
        }
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      if (h0 + j >= heads) continue;
      uint16_t *d = dst + (int64_t)(h0 + j) * D + lane * VPL;
      if constexpr (VPL == 2)
        *reinterpret_cast<uint32_t *>(d) = dev::pack_bf16x2(acc[j][0], acc[j][1]);
      else
        *reinterpret_cast<uint2 *>(d) = make_uint2(dev::pack_bf16x2(acc[j][0], acc[j][1]),
                                                  dev::pack_bf16x2(acc[j][2], acc[j][3]));
    }
  }
}

}  // namespace pkv
