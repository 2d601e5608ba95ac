// pkv_shared.cu -- decode attention of sequences that share a prefix's pages.
//
// For sequence b of a group whose first n_g tokens lie in the same pages:
//   (o_p, lse_p) over keys [0, n_g),  (o_s, lse_s) over its own keys [n_g, L_b),
//   out = (e^lse_p o_p + e^lse_s o_s) / (e^lse_p + e^lse_s).
// The prefix half is a matrix product: the group's query rows (sequence, head of the kv
// head's group) against the prefix's keys, each page read once for up to 128 rows
// (pkv_tiles.cu); its splits leave (o, lse) partials.  The other half, tail_kernel below,
// streams each sequence's own keys like the decode kernel does, and merges.  It is a
// programmatic dependent of the first: its CTAs fill the SMs as the prefix's leave them,
// and wait for the prefix's partials only before they merge.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "decode_device.cuh"

namespace pkv {

struct TailArgs {
  const uint16_t *q;            // [B][Hq][D]
  const int32_t *block_tables;  // [B][max_blocks]
  const int32_t *context_lens;  // [B]
  const int32_t *group_start;   // [num_groups + 1]
  const int32_t *prefix_lens;   // [num_groups]
  float *o_part;                // [B][Hq][n_rows][D]: the prefix's rows, then the tail's
  float *lse_part;              // [B][Hq][n_rows]
  uint16_t *out;                // [B][Hq][D]
  uint32_t *counters;           // [B][Hkv] tail partitions finished; zero between calls
  int64_t num_blocks;
  int32_t max_blocks, num_groups, max_prefix, max_suffix, num_q_heads, num_kv_heads, group;
  int32_t block_size, log2_bs, box_rows, partition_tokens, n_rows;
  int32_t row_keys;             // prefix keys behind one of its rows
  float scale_log2;
};

// The n partition results of one query head (rows of o_rows and lse_rows, as merge_rows
// takes them) and the CTA's own result (normalised own[v], base-2 own_lse; -inf: none) into
// bf16 dst[0 .. D).  One warp; 16 rows in flight.  Nothing at all gives zeros.
template <int D>
__device__ __forceinline__ void merge_rows_own(uint16_t *dst, const float *o_rows,
                                               const float *lse_rows, int n, int lane,
                                               const float (&own)[D / 32], float own_lse) {
  constexpr int VPL = D / 32, kFly = 16;
  float M = own_lse, den = own_lse == -INFINITY ? 0.f : 1.f, acc[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) acc[v] = own_lse == -INFINITY ? 0.f : own[v];
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
    if (Mn == -INFINITY) continue;  // rows without keys only, so far
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

// One CTA per (sequence, kv head, partition of P tokens of the sequence's own keys): the
// decode kernel's producer ring and consumer warps from the first key past the prefix.
// The CTA of a sequence held whole, or the last of its partitions to finish (an atomic
// ticket; nobody waits), merges the prefix's and the tail's results.
template <int D, int STAGES>
__global__ void __launch_bounds__(kThreads, split_occupancy(D))
    tail_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                const TailArgs a) {
  constexpr int kTileBytes = kChunk * D * 2;
  constexpr int kStageBytes = 2 * kTileBytes;
  constexpr int KS = D / 16;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = dev::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *const base_ptr = smem_raw + (base - raw);
  const uint32_t bar_full = base + STAGES * kStageBytes;
  const uint32_t bar_empty = bar_full + STAGES * 8;
  volatile int *const s_flag =
      reinterpret_cast<volatile int *>(base_ptr + STAGES * kStageBytes + STAGES * 16);
  volatile int *const s_last = s_flag + 1;
  uint8_t *const q_area = base_ptr + STAGES * kStageBytes + STAGES * 16 + 16;

  const int part = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t head0 = (int64_t)b * a.num_q_heads + g * a.group;
  // the group's query rows into shared memory, and the sequence's sizes, all in flight
  if (tid < a.group * D / 8)
    *reinterpret_cast<uint4 *>(q_area + tid * 16) =
        __ldg(reinterpret_cast<const uint4 *>(a.q + head0 * D) + tid);
  int L = __ldg(a.context_lens + b);
  int skip = 0;  // the prefix: 0 for a sequence of no group
  for (int c = 0; c < a.num_groups; c += 32) {
    const int i = c + lane;
    int s = 0, e = 0, p = 0;
    if (i < a.num_groups) {
      s = __ldg(a.group_start + i);
      e = __ldg(a.group_start + i + 1);
      p = __ldg(a.prefix_lens + i);
    }
    const unsigned mine = __ballot_sync(0xffffffffu, s <= b && b < e);
    if (mine) {
      skip = __shfl_sync(0xffffffffu, p, __ffs(mine) - 1);
      break;
    }
  }
  const int cap = (int)min((int64_t)a.max_blocks * a.block_size, (int64_t)0x7fffffff);
  skip = min(max(skip, 0), min(cap, a.max_prefix)) >> a.log2_bs << a.log2_bs;
  if (L < 0 || L > cap || L - skip > a.max_suffix) {
    if (tid == 0 && part == 0) raise_error(PKV_DEVERR_CONTEXT_LEN);
    L = L < 0 ? 0 : min(L, min(cap, skip + min(a.max_suffix, 0x7fffffff - skip)));
  }
  const int n_pre = (skip + a.row_keys - 1) / a.row_keys;  // the prefix's rows
  const int n_own = max(L - skip, 0);
  const int n_tail = (n_own + a.partition_tokens - 1) / a.partition_tokens;
  if (part >= max(n_tail, 1)) return;
  const int t_begin = skip + part * a.partition_tokens;
  const int t_end = min(t_begin + a.partition_tokens, max(L, skip));
  const int n_chunks = (t_end - t_begin + kChunk - 1) / kChunk;

  if (tid == 0) {
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      dev::mbar_init(bar_full + 8 * s, 1);
      dev::mbar_init(bar_empty + 8 * s, kConsumerWarps);
    }
    *s_flag = 0;
    *s_last = 0;
    dev::fence_mbar_init();
  }
  __syncthreads();

  if (warp == kConsumerWarps) {
    // ------------------------------------------------------------- producer warp
    const uint64_t policy = dev::policy_evict_first();
    const int rb = a.box_rows;
    const uint32_t box_bytes = (uint32_t)rb * 128u;
    const int32_t *trow = a.block_tables + (int64_t)b * a.max_blocks;
    const int lb_last = (t_end - 1) >> a.log2_bs;
    int win = t_begin >> a.log2_bs;
    int tb = (n_chunks > 0 && win + lane <= lb_last) ? __ldg(trow + win + lane) : 0;
    for (int c = 0; c < n_chunks; ++c) {
      const int s = c % STAGES;
      if (c >= STAGES &&
          !__all_sync(0xffffffffu, dev::mbar_wait(bar_empty + 8 * s, ((c / STAGES) - 1) & 1))) {
        if (lane == 0) {
          raise_error(PKV_DEVERR_TIMEOUT);
          *s_flag = 1;
        }
        break;
      }
      const int k0 = t_begin + c * kChunk;
      const int nk = min(kChunk, t_end - k0);
      const int nbox = (nk + rb - 1) / rb;
      const int lb_hi = (k0 + (nbox - 1) * rb) >> a.log2_bs;
      if (lb_hi >= win + 32) {  // slide the table window
        win = k0 >> a.log2_bs;
        tb = (win + lane <= lb_last) ? __ldg(trow + win + lane) : 0;
      }
      const int key = k0 + lane * rb;
      const int src = min(max((key >> a.log2_bs) - win, 0), 31);
      const int64_t phys_raw = __shfl_sync(0xffffffffu, tb, src);
      if (lane == 0) dev::mbar_arrive_expect_tx(bar_full + 8 * s, 2u * nbox * box_bytes * (D / 64));
      __syncwarp();
      if (lane < nbox) {
        int64_t phys = phys_raw;
        if (phys < 0 || phys >= a.num_blocks) {
          raise_error(PKV_DEVERR_BLOCK_ID);
          phys = 0;
        }
        const int off = key & (a.block_size - 1);
        const int32_t row = (int32_t)((phys * a.num_kv_heads + g) * a.block_size + off);
        const uint32_t dk = base + s * kStageBytes + lane * box_bytes;
        issue_box<D>(dk, dk + kTileBytes, &tmk, &tmv, row, bar_full + 8 * s, policy);
      }
      __syncwarp();
    }
  } else {
    // ----------------------------------------------------------- consumer warps
    WarpAcc<D> acc;
    acc_reset(acc);
    uint32_t qb[KS][2];
    {
      const uint32_t *qs = reinterpret_cast<const uint32_t *>(q_area);
      const int gid = lane >> 2, tig = lane & 3;
      const bool hv = gid < a.group;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qb[ks][0] = hv ? qs[gid * (D / 2) + 8 * ks + tig] : 0u;
        qb[ks][1] = hv ? qs[gid * (D / 2) + 8 * ks + 4 + tig] : 0u;
      }
    }
    for (int c = 0; c < n_chunks; ++c) {
      const int s = c % STAGES;
      if (!__all_sync(0xffffffffu, dev::mbar_wait(bar_full + 8 * s, (c / STAGES) & 1))) {
        if (lane == 0) {
          raise_error(PKV_DEVERR_TIMEOUT);
          *s_flag = 1;
        }
        break;
      }
      const int key0 = t_begin + c * kChunk + 16 * warp;
      const int nvalid = min(16, t_end - key0);
      if (nvalid > 0) {
        const uint32_t kb = base + s * kStageBytes;
        warp_tile<D>(acc, qb, kb, kb + kTileBytes, warp, lane, nvalid, a.scale_log2);
      }
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(bar_empty + 8 * s);
    }
    consumer_bar();
    MergeArea r;
    r.o = reinterpret_cast<float *>(base_ptr);
    r.m = r.o + kConsumerWarps * a.group * D;
    r.l = r.m + kConsumerWarps * kMaxGroup;
    warp_stash<D>(acc, r, a.group, warp, lane);
    consumer_bar();
    bool merge = n_tail <= 1;
    if (!merge) {
      for (int i = tid; i < a.group * D; i += kConsumers) {
        const int h = i / D, d = i - h * D;
        float M2, den;
        const float val = cta_merge<D>(r, a.group, h, d, &M2, &den);
        const int64_t row = (head0 + h) * a.n_rows + n_pre + part;
        a.o_part[row * D + d] = val;
        if (d == 0) a.lse_part[row] = (M2 + log2f(den)) * kLn2;
      }
      consumer_bar();
      if (tid == 0) {
        int last = 0;
        if (!*s_flag) {
          const unsigned old = dev::atomic_add_acq_rel(a.counters + (int64_t)b * a.num_kv_heads + g, 1u);
          last = (old + 1 == (unsigned)n_tail);
        }
        *s_last = last;
      }
      consumer_bar();
      merge = *s_last != 0;
      if (merge && tid == 0) a.counters[(int64_t)b * a.num_kv_heads + g] = 0u;
    }
    // the prefix's partials are complete and visible past this point
    if (merge) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      constexpr int VPL = D / 32;
      for (int h = warp; h < a.group; h += kConsumerWarps) {
        float own[VPL], own_lse = -INFINITY;
        if (n_tail == 1) {
          float M2, den;
#pragma unroll
          for (int v = 0; v < VPL; ++v) own[v] = cta_merge<D>(r, a.group, h, lane * VPL + v, &M2, &den);
          own_lse = M2 + log2f(den);
        } else {
#pragma unroll
          for (int v = 0; v < VPL; ++v) own[v] = 0.f;
        }
        merge_rows_own<D>(a.out + (head0 + h) * D, a.o_part + (head0 + h) * a.n_rows * D,
                          a.lse_part + (head0 + h) * a.n_rows, n_pre + (n_tail > 1 ? n_tail : 0),
                          lane, own, own_lse);
      }
    }
  }

  // ---- a timed-out wait leaves copies possibly in flight: wait for them (bounded)
  __syncthreads();
  if (tid == 0 && *s_flag) {
    for (int s = 0; s < STAGES; ++s) {
      const int c_last = s + ((n_chunks - 1 - s) / STAGES) * STAGES;
      if (c_last >= 0 && c_last < n_chunks) (void)dev::mbar_wait(bar_full + 8 * s, (c_last / STAGES) & 1);
    }
  }
}

cudaError_t read_shared_errors(uint32_t *flags, int clear) { return read_tu_errors(flags, clear); }

namespace {

bool g_tail_attr[kMaxDevices][2];

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// How a call is cut: split_keys prefix keys per tile CTA, partition_tokens tail tokens per
// tail CTA, and the workspace.
struct SharedPlan {
  int32_t split_keys, splits, cluster, partition_tokens, parts, n_rows;
  int64_t tiles;  // row tiles over all groups, at most
  size_t o_part, lse_part, total;
};

SharedPlan shared_plan(int32_t num_seqs, int32_t hq, int32_t hkv, int32_t d, int32_t num_groups,
                       int32_t max_prefix, int32_t max_suffix, int sms) {
  SharedPlan p;
  const int32_t groups = std::min(num_groups, num_seqs);
  const int64_t tile_seqs = kTileRows / (hq / hkv);  // sequences of a tile
  p.tiles = num_seqs / tile_seqs + groups;
  // About one tile CTA per SM: the prefix is cut into as many splits as that takes, in
  // clusters (measured on 152 SMs with 1 CTA each: 36 clusters of 4 fit at once, 76 of 2,
  // but only 15 of 8).
  const int64_t units = std::max<int64_t>((num_seqs + tile_seqs - 1) / tile_seqs, groups) * hkv;
  const int64_t blocks = ((int64_t)max_prefix + kTileKeys - 1) / kTileKeys;
  p.cluster = 1;
  int64_t splits = 1;
  for (int32_t c = kPrefixCluster; c > 1; c /= 2) {
    const int64_t fit = (c == 2 ? sms : sms - sms / 19) / c;  // clusters at once
    if (units > fit || blocks < c) continue;
    const int64_t n = c * std::min(fit / units, blocks / c);
    if (n <= splits) continue;
    p.cluster = c;
    splits = n;
  }
  p.split_keys = (int32_t)std::min<int64_t>(std::max<int64_t>((blocks + splits - 1) / splits, 1) * kTileKeys,
                                            1 << 29);
  p.splits = (int32_t)splits;
  const int32_t mlen = std::max(max_suffix, 1);
  p.partition_tokens = paged_decode_plan(num_seqs, hq, hkv, d, mlen, sms);
  p.parts = (mlen + p.partition_tokens - 1) / p.partition_tokens;
  p.n_rows = p.splits / p.cluster + p.parts;
  const size_t prow = (size_t)num_seqs * hq * p.n_rows;
  p.o_part = up256((size_t)num_seqs * hkv * 4);
  p.lse_part = p.o_part + up256(prow * d * sizeof(float));
  p.total = p.lse_part + up256(prow * sizeof(float));
  return p;
}

template <int D>
int launch_tail(const CUtensorMap &tmk, const CUtensorMap &tmv, const TailArgs &a, dim3 grid,
                bool programmatic, cudaStream_t stream) {
  constexpr int S = split_stages(D);
  {
    std::lock_guard<std::mutex> lk(attn_mutex());
    int dev = 0;
    const int rc = current_device(&dev);
    if (rc) return rc;
    bool &set = g_tail_attr[dev][D == 64 ? 0 : 1];
    if (!set) {
      cudaError_t e = cudaFuncSetAttribute(tail_kernel<D, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)split_smem(D));
      if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute");
      e = cudaFuncSetAttribute(tail_kernel<D, S>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
      if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute(carveout)");
      set = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = split_smem(D);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = programmatic ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tail_kernel<D, S>, tmk, tmv, a);
  return e == cudaSuccess ? PKV_OK : cuda_error(e, "tail_kernel launch");
}

int sm_count(int *sms) {
  std::lock_guard<std::mutex> lk(attn_mutex());
  return device_sms(sms);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

PKV_API size_t paged_decode_shared_prefix_workspace_size(int32_t num_seqs, int32_t num_q_heads,
                                                         int32_t num_kv_heads, int32_t head_dim,
                                                         int32_t num_groups, int32_t max_prefix_len,
                                                         int32_t max_suffix_len) {
  if (num_groups < 0 || max_prefix_len < 0 || max_suffix_len < 0 ||
      paged_decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, std::max(max_suffix_len, 1), 1) <= 0)
    return 0;
  int sms = 0;
  if (sm_count(&sms) != PKV_OK || sms <= 0) sms = 152;
  return shared_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, num_groups, max_prefix_len,
                     max_suffix_len, sms).total;
}

PKV_API int paged_decode_shared_prefix_attention(
    pkv_bf16 *out, const pkv_bf16 *q, const pkv_bf16 *k_cache, const pkv_bf16 *v_cache,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens,
    const int32_t *group_start, const int32_t *prefix_lens, int32_t num_groups,
    int32_t max_prefix_len, int32_t max_suffix_len, int32_t num_seqs, int32_t num_q_heads,
    const pkv_cache_desc *cache, float scale, void *workspace, size_t workspace_bytes,
    void *stream) {
  const char *const fn = "paged_decode_shared_prefix_attention";
  int rc = check_decode(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                        std::max(max_prefix_len, max_suffix_len), num_seqs, num_q_heads, cache, fn);
  if (rc) return rc;
  if (num_groups < 0 || max_prefix_len < 0 || max_suffix_len < 0)
    return set_error(PKV_ERR_SHAPE, "%s: negative num_groups, max_prefix_len or max_suffix_len", fn);
  if (num_seqs == 0) {
    clear_error();
    return PKV_OK;
  }
  if (!out || (num_groups > 0 && (!group_start || !prefix_lens)))
    return set_error(PKV_ERR_NULL, "%s: NULL out, group_start or prefix_lens", fn);
  if (reinterpret_cast<uintptr_t>(out) & 7u)
    return set_error(PKV_ERR_ALIGN, "%s: out must be 8-byte aligned", fn);
  const int D = cache->head_dim, hkv = cache->num_kv_heads;
  int sms = 0;
  if ((rc = sm_count(&sms))) return rc;
  const SharedPlan p = shared_plan(num_seqs, num_q_heads, hkv, D, num_groups, max_prefix_len,
                                   max_suffix_len, sms);
  if (!workspace || workspace_bytes < p.total)
    return set_error(PKV_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, workspace_bytes,
                     p.total);
  if (!aligned16(workspace))
    return set_error(PKV_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
  CUtensorMap tmk, tmv;
  {
    std::lock_guard<std::mutex> lk(attn_mutex());
    if ((rc = maps_for(k_cache, v_cache, *cache, &tmk, &tmv))) return rc;
  }
  char *const ws = static_cast<char *>(workspace);
  TailArgs a = {};
  a.q = q;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.group_start = group_start;
  a.prefix_lens = prefix_lens;
  a.o_part = reinterpret_cast<float *>(ws + p.o_part);
  a.lse_part = reinterpret_cast<float *>(ws + p.lse_part);
  a.out = out;
  a.counters = reinterpret_cast<uint32_t *>(ws);
  a.num_blocks = cache->num_blocks;
  a.max_blocks = max_blocks_per_seq;
  a.num_groups = num_groups;
  a.max_prefix = max_prefix_len;
  a.max_suffix = max_suffix_len;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = hkv;
  a.group = num_q_heads / hkv;
  a.block_size = cache->block_size;
  a.log2_bs = ilog2(cache->block_size);
  a.box_rows = std::min(cache->block_size, (int32_t)kChunk);
  a.partition_tokens = p.partition_tokens;
  a.n_rows = p.n_rows;
  a.row_keys = p.split_keys * p.cluster;
  a.scale_log2 = scale * kLog2e;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool prefix = num_groups > 0 && max_prefix_len >= cache->block_size;
  if (prefix) {
    PrefixLaunch l;
    l.q = q;
    l.block_tables = block_tables;
    l.context_lens = context_lens;
    l.group_start = group_start;
    l.prefix_lens = prefix_lens;
    l.o_part = a.o_part;
    l.lse_part = a.lse_part;
    l.num_seqs = num_seqs;
    l.num_groups = num_groups;
    l.max_blocks = max_blocks_per_seq;
    l.max_prefix = max_prefix_len;
    l.num_q_heads = num_q_heads;
    l.split_keys = p.split_keys;
    l.splits = p.splits;
    l.cluster = p.cluster;
    l.n_rows = p.n_rows;
    l.tiles = p.tiles;
    l.scale = scale;
    if ((rc = launch_prefix(tmk, tmv, *cache, l, s))) return rc;
  }
  const dim3 grid((unsigned)p.parts, (unsigned)hkv, (unsigned)num_seqs);
  rc = D == 64 ? launch_tail<64>(tmk, tmv, a, grid, prefix, s) : launch_tail<128>(tmk, tmv, a, grid, prefix, s);
  if (!rc) clear_error();
  return rc;
}
