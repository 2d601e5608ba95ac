// pkv_shared.cu -- decode attention of sequences that share a prefix's pages.
//
// For sequence b of a group whose first n_g tokens lie in the same pages:
//   (o_p, lse_p) over keys [0, n_g),  (o_s, lse_s) over its own keys [n_g, L_b),
//   out = (e^lse_p o_p + e^lse_s o_s) / (e^lse_p + e^lse_s).
// The prefix half is a matrix product: the group's query rows (sequence, head of the kv
// head's group) against the prefix's keys, each page read once for up to 128 rows
// (pkv_tiles.cu); its splits leave (o, lse) partials.  The other half, tail_kernel below,
// streams each sequence's own keys like the decode kernel does.  It is a programmatic
// dependent of the first, so that its CTAs run beside the prefix's, on the SMs these leave,
// and only store their parts.  Its last CTAs merge, a warp for a few heads of a sequence: they
// wait for the prefix's grid and for the sequence's own parts.  Measured: 64 sequences of 1 to
// 1024 own keys over 8192 shared ones (24 / 8 heads of 128) 37.5 us, of which the prefix's
// CTAs, 64 of them, run for 29; without sharing 258 us.  (Merged by whichever part came last,
// by tickets, the last tile CTA of a group had 126 rows to merge alone, 7 us; merged by each
// tail CTA after waiting for the prefix, the tail held its SMs until the prefix was done.)
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "shared_device.cuh"

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
  uint32_t *counters;           // [B][Hkv] own parts stored, then runs merged; zero between calls
  int64_t num_blocks;
  int32_t num_seqs, num_groups, num_q_heads, num_kv_heads, group, box_rows;
  int32_t parts, tail_ctas;     // own parts at most; CTAs ahead of the merging ones
  int32_t merge_heads;          // heads a merging warp takes at a time
  int32_t sorted;               // the longest tails first (num_seqs <= kSortSeqs)
  float scale_log2;
  SharedCut cut;
};

// Stages of the ring and CTAs per SM.  At head_dim 128 three stages and two CTAs; with more
// CTAs than those hold at once, two stages and three: their starts and ends, 5 us of 12, lie
// under the others' streams (64 sequences of 1 to 1024 own keys over 8192: 42.5 against 37.5
// us, and without the order by length below either 47.5; 16 of 1 to 256, which all fit: 55.0
// against 56.3 us).
constexpr int tail_stages(int d, bool many) { return d == 64 ? 4 : many ? 2 : 3; }
constexpr int tail_occupancy(int d, int stages) { return d == 64 || stages == 2 ? 3 : 2; }
constexpr size_t tail_smem(int d, int stages) {
  return 1024 + (size_t)stages * 2 * kChunk * d * 2 + stages * 16 + 16 + (size_t)kMaxGroup * d * 2;
}
constexpr size_t kTailStatic = 1024;  // of the kernel's own, at most
static_assert(3 * (tail_smem(64, 4) + kTailStatic + 1024) <= 228 * 1024 &&
                  3 * (tail_smem(128, 2) + kTailStatic + 1024) <= 228 * 1024 &&
                  2 * (tail_smem(128, 3) + kTailStatic + 1024) <= 228 * 1024,
              "tail CTAs per SM");

constexpr int kSortSeqs = kThreads;  // one sequence per thread

// One CTA per (sequence, kv head, partition of P tokens of the sequence's own keys): the
// decode kernel's producer ring and consumer warps from the first key past the prefix; then
// the CTAs that merge.  These are fewer than the CTAs that fit at once, so that they cannot
// keep out the ones they wait for, and every wait is bounded.
//
// With more CTAs than fit at once the longest sequences go first, so that none of them starts
// when the others end (64 sequences of 1 to 1024 own keys over 8192 shared ones: in the order of
// the batch 42.4 against 37.5 us).
template <int D, int STAGES>
__global__ void __launch_bounds__(kThreads, tail_occupancy(D, STAGES))
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
  uint8_t *const q_area = base_ptr + STAGES * kStageBytes + STAGES * 16 + 16;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ __align__(16) uint32_t s_tail[kSortSeqs];
  __shared__ int s_pick[3];
  // Length and prefix of sequence `seq`, the same or (each) another one per lane; whole warps.
  auto sizes = [&](int seq, bool each, int &L, int &skip) {
    const int given = seq < a.num_seqs ? __ldg(a.context_lens + seq) : 0;
    skip = 0;
    for (int c = 0, carry = 0; c < a.num_groups; c += 32) {
      int s, len;
      const int p = c + lane < a.num_groups ? __ldg(a.prefix_lens + c + lane) : 0;
      disjoint_group(a.group_start, a.num_groups, a.num_seqs, a.num_seqs, c, lane, carry, s, len);
      // the groups that hold it, or (each) all of them in turn
      unsigned look = __ballot_sync(0xffffffffu, each ? c + lane < a.num_groups : s <= seq && seq < s + len);
      for (; look; look &= look - 1) {
        const int i = __ffs(look) - 1;
        const int si = __shfl_sync(0xffffffffu, s, i), li = __shfl_sync(0xffffffffu, len, i);
        const int pi = __shfl_sync(0xffffffffu, p, i);
        if (si <= seq && seq < si + li) skip = shared_pages(a.cut, pi);
      }
    }
    L = shared_len(a.cut, given, skip);
    return L == given;
  };
  if ((int)blockIdx.x >= a.tail_ctas) {
    // ------------------------------------------------------------- merging CTAs
    const int first = ((int)blockIdx.x - a.tail_ctas) * (kThreads / 32) + warp;
    const int step = ((int)gridDim.x - a.tail_ctas) * (kThreads / 32);
    bool waited = false;
    const int runs = (a.group + a.merge_heads - 1) / a.merge_heads;  // runs of heads in a unit
    for (int64_t task = first; task < (int64_t)a.num_seqs * a.num_kv_heads * runs; task += step) {
      const int unit = (int)(task / runs), h0 = (int)(task % runs) * a.merge_heads;
      const int heads = min(a.merge_heads, a.group - h0);
      const int seq = unit / a.num_kv_heads, g = unit - seq * a.num_kv_heads;
      int L, skip;
      (void)sizes(seq, false, L, skip);
      const int n_tail = own_rows(a.cut, L, skip), n = prefix_rows(a.cut, skip) + n_tail;
      const int64_t row = (int64_t)seq * a.num_q_heads + g * a.group + h0;
      if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the prefix's rows
      waited = true;
      uint32_t *const counter = a.counters + unit;
      if (n_tail > 0 && dev::ld_acquire(counter) < (unsigned)n_tail) {
        const uint64_t t0 = dev::globaltimer_ns();
        uint32_t tries = 0;
        while (dev::ld_acquire(counter) < (unsigned)n_tail)
          if ((++tries & 63u) == 0 && dev::globaltimer_ns() - t0 > 2000000000ull) {
            raise_error(PKV_DEVERR_TIMEOUT);
            break;
          }
      }
      __syncwarp();
      uint16_t *const dst = a.out + row * D;
      const float *const o = a.o_part + row * a.cut.n_rows * D, *const lse = a.lse_part + row * a.cut.n_rows;
      if (heads > 1 && n <= 32)
        merge_heads<D>(dst, o, lse, heads, a.cut.n_rows, n, lane);
      else
        for (int h = 0; h < heads; ++h)
          merge_partials<D>(dst + h * D, o + (int64_t)h * a.cut.n_rows * D, lse + h * a.cut.n_rows, n, lane);
      // the unit's last run to be merged leaves its counter ready for the next call
      if (n_tail > 0 && lane == 0 && atomicAdd(counter, 1u) + 1 == (unsigned)(n_tail + runs)) *counter = 0u;
    }
    // (Every warp here waits for the prefix's grid, so this one does not end before it.)
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int part = (int)blockIdx.x % a.parts, g = (int)blockIdx.x / a.parts % a.num_kv_heads;
  int b = (int)blockIdx.x / (a.parts * a.num_kv_heads), L, skip;
  bool good;
  if (a.sorted) {  // the b-th longest tail
    good = sizes(tid, true, L, skip);
    // one key each: the chunks, then the first of equals; past the last sequence the least
    const uint32_t mine = tid < a.num_seqs
        ? (uint32_t)min((max(L - skip, 0) + kChunk - 1) / kChunk, 0x7fffff) << 8 | (255u - tid)
        : 0u;
    s_tail[tid] = mine;
    __syncthreads();
    if (tid < a.num_seqs) {
      int rank = 0;
#pragma unroll 4
      for (int i = 0; i < a.num_seqs; i += 4) {
        const uint4 k = *reinterpret_cast<const uint4 *>(s_tail + i);
        rank += (k.x > mine) + (k.y > mine) + (k.z > mine) + (k.w > mine);
      }
      if (rank == b) {
        s_pick[0] = tid;
        s_pick[1] = L;
        s_pick[2] = skip;
        if (!good && part == 0 && g == 0) raise_error(PKV_DEVERR_CONTEXT_LEN);
      }
    }
    __syncthreads();
    b = s_pick[0];
    L = s_pick[1];
    skip = s_pick[2];
  } else {
    good = sizes(b, false, L, skip);
    if (!good && tid == 0 && part == 0 && g == 0) raise_error(PKV_DEVERR_CONTEXT_LEN);
  }
  const int64_t head0 = (int64_t)b * a.num_q_heads + g * a.group;
  if (tid < a.group * D / 8)  // the group's query rows
    *reinterpret_cast<uint4 *>(q_area + tid * 16) =
        __ldg(reinterpret_cast<const uint4 *>(a.q + head0 * D) + tid);
  const int n_pre = prefix_rows(a.cut, skip), n_tail = own_rows(a.cut, L, skip);
  if (part >= n_tail) return;
  const int t_begin = skip + part * a.cut.partition_tokens;
  const int t_end = min(t_begin + a.cut.partition_tokens, L);
  const int n_chunks = (t_end - t_begin + kChunk - 1) / kChunk;

  if (tid == 0) {
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      dev::mbar_init(bar_full + 8 * s, 1);
      dev::mbar_init(bar_empty + 8 * s, kConsumerWarps);
    }
    *s_flag = 0;
    dev::fence_mbar_init();
  }
  __syncthreads();

  if (warp == kConsumerWarps) {
    // ------------------------------------------------------------- producer warp
    const uint64_t policy = dev::policy_evict_first();
    const int rb = a.box_rows;
    const uint32_t box_bytes = (uint32_t)rb * 128u;
    const int32_t *trow = a.block_tables + (int64_t)b * a.cut.max_blocks;
    const int lb_last = (t_end - 1) >> a.cut.log2_bs;
    int win = t_begin >> a.cut.log2_bs;
    int tb = win + lane <= lb_last ? __ldg(trow + win + lane) : 0;
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
      const int lb_hi = (k0 + (nbox - 1) * rb) >> a.cut.log2_bs;
      if (lb_hi >= win + 32) {  // slide the table window
        win = k0 >> a.cut.log2_bs;
        tb = (win + lane <= lb_last) ? __ldg(trow + win + lane) : 0;
      }
      const int key = k0 + lane * rb;
      const int src = min(max((key >> a.cut.log2_bs) - win, 0), 31);
      const int64_t phys_raw = __shfl_sync(0xffffffffu, tb, src);
      if (lane == 0) dev::mbar_arrive_expect_tx(bar_full + 8 * s, 2u * nbox * box_bytes * (D / 64));
      __syncwarp();
      if (lane < nbox) {
        int64_t phys = phys_raw;
        if (phys < 0 || phys >= a.num_blocks) {
          raise_error(PKV_DEVERR_BLOCK_ID);
          phys = 0;
        }
        const int off = key & (a.cut.block_size - 1);
        const int32_t row = (int32_t)((phys * a.num_kv_heads + g) * a.cut.block_size + off);
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
    for (int i = tid; i < a.group * D; i += kConsumers) {
      const int h = i / D, d = i - h * D;
      float M2, den;
      const float val = cta_merge<D>(r, a.group, h, d, &M2, &den);
      const int64_t row = (head0 + h) * a.cut.n_rows + n_pre + part;
      a.o_part[row * D + d] = val;
      if (d == 0) a.lse_part[row] = (M2 + log2f(den)) * kLn2;
    }
    consumer_bar();  // orders every thread's stores before the release
    if (tid == 0 && !*s_flag) dev::red_add_release(a.counters + (int64_t)b * a.num_kv_heads + g, 1u);
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

bool g_tail_attr[kMaxDevices][3];
std::atomic<int> g_mode{PKV_SHARED_AUTO};  // PKV_SHARED_*, process-wide

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// How a call is cut: split_keys prefix keys per tile CTA, partition_tokens tail tokens per
// tail CTA, and the workspace.
struct SharedPlan {
  int32_t split_keys, splits, partition_tokens, parts, n_rows, sorted, merge_ctas, merge_heads;
  int32_t plain, plain_len;  // whether the plain decode takes the call by its sizes, and its length
  int32_t stages;  // of the tail's ring
  int64_t tiles;  // row tiles over all groups, at most
  size_t partials, o_part, lse_part, total;
};

// Partial rows that no call of up to these sizes passes, whatever cut it takes: never fewer for
// larger sizes, though a cut may well have fewer rows for them (64 sequences take 9 splits where
// 42, one row tile, take 19), so that a workspace sized by the largest sizes serves all others.
//  * the prefix's: n > 1 splits only where the tiles' CTAs all fit at once, so with t row tiles
//    at most tile_seqs * t sequences, sms / (t * hkv) rows each;
//  * the own keys': parts of at least 256 tokens, but for a single part.
int64_t most_rows(int32_t num_seqs, int32_t hq, int32_t hkv, bool groups, int64_t blocks, int32_t mlen,
                  int sms) {
  const int64_t tile_seqs = kTileRows / (hq / hkv), units = (int64_t)num_seqs * hkv;
  int64_t seq_rows = num_seqs;  // one split
  const int64_t tiles = groups ? std::min<int64_t>((num_seqs + tile_seqs - 1) / tile_seqs, sms / hkv) : 0;
  for (int64_t t = 1; t <= tiles; ++t)
    seq_rows = std::max(seq_rows, std::min<int64_t>(t * tile_seqs, num_seqs) *
                                      std::min<int64_t>({std::max<int64_t>(blocks, 1), 1024, sms / (t * hkv)}));
  return seq_rows * hq + units * (hq / hkv) * (((int64_t)mlen + 255) / 256);
}

// The words that are zero between calls -- the plain decode's two and a counter per (sequence,
// kv head) -- have the front of the workspace to themselves, as long for all calls of up to
// this many: no call's partial rows lie where another's counters are, whatever their sizes.
constexpr size_t kWords = 65536;

// The longest prefix and the longest own part: what a row stands for, and a place in a
// sequence with one such step added, stay within 31 bits.
constexpr int32_t kMaxSharedLen = 1 << 29;

SharedPlan shared_plan(int32_t num_seqs, int32_t hq, int32_t hkv, int32_t d, int32_t num_groups,
                       int32_t max_prefix, int32_t max_suffix, int sms) {
  SharedPlan p;
  const int32_t groups = std::min(num_groups, num_seqs);
  const int64_t tile_seqs = kTileRows / (hq / hkv);  // sequences of a tile
  p.tiles = groups > 0 ? (num_seqs - groups) / tile_seqs + groups : 0;  // at most, however they are cut
  const int64_t units = p.tiles * hkv;
  const int64_t blocks = groups > 0 ? ((int64_t)max_prefix + kTileKeys - 1) / kTileKeys : 0;
  const int32_t mlen = std::max(max_suffix, 1);
  // The prefix's CTAs take an SM each; the tail's run beside them on the others, and take
  // theirs over.  So: as many splits, and tail parts as short, as make the longest of a tile
  // CTA's time, the longest part's and the whole work over the SMs the shortest.  Measured, in
  // us, with the merge that follows: a tile CTA 8.1 and, per block of 128 keys, what the TMA
  // unit needs for its boxes of 16 rows (63 cycles each and 64 bytes a cycle at 1.93 GHz) or
  // the HBM for all CTAs' (6.5 TB/s); a part 8.7 and 31 KB a us at head_dim 64, 46 at 128, if
  // it starts at once.  Of an SM, a part takes 4.5 and 34 KB a us, 2 or 3 at a time, all of
  // them at most the HBM's.  Own lengths are taken at half the longest.  (The sizes do not tell the
  // block size: `tma` is for 16 rows.  By the same formula a block takes 2.6 us at 8 rows, head_dim
  // 128, and 0.79 at 64, so that longer pages get more splits than they need.)  (Parts as long as the
  // plain decode's, for 16 sequences of 1 to 512 own keys over 2048, 32 / 8 heads of 64: 11.6
  // us; chosen so, 10.0.)
  const double tma = d == 64 ? 0.79 : 1.57;
  double best = 0, shared = 0;  // the choice's cost, and its time with the launch's 3 us once
  int occ = 0;
  const int32_t longest = paged_decode_plan(num_seqs, hq, hkv, d, mlen, sms);
  for (int32_t P = longest, next = 256;; P = next, next *= 2) {
    const int32_t parts = (mlen + P - 1) / P;
    const double tail_ctas = (double)num_seqs * hkv * parts;
    const int32_t stages = tail_stages(d, tail_ctas > (double)sms * tail_occupancy(d, tail_stages(d, false)));
    const int fit = tail_occupancy(d, stages);
    const double own = 0.5 * mlen / parts * d * 4;  // bytes of a tail CTA
    const double tail = std::max(tail_ctas * (4.5 + own / 34e3) / fit, tail_ctas * own / 6.5e6 * sms);
    const double part = 8.7 + (double)std::min(P, mlen) * d * 4 / (d == 64 ? 31e3 : 46e3);
    for (int64_t n = 1; n <= std::min<int64_t>(blocks, 1024) || n == 1; ++n) {
      const double ctas = (double)units * n;
      if (n > 1 && ctas > sms) break;
      const double hbm = (double)groups * hkv * n * kTileKeys * d * 4 / 6.5e6 * std::min(1., sms / std::max(ctas, 1.));
      const double tile = 8.1 + (double)((blocks + n - 1) / n) * std::max(tma, hbm);
      const double late = ctas + tail_ctas / fit <= sms ? 0 : 5;  // or the tail begins after it
      // (of equals, the one with the prefix done first)
      const double t = std::max({tile, part, (tail + std::min<double>(ctas, sms) * tile) / sms}) + late + 0.1 * tile;
      if (best == 0 || t < (P == longest ? best : 0.97 * best)) {
        best = t;
        p.splits = (int32_t)n;
        p.partition_tokens = P;
        p.parts = parts;
        p.stages = stages;
        occ = fit;
        shared = std::max({tile, part, 3 + (tail + ctas * (tile - 3)) / sms}) + late;
      }
    }
    if (next >= longest) break;
  }
  const double tail_ctas = (double)num_seqs * hkv * p.parts;
  p.split_keys = (int32_t)(std::max<int64_t>((blocks + p.splits - 1) / p.splits, 1) * kTileKeys);
  p.sorted = num_seqs <= kSortSeqs && mlen >= 512 && units * p.splits + tail_ctas / occ > sms;
  p.n_rows = p.splits + p.parts;
  // A warp per head, or per as many heads as keep the merging CTAs within half of those that
  // fit at once.
  const int64_t warps = kThreads / 32, cap = (int64_t)sms * occ / 2 * warps;
  const int32_t group = hq / hkv;
  int64_t tasks;
  for (p.merge_heads = 1;; ++p.merge_heads) {
    tasks = (int64_t)num_seqs * hkv * ((group + p.merge_heads - 1) / p.merge_heads);
    if (tasks <= cap || p.merge_heads == group) break;
  }
  p.merge_ctas = (int32_t)((std::min(tasks, cap) + warps - 1) / warps);
  const size_t prow = (size_t)num_seqs * hq * p.n_rows;
  p.partials = up256((std::max((size_t)num_seqs * hkv, kWords) + 2) * 4);
  p.o_part = p.partials;
  p.lse_part = p.o_part + up256(prow * d * sizeof(float));
  p.plain_len = (int32_t)std::min<int64_t>((int64_t)max_prefix + max_suffix, 0x7fffffff);
  const size_t most = (size_t)most_rows(num_seqs, hq, hkv, groups > 0, blocks, mlen, sms);
  p.total = p.partials + std::max(up256(most * d * sizeof(float)) + up256(most * sizeof(float)),
                                  decode_workspace_bound(num_seqs, hq, hkv, d, p.plain_len, sms));
  // The plain decode, one launch, is the faster one where little is read twice, and where
  // there are so many short groups that their CTAs' starts cost more than the reads (the last
  // term: tasks a merging warp has after its second, 14 us each).  Plain: 5.5 us and every key
  // at 7.5 TB/s, shared pages coming from L2 in part.  Measured, shared against plain, us: 3
  // sequences over 512 tokens 8.3, 7.5; 16 over 2048 10.0, 12.7; 64 over 8192 38, 258; groups
  // of 4 over 1000 tokens (32 / 8 heads of 64), 16 of them 20, 30, 64 of them 71, 76, 256 of
  // them 339, 276; 256 groups of 16 over 250 tokens 745, 366.
  shared += std::max(0., (double)tasks / cap - 2) * 14;
  const double plain = 5.5 + (double)num_seqs * hkv * (max_prefix + 0.5 * mlen) * d * 4 / 7.5e6;
  p.plain = plain < 0.9 * shared;
  return p;
}

template <int D, int S>
int launch_tail(const CUtensorMap &tmk, const CUtensorMap &tmv, const TailArgs &a, dim3 grid,
                bool programmatic, cudaStream_t stream) {
  {
    std::lock_guard<std::mutex> lk(attn_mutex());
    int dev = 0;
    const int rc = current_device(&dev);
    if (rc) return rc;
    bool &set = g_tail_attr[dev][D == 64 ? 0 : S - 1];
    if (!set) {
      cudaError_t e = cudaFuncSetAttribute(tail_kernel<D, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)tail_smem(D, S));
      if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute");
      e = cudaFuncSetAttribute(tail_kernel<D, S>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
      if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute(carveout)");
      set = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = tail_smem(D, S);
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

PKV_API int32_t pkv_set_shared_prefix(int32_t mode) {
  if (mode != PKV_SHARED_AUTO && mode != PKV_SHARED_ALWAYS && mode != PKV_SHARED_NEVER)
    return set_error(PKV_ERR_UNSUPPORTED, "pkv_set_shared_prefix: unknown mode %d", mode);
  clear_error();
  return g_mode.exchange(mode);
}

PKV_API size_t paged_decode_shared_prefix_workspace_size(int32_t num_seqs, int32_t num_q_heads,
                                                         int32_t num_kv_heads, int32_t head_dim,
                                                         int32_t num_groups, int32_t max_prefix_len,
                                                         int32_t max_suffix_len) {
  if (num_groups < 0 || max_prefix_len < 0 || max_suffix_len < 0 || max_prefix_len > kMaxSharedLen ||
      max_suffix_len > kMaxSharedLen ||
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
  if (max_prefix_len > kMaxSharedLen || max_suffix_len > kMaxSharedLen)
    return set_error(PKV_ERR_UNSUPPORTED, "%s: max_prefix_len or max_suffix_len over 2^29", fn);
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
  const int64_t tail_ctas = (int64_t)p.parts * hkv * num_seqs;
  if (tail_ctas > 0x7fff0000LL || (int64_t)num_seqs * num_q_heads > 0x7fffffffLL)
    return set_error(PKV_ERR_UNSUPPORTED, "%s: too many parts", fn);
  const int mode = g_mode.load(std::memory_order_relaxed);
  if (mode == PKV_SHARED_NEVER || (mode == PKV_SHARED_AUTO && p.plain)) {
    // cut to the table: fewer tokens may take more parts, but none that the bound has no room for
    const int64_t cap = (int64_t)max_blocks_per_seq * cache->block_size;
    const int32_t len = (int32_t)std::min<int64_t>(p.plain_len, cap);
    rc = decode_attention_words(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                                len, num_seqs, num_q_heads, cache, scale,
                                static_cast<uint32_t *>(workspace),
                                static_cast<char *>(workspace) + p.partials,
                                workspace_bytes - p.partials, static_cast<cudaStream_t>(stream), fn);
    if (!rc) clear_error();
    return rc;
  }
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
  a.counters = reinterpret_cast<uint32_t *>(ws) + 2;
  a.num_blocks = cache->num_blocks;
  a.num_seqs = num_seqs;
  a.num_groups = num_groups;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = hkv;
  a.group = num_q_heads / hkv;
  a.box_rows = std::min(cache->block_size, (int32_t)kChunk);
  a.scale_log2 = scale * kLog2e;
  a.cut.max_blocks = max_blocks_per_seq;
  a.cut.block_size = cache->block_size;
  a.cut.log2_bs = ilog2(cache->block_size);
  a.cut.max_prefix = max_prefix_len;
  a.cut.max_suffix = max_suffix_len;
  a.sorted = p.sorted;
  a.cut.split_keys = p.split_keys;
  a.cut.partition_tokens = p.partition_tokens;
  a.cut.n_rows = p.n_rows;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool prefix = num_groups > 0 && max_prefix_len >= cache->block_size;
  if (prefix) {
    PrefixLaunch l;
    l.q = q;
    l.k_cache = k_cache;
    l.v_cache = v_cache;
    l.block_tables = block_tables;
    l.context_lens = context_lens;
    l.group_start = group_start;
    l.prefix_lens = prefix_lens;
    l.o_part = a.o_part;
    l.lse_part = a.lse_part;
    l.num_seqs = num_seqs;
    l.num_groups = num_groups;
    l.num_q_heads = num_q_heads;
    l.split_keys = p.split_keys;
    l.splits = p.splits;
    l.tiles = p.tiles;
    l.scale = scale;
    l.cut = &a.cut;
    if ((rc = launch_prefix(tmk, tmv, *cache, l, s))) return rc;
  }
  a.parts = p.parts;
  a.merge_heads = p.merge_heads;
  a.tail_ctas = (int32_t)tail_ctas;
  const dim3 grid((unsigned)(tail_ctas + p.merge_ctas));
  rc = D == 64         ? launch_tail<64, 4>(tmk, tmv, a, grid, prefix, s)
       : p.stages == 2 ? launch_tail<128, 2>(tmk, tmv, a, grid, prefix, s)
                       : launch_tail<128, 3>(tmk, tmv, a, grid, prefix, s);
  if (!rc) clear_error();
  return rc;
}
