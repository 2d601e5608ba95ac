// pkv_decode_q8.cu -- single-token attention over the 8-bit paged cache, and the whole step.
//
//   s_t = scale * ks[n] * <q, ck_t>,   out = sum_t softmax(s)_t * vs[n] * cv_t,   n = t's page
//
// HBM-bound: 2 bytes of K and V per (key, dim) feed G = Hq / Hkv query heads.  What differs from
// the bf16 decode:
//  * Codes are exact in fp16, so the products are mma.sync m16n8k16 fp16 tiles (16 keys x 8 heads)
//    with fp32 accumulators.  (Of fp8 operands mma.sync is far slower here, and tcgen05's least
//    tile is 64 or 128 rows where a kv head has at most 8.)  q, scaled by a power of two for its
//    largest value to be in [2^14, 2^15), is fp16 without loss down to 2^-28 of that value; the
//    weights, times the page's V scale over the largest so far, are fp16 with the largest between
//    2^10 and 2^15.  Scales of K apply to the scores.  (bf16 weights, without those two scalings,
//    want a second product for their low halves.)
//  * The fragments' element order along dims (K) and along keys (V) is free, as long as both
//    operands agree: a lane's 16 bytes of a K row are widened in registers, two bytes at a time; V
//    comes by transposing byte loads, its keys ordered to suit the widening.
//  * The batch's keys, in 128-key chunks, are one list (sequence, kv head, chunk), cut into shares
//    of even cost whatever lies at the cuts.  A chunk costs as much as the end of a (sequence, kv
//    head): by chunks alone, the shares of many short contexts were the last (256 contexts of 16 to
//    8192 tokens 51.0 against 40.3 us; 2 : 1 43.1, 2 : 3 41.2).  A (sequence, kv head) that several
//    shares cut is merged by the last of them to end, in the order of the keys whoever that is.
//  * One CTA per SM, of several groups: a producer and four consumer warps with a ring, and a
//    share, of their own.  As CTAs of their own, three to an SM, groups drew even parts of an SM's
//    rate only on average: of equal shares the last was done 60 us after the start where the mean
//    was 46 (256 contexts of 16 to 8192 tokens).
// What bounds it: int8, the consumers' issue slots (a code pair takes 1.5 instructions to widen); e4m3
// of 128, HBM; short batches, the start: 2.5 us until the first box is asked for and 2 for it to come.
// Measured (one GPU of 152 SMs; a plain copy runs at 6.8 TB/s): 64 contexts of 128 to 4096 keys, 8 kv
// heads of 128 e4m3 47.2 us, 6.0 TB/s; 256 of 16 to 8192, 4 of 64 int8 41.0 us, 4.7 TB/s; 4 of 32768, 8
// of 128 int8 46.5 us, 5.7 TB/s; 16 of 2048, 8 of 64 e4m3 13.4 us; one of 128, 8 of 64 4.9 us.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "decode_device.cuh"
#include "q8_device.cuh"

namespace pkv {
namespace {

constexpr int kQ8Keys = 128;           // keys of a stage: 32 for each consumer warp
constexpr int kChunkCost = 1, kEndCost = 1;  // of a chunk, and of a (sequence, kv head)'s end
// A share's cost at least (fewer shares otherwise).  As much as lies between two chunks' beginnings,
// so that no share is empty.
constexpr int kMinCost = 2;
static_assert(kMinCost >= kChunkCost + kEndCost, "no empty shares");
constexpr int kQ8MaxShares = 1024;
// Rows of a product's second operand.  A chunk of several queries a sequence takes two such tiles, so
// that codes are widened once for up to 16 rows.
constexpr int kRowTile = 8;
static_assert(kRowTile >= kMaxGroup, "a query's heads fit a tile");

// Groups of a CTA: with two tiles of rows two at most, for 168 registers a thread.
__host__ __device__ constexpr int q8_groups(int d, int nt) { return d == 64 && nt == 1 ? 3 : 2; }
constexpr int q8_stages(int d) { return d == 64 ? 4 : 3; }  // of a group's ring
__host__ __device__ constexpr int q8_threads(int d, int nt) { return q8_groups(d, nt) * (kConsumers + 32); }

struct alignas(16) Q8Desc {     // one stage's chunk
  int32_t nkeys;                // keys in range
  int32_t flags;                // kBegins, kEnds: of this share's part of the (sequence, kv head);
                                // kLastOne: of its chunks; above, its rows: (query, head of the group)
  int32_t row0;                 // its first row of q
  int32_t g;
  int32_t seen;                 // keys of the chunk that the first query sees; the i-th sees i more
  int32_t slot;                 // partial row the result goes to; -1: the whole context is here
  int32_t share0, parts;        // shares that cut it: share0 .. share0 + parts - 1
  __device__ int rows() const { return flags >> 8; }
};
static_assert(sizeof(Q8Desc) == 32, "stored and read 16 bytes at a time; the barriers lie behind");
constexpr int32_t kBegins = 1, kEnds = 2, kLastOne = 4;

template <int D, int NT>
struct Q8Smem {  // offsets from the 1024-byte aligned base
  static constexpr int kStages = q8_stages(D);
  static constexpr uint32_t kStage = 2 * kQ8Keys * D;
  static constexpr uint32_t kQ = NT * kRowTile * D * 2;
  // of each group, from group * kGroup
  static constexpr uint32_t q = kStages * kStage;
  static constexpr uint32_t scales = q + kStages * kQ;             // (K's, V's) of a stage's boxes
  static constexpr uint32_t desc = scales + kStages * 128;
  static constexpr uint32_t bars = desc + kStages * (uint32_t)sizeof(Q8Desc);  // full, empty
  static constexpr uint32_t misc = bars + kStages * 16;            // flag, last, issued
  static constexpr uint32_t kGroup = (misc + 16 + 1023) / 1024 * 1024;
  // of the CTA
  static constexpr uint32_t sums = q8_groups(D, NT) * kGroup;          // the prefix scan: per warp,
  static constexpr uint32_t incl = sums + q8_threads(D, NT) / 32 * 8;  // per thread within its warp
  static constexpr uint32_t total = incl + q8_threads(D, NT) * 8;
};
template <int D, int NT>
constexpr size_t q8_smem() { return 1024 + Q8Smem<D, NT>::total; }
static_assert(q8_smem<64, 2>() <= 227 * 1024 && q8_smem<128, 2>() <= 227 * 1024, "the groups fit an SM");
// A share's result in its last stage: per warp and head a row of D floats (4 apart, so that the
// lanes' stores lie in different banks), then the references and the sums.
__host__ __device__ constexpr int q8_row(int d) { return d + 4; }
static_assert(kConsumerWarps * kRowTile * (q8_row(128) + 2) * 4 <= (int)Q8Smem<128, 1>::kStage &&
                  kConsumerWarps * kRowTile * (q8_row(64) + 2) * 4 <= (int)Q8Smem<64, 1>::kStage,
              "the warps' results of a tile of rows fit a stage");

struct Q8Args {
  const uint16_t *q;            // [B][Hq][D]
  uint16_t *out;
  const int32_t *tables, *lens;
  // NULL: row b of q is sequence b's one query.  Else what is listed as sequence b: its sequence (-1:
  // none), its first row of q, its queries, the keys that the first of them sees; lens is the last's.
  const int4 *queries;
  const float *k_scale, *v_scale;
  float *o_part;                // [2 * shares][rows][D]: a share's first part, then its last's
  float *lse_part;              // [2 * shares][rows], base 2
  uint32_t *counters;           // [2][kQ8MaxShares] by the first that cuts: a context, a run of its
                                // shares; zero between calls
  int64_t num_blocks;
  int32_t max_blocks, max_len, num_seqs, num_q_heads, num_kv_heads, group;
  int32_t rows;                 // of a listed sequence and kv head, at most: group * its queries
  int32_t block_size, log2_bs, box_rows, log2_box;
  int32_t depth;                // 1: the first map leads to the other pool too
  int32_t v_first;              // V's rows lie first in a box
  float scale_log2;
  int32_t step;  // behind a step's write, which may still run: tables and lengths are read ahead of its end
};

// A stage is filled by 128-byte-swizzled boxes, one pool's rows of a box and then the other's: rows
// of 128 bytes hold one key (head_dim 128) or two (64).  Where the 16-byte chunk of dims 16 c ..
// 16 c + 15 of key `key` of the first (v = 0) or second (v = 1) lies.
template <int D>
__device__ __forceinline__ uint32_t chunk_off(int key, int c, int v, int log2_box) {
  const int in_box = key & ((1 << log2_box) - 1);
  const uint32_t row = (uint32_t)(((2 * (key >> log2_box) + v) << log2_box) + in_box) * D & ~127u;
  const uint32_t col = D == 128 ? (uint32_t)c : (uint32_t)(((key & 1) << 2) | c);
  return row + ((col ^ ((row >> 7) & 7)) << 4);
}
// Which key of 16 row r of the score product is.  (Row r + 8 is not key r + 8, so that the 8 rows
// that a transposing load reads together lie in 8 different bank groups.)
__device__ __forceinline__ int key_of(int r) { return r < 8 ? r : 8 | ((r & 7) ^ 4); }

__device__ __forceinline__ void lds(uint32_t (&w)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr));
}
// Two 16x16 byte matrices, transposed: matrix m's rows are the 16 bytes at lanes 16 m .. 16 m + 15's
// addresses; r[2m + i] holds bytes gid + 8 i of its rows 4 tig .. 4 tig + 3.
__device__ __forceinline__ void ldsm_b8_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// D(16x8, f32) += A(16x16, fp16, row) * B(16x8, fp16, col)
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// mbar_wait for waits that are mostly long: the thread may sleep up to 20 us at a time, so that
// waiting warps take no issue slots from the working ones.  The same 2 s limit.
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = dev::globaltimer_ns();
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    if (done) return true;
    if (dev::globaltimer_ns() - t0 > 2000000000ull) return false;
  }
}

// The largest of three (FMNMX3).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Weights are taken against a reference that moves only when a score is more than kSlack (in base
// 2) over it, to that score: fp16 weights of 2^kTop at the reference have room for 2^kSlack more.
// So most steps need no maximum over the warp.
constexpr float kTop = 10.f, kSlack = 5.f;

// V's codes as fp16 operands.  int8: behind 0x64 the byte c + 128 is the fp16 1024 + c + 128.
template <int KIND>
__device__ __forceinline__ void v_pairs(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if constexpr (KIND == PKV_Q8_INT8) {  // bytes 0, 2 and 1, 3
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"((w & 0x00ff00ffu) ^ 0x64806480u), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(((w >> 8) & 0x00ff00ffu) ^ 0x64806480u), "r"(0x64806480u));
  } else {
    lo = q8::pair<KIND, 0>(w);
    hi = q8::pair<KIND, 1>(w);
  }
}

// K's codes as fp16 operands.  int8: the byte c + 128 alone is the fp16 number (c + 128) 2^-24; the
// sum over dims of 128 q is taken off where the accumulator begins.  (So no subtraction for each
// pair.  The sums' rounding is that of products with |code| up to 255.)  V's codes come without a
// bias: theirs would grow with every key while the sum of v need not.
template <int KIND>
__device__ __forceinline__ void k_pairs(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if constexpr (KIND == PKV_Q8_INT8) {  // bytes 0, 2 and 1, 3
    lo = (w & 0x00ff00ffu) ^ 0x00800080u;
    hi = ((w >> 8) & 0x00ff00ffu) ^ 0x00800080u;
  } else {
    lo = q8::pair<KIND, 0>(w);
    hi = q8::pair<KIND, 1>(w);
  }
}

// A consumer warp's state for a tile of rows.  Lane (gid, tig): O^T fragments, rows gid and gid + 8 of
// m-tile mt being dims 16 mt + gid and + 8, for the tile's rows 2 tig and 2 tig + 1.
template <int D>
struct Q8Acc {
  float o[D / 16][4];
  float m0, m1, l0, l1;     // the rows' references; sums of weights, per lane
  uint32_t q[D / 16][2];    // fragments of q
  float f0, f1;             // scores' factors of the two rows, without K's scale (and the codes' unit)
  float b0, b1;             // what the two rows' raw scores begin with
  int i0, i1;               // the rows' queries
};
// What raw scores of the two rows under a scale of K are to be multiplied by.  int8's codes are in units of 2^-24,
// which comes last: with the rows' factor it would leave fp32 from q of 2^117 on, at a scale of 1.
template <int D, int KIND>
__device__ __forceinline__ void score_factors(const Q8Acc<D> &a, float k_scale, float &f0, float &f1) {
  uint64_t f = q8::mul2(q8::f32x2(a.f0, a.f1), q8::f32x2(k_scale, k_scale));
  if constexpr (KIND == PKV_Q8_INT8) f = q8::mul2(f, q8::f32x2(16777216.f, 16777216.f));
  f0 = q8::split(f).x;
  f1 = q8::split(f).y;
}
// For all tiles: the largest V scale so far, and 1 over it: o is in units of vref.
struct Q8Ref {
  float vref, vinv;
};

// A tile's query rows at qs ([rows][D] bf16, shared) as fragments: row gid, the dims that this lane's K
// bytes hold (D/4 tig ..).
template <int D, int KIND>
__device__ __forceinline__ void load_q(Q8Acc<D> &a, uint32_t qs, int rows, int lane, float scale_log2) {
  const int gid = lane >> 2, tig = lane & 3;
  uint32_t w[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) w[i] = 0u;
  if (gid < rows) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t v[4];
      lds(v, qs + (uint32_t)(gid * D + (D / 4) * tig + 8 * i) * 2u);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[4 * i + k] = v[k];
    }
  }
  uint32_t mb = 0;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) mb = __vmaxu2(mb, w[i] & 0x7fff7fffu);
  mb = max(mb & 0xffffu, mb >> 16);
  mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
  mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
  // 2^(14 - exponent of the largest), as far as that and its inverse are normal numbers
  const int e = min(max(14 - ((int)(mb >> 7) - 127), -126), 126);
  const float up = __uint_as_float((uint32_t)(e + 127) << 23);
  const float down = __uint_as_float((uint32_t)(127 - e) << 23) * scale_log2;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const float lo = dev::bf16lo_to_f32(w[i]) * up, hi = dev::bf16hi_to_f32(w[i]) * up;
    w[i] = q8::pack_f16x2(lo, hi);
    sum += lo + hi;
  }
  float begin = 0.f;
  if constexpr (KIND == PKV_Q8_INT8) {
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    begin = -128.f * 5.9604645e-8f * sum;
  }
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {  // dims 4 i .. 4 i + 3 in the order of k_pairs' bytes
    if constexpr (KIND == PKV_Q8_INT8) {
      a.q[i][0] = __byte_perm(w[2 * i], w[2 * i + 1], 0x5410);
      a.q[i][1] = __byte_perm(w[2 * i], w[2 * i + 1], 0x7632);
    } else {
      a.q[i][0] = w[2 * i];
      a.q[i][1] = w[2 * i + 1];
    }
  }
  a.f0 = __shfl_sync(0xffffffffu, down, 8 * tig);  // lanes of rows 2 tig and 2 tig + 1
  a.f1 = __shfl_sync(0xffffffffu, down, 8 * tig + 4);
  a.b0 = __shfl_sync(0xffffffffu, begin, 8 * tig);
  a.b1 = __shfl_sync(0xffffffffu, begin, 8 * tig + 4);
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) a.o[mt][0] = a.o[mt][1] = a.o[mt][2] = a.o[mt][3] = 0.f;
  a.m0 = a.m1 = -INFINITY;
  a.l0 = a.l1 = 0.f;
}

// Where a lane reads in a stage, of its warp's 32 keys.
struct Q8Lane {
  uint32_t k[2][2];  // K: its first chunk of rows gid and gid + 8 of each 16 keys
  uint32_t v;        // V: the first chunk of its row of the two transposed matrices
};
template <int D, int KIND>
__device__ __forceinline__ Q8Lane q8_lane(int warp, int lane, int log2_box, int v_first) {
  const int gid = lane >> 2, tig = lane & 3, r = lane & 15;
  Q8Lane x;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    x.k[t][0] = chunk_off<D>(32 * warp + 16 * t + gid, (D / 64) * tig, v_first, log2_box);
    x.k[t][1] = chunk_off<D>(32 * warp + 16 * t + key_of(gid + 8), (D / 64) * tig, v_first, log2_box);
  }
  // V's rows in the order of the weights' rows: 2 t, 2 t + 1, 2 t + 8, 2 t + 9 as the bytes of a word
  // that v_pairs takes together
  const int r1 = KIND == PKV_Q8_INT8 ? (r >> 1) & 1 : r & 1, r8 = KIND == PKV_Q8_INT8 ? r & 1 : (r >> 1) & 1;
  x.v = chunk_off<D>(32 * warp + 16 * (lane >> 4) + key_of(2 * (r >> 2) + r1 + 8 * r8), 0, v_first ^ 1, log2_box);
  return x;
}

// Raw scores of 16 keys, rows gid and gid + 8 (key_of(row)) x each tile's rows 2 tig, 2 tig + 1: the K
// chunks of these keys are at k0 and k1.
template <int D, int KIND, int NT>
__device__ __forceinline__ void q8_scores(const Q8Acc<D> (&a)[NT], float (&s)[NT][2][4], int t, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    s[n][t][0] = s[n][t][2] = a[n].b0;
    s[n][t][1] = s[n][t][3] = a[n].b1;
  }
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {  // (the next chunk is the other of a pair)
    uint32_t x[4], y[4];
    lds(x, k0 ^ (16u * i));
    lds(y, k1 ^ (16u * i));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t x0, x1, y0, y1;
      k_pairs<KIND>(x[k], x0, x1);
      k_pairs<KIND>(y[k], y0, y1);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(s[n][t], x0, y0, x1, y1, a[n].q[4 * i + k][0], a[n].q[4 * i + k][1]);
    }
  }
}

// Scores, softmax and weighted sum of the warp's 32 keys (the first nvalid of them in range; of these,
// with MASK, query i sees the first seen + i) of a stage at sb, the boxes' scales (K's, V's) at sc.  Two tiles
// take keys that are not all in range with MASK: their rows' factors come after the scores.
template <int D, int KIND, int NT, bool MASK>
__device__ __forceinline__ void q8_tiles(Q8Acc<D> (&a)[NT], Q8Ref &ref, uint32_t sb, const Q8Lane &at, const float2 *sc,
                                         int log2_box, int warp, int lane, int nvalid, int seen) {
  const int gid = lane >> 2, tig = lane & 3;
  float s[NT][2][4], vs[4], ks[4], f0[4], f1[4];
#pragma unroll
  for (int t = 0; t < 2; ++t) q8_scores<D, KIND, NT>(a, s, t, sb + at.k[t][0], sb + at.k[t][1]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 8 keys lie in one box; one box may hold more of these
    if (i == 0 || (i == 2 && log2_box < 5) || log2_box < 4) {
      const float2 f = sc[(32 * warp + 8 * i) >> log2_box];
      vs[i] = f.y;
      ks[i] = f.x;
      if (NT == 1) {
        score_factors<D, KIND>(a[0], f.x, f0[i], f1[i]);
      }
    } else {
      vs[i] = vs[i - 1];
      ks[i] = ks[i - 1];
      if (NT == 1) {
        f0[i] = f0[i - 1];
        f1[i] = f1[i - 1];
      }
    }
  }
  auto key = [&](int i) { return 16 * (i >> 1) + key_of(gid + 8 * (i & 1)); };  // of the lane, in each 8 keys
  if ((NT == 1 || MASK) && nvalid < 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (8 * i >= nvalid) vs[i] = 0.f;  // its box may not have been loaded
      // Scores of -inf, by a factor of their own: by 0, NaN or one below 0 they would be something else.
      if (!MASK && key(i) >= nvalid) {
        s[0][i >> 1][2 * (i & 1)] = s[0][i >> 1][2 * (i & 1) + 1] = -INFINITY;
        f0[i] = f1[i] = 1.f;
      }
    }
  }
  const float vmax = max3(max3(vs[0], vs[1], vs[2]), vs[3], vs[3]);
  const bool grows = vmax > ref.vref;
  float vscale = 1.f;  // what O is to be scaled by for a larger V scale
  auto grow = [&] {
    ref.vinv = 1.f / vmax;
    vscale = ref.vref * ref.vinv;
    ref.vref = vmax;
  };
  if (NT > 1 && grows) grow();
  uint32_t b[NT][2][2];  // the weights as B operands of the two tiles of keys
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    Q8Acc<D> &c = a[n];
    float sh0 = kTop - softmax_ref(c.m0), sh1 = kTop - softmax_ref(c.m1);
    float x[2][4];  // scores over the reference, plus kTop
    auto unseen = [&](int i, int query) { return key(i) >= min(nvalid, seen + query); };
    if (NT > 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) score_factors<D, KIND>(c, ks[i], f0[i], f1[i]);
    }
    auto shifted = [&] {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i >> 1][2 * (i & 1)] = fmaf(s[n][i >> 1][2 * (i & 1)], f0[i], sh0);
        x[i >> 1][2 * (i & 1) + 1] = fmaf(s[n][i >> 1][2 * (i & 1) + 1], f1[i], sh1);
      }
      if (MASK) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (unseen(i, c.i0)) x[i >> 1][2 * (i & 1)] = -INFINITY;
          if (unseen(i, c.i1)) x[i >> 1][2 * (i & 1) + 1] = -INFINITY;
        }
      }
    };
    shifted();
    float mx0 = max3(max3(x[0][0], x[0][2], x[1][0]), x[1][2], x[1][2]);
    float mx1 = max3(max3(x[0][1], x[0][3], x[1][1]), x[1][3], x[1][3]);
    // (A reference of -inf, no score over that so far, moves with the first one that is.)
    const bool over = mx0 > kTop + kSlack || mx1 > kTop + kSlack || (c.m0 == -INFINITY && mx0 > -INFINITY) ||
                      (c.m1 == -INFINITY && mx1 > -INFINITY);
    if (grows || __any_sync(0xffffffffu, over)) {
      if (NT == 1 && grows) grow();
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
      }
      const float mn0 = fmaxf(c.m0, mx0 - sh0), mn1 = fmaxf(c.m1, mx1 - sh1);
      float al0 = dev::ex2(c.m0 - softmax_ref(mn0)), al1 = dev::ex2(c.m1 - softmax_ref(mn1));
      c.m0 = mn0;
      c.m1 = mn1;
      c.l0 *= al0;
      c.l1 *= al1;
      al0 *= vscale;
      al1 *= vscale;
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        c.o[mt][0] *= al0;
        c.o[mt][1] *= al1;
        c.o[mt][2] *= al0;
        c.o[mt][3] *= al1;
      }
      sh0 = kTop - softmax_ref(mn0);
      sh1 = kTop - softmax_ref(mn1);
      shifted();
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float r0 = vs[2 * t] * ref.vinv, r1 = vs[2 * t + 1] * ref.vinv;
      const float p0 = dev::ex2(x[t][0]), p1 = dev::ex2(x[t][1]), p2 = dev::ex2(x[t][2]), p3 = dev::ex2(x[t][3]);
      c.l0 += p0 + p2;
      c.l1 += p1 + p3;
      float w0 = p0 * r0, w1 = p1 * r0, w2 = p2 * r1, w3 = p3 * r1;
      if (MASK) {  // (a V scale of NaN is for those who see it)
        if (unseen(2 * t, c.i0)) w0 = 0.f;
        if (unseen(2 * t, c.i1)) w1 = 0.f;
        if (unseen(2 * t + 1, c.i0)) w2 = 0.f;
        if (unseen(2 * t + 1, c.i1)) w3 = 0.f;
      }
      b[n][t][0] = dev::movmatrix_trans(q8::pack_f16x2(w0, w1));
      b[n][t][1] = dev::movmatrix_trans(q8::pack_f16x2(w2, w3));
    }
  }
  uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
  if (KIND == PKV_Q8_E4M3 && (NT == 1 || MASK) && nvalid < 32) {  // rows past the range may hold NaN codes
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      keep[t] = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (16 * t + key_of(2 * tig + (k & 1) + 8 * (k >> 1)) < nvalid) keep[t] |= 0xffu << (8 * k);
    }
  }
  if (KIND == PKV_Q8_E4M3 && MASK) {  // so may pages whose scale is NaN (the weights are NaN where they count)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (vs[2 * t] != vs[2 * t]) keep[t] &= 0xffff0000u;
      if (vs[2 * t + 1] != vs[2 * t + 1]) keep[t] &= 0x0000ffffu;
    }
  }
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt) {
    uint32_t v[4];
    ldsm_b8_trans(v, (sb + at.v) ^ (16u * mt));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (KIND == PKV_Q8_E4M3) {
        v[2 * t] &= keep[t];
        v[2 * t + 1] &= keep[t];
      }
      uint32_t y0, y1, z0, z1;
      v_pairs<KIND>(v[2 * t], y0, y1);
      v_pairs<KIND>(v[2 * t + 1], z0, z1);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(a[n].o[mt], y0, z0, y1, z1, b[n][t][0], b[n][t][1]);
    }
  }
}

// Reduces l over the warp and writes the warp's (m, l, O) of a tile's first n rows.  Where V is large, l and O
// are written 2^kDown times, the references kDown higher: of weights up to 2^(kTop + kSlack), sums of up to
// 2^(kDown - kTop - kSlack) keys are then no larger than V itself.  (Where it is small, O might become too small.)
constexpr float kDown = 40.f;
template <int D>
__device__ __forceinline__ void q8_stash(const Q8Acc<D> &a, float vref, const MergeArea &r, int n, int warp, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
  float l0 = a.l0, l1 = a.l1;
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, x);
    l1 += __shfl_xor_sync(0xffffffffu, l1, x);
  }
  const int h0 = 2 * tig, h1 = h0 + 1;
  const float higher = vref > 1.f ? kDown : 0.f, down = vref > 1.f ? dev::ex2(-kDown) : 1.f, unit = vref * down;
  if (gid == 0) {
    r.m[warp * kRowTile + h0] = a.m0 + higher;
    r.m[warp * kRowTile + h1] = a.m1 + higher;
    r.l[warp * kRowTile + h0] = l0 * down;
    r.l[warp * kRowTile + h1] = l1 * down;
  }
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int h = h0 + (k & 1);
      if (h < n) r.o[(warp * n + h) * q8_row(D) + 16 * mt + gid + 8 * (k >> 1)] = a.o[mt][k] * unit;
    }
}

// Four dims of one row from the four warps' results: the normalised output and the base-2
// log-sum (of weights 2^kTop at the reference, in every partial alike).
template <int D>
__device__ __forceinline__ float4 q8_joined(const MergeArea &r, int n, int h, int d, float *lse) {
  float m[kConsumerWarps], M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kConsumerWarps; ++w) M = fmaxf(M, m[w] = r.m[w * kRowTile + h]);
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
#pragma unroll
  for (int w = 0; w < kConsumerWarps; ++w) {
    const float wt = dev::ex2(m[w] - softmax_ref(M));
    const float4 o = *reinterpret_cast<const float4 *>(r.o + (w * n + h) * q8_row(D) + d);
    x.x += wt * o.x;
    x.y += wt * o.y;
    x.z += wt * o.z;
    x.w += wt * o.w;
    den += wt * r.l[w * kRowTile + h];
  }
  *lse = M + log2f(den);
  const float inv = den == 0.f ? 1.f : 1.f / den;
  return make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
}

__device__ __forceinline__ float4 times(const float4 &x, float f) { return make_float4(x.x * f, x.y * f, x.z * f, x.w * f); }
__device__ __forceinline__ void store4(uint16_t *dst, const float4 &x) {
  *reinterpret_cast<uint2 *>(dst) = make_uint2(dev::pack_bf16x2(x.x, x.y), dev::pack_bf16x2(x.z, x.w));
}

// The shares of a context cut into more than kOneJoin are joined kRunParts at a time, by the last of
// each such run, and then the runs, by the last of those: all at once, the last share of 128 (one context of 32768
// tokens, one kv head of 8 x 128) read 16 rows after one another for 26 us; 17 shares in two steps
// took 1.5 us more.
constexpr int kOneJoin = 32, kRunParts = 16;
// Shares' rows are kept this many times their values: of so many, each as large as bf16 goes, the sum stays one.
constexpr float kShareUnit = 1.f / kQ8MaxShares;

// Where part p of a context cut from share0 on has its row.
__device__ __forceinline__ int64_t q8_row_of(const Q8Args &a, int share0, int p, int h) {
  return (int64_t)(p == 0 ? 2 * share0 + 1 : 2 * (share0 + p)) * a.rows + h;
}

// Four dims of row h from the rows of parts p0, p0 + step, .. (n of them), in that order: those of
// `sub`, sub + every, ... are this lane's, the others its neighbours'.  The normalised result and its
// base-2 log-sum.
template <int D>
__device__ __forceinline__ float4 q8_merge(const Q8Args &a, int share0, int p0, int step, int n, int h, int d,
                                           int sub, int every, float *lse) {
  float M = -INFINITY, den = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = sub; k0 < n; k0 += 8 * every) {
    float lk[8];
    float4 o[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int k = k0 + u * every;
      lk[u] = -INFINITY;
      o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < n) {
        const int64_t row = q8_row_of(a, share0, p0 + k * step, h);
        lk[u] = __ldcg(a.lse_part + row);
        o[u] = __ldcg(reinterpret_cast<const float4 *>(a.o_part + row * D + d));
      }
    }
    float Mn = M;
#pragma unroll
    for (int u = 0; u < 8; ++u) Mn = fmaxf(Mn, lk[u]);
    const float ref = softmax_ref(Mn), sc = dev::ex2(M - ref);
    den *= sc;
    x.x *= sc;
    x.y *= sc;
    x.z *= sc;
    x.w *= sc;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float wt = dev::ex2(lk[u] - ref);
      den += wt;
      x.x += wt * o[u].x;
      x.y += wt * o[u].y;
      x.z += wt * o[u].z;
      x.w += wt * o[u].w;
    }
    M = Mn;
  }
  for (int e = 1; e < every; e <<= 1) {  // `every` neighbouring lanes (a power of two)
    const float M2 = __shfl_xor_sync(0xffffffffu, M, e), Mn = fmaxf(M, M2);
    const float s1 = dev::ex2(M - softmax_ref(Mn)), s2 = dev::ex2(M2 - softmax_ref(Mn));
    den = s1 * den + s2 * __shfl_xor_sync(0xffffffffu, den, e);
    x.x = s1 * x.x + s2 * __shfl_xor_sync(0xffffffffu, x.x, e);
    x.y = s1 * x.y + s2 * __shfl_xor_sync(0xffffffffu, x.y, e);
    x.z = s1 * x.z + s2 * __shfl_xor_sync(0xffffffffu, x.z, e);
    x.w = s1 * x.w + s2 * __shfl_xor_sync(0xffffffffu, x.w, e);
    M = Mn;
  }
  *lse = M + log2f(den);
  const float inv = den == 0.f ? 1.f : 1.f / den;
  return make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
}

// A barrier of one group's consumer warps.
__device__ __forceinline__ void group_bar(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kConsumers) : "memory");
}

// The end of a share's part of a context: the warps' results, a tile of rows after the other through
// the stage at `area`, into the output or a partial row (cf. finish_partition), and joins.
template <int D, int NT, bool LISTED>
__device__ __forceinline__ void q8_finish(const Q8Args &a, const Q8Acc<D> (&acc)[NT], float vref, float *area,
                                          const Q8Desc &d, int grp, int tid, volatile int *s_flag, volatile int *s_last) {
  constexpr int T = kConsumers;
  const int all = LISTED ? d.rows() : a.group, items = all * (D / 4);  // four dims of a row
  auto out_of = [&](int row) {
    const int i = LISTED ? row / a.group : 0;
    return a.out + ((int64_t)(d.row0 + i) * a.num_q_heads + d.g * a.group + (row - i * a.group)) * D;
  };
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int rows = NT > 1 ? min(all - n * kRowTile, kRowTile) : all;
    if (rows <= 0) break;
    group_bar(grp);  // every warp is done with the stage's keys, or with the last tile's results
    MergeArea r;
    r.o = area;
    r.m = r.o + kConsumerWarps * rows * q8_row(D);
    r.l = r.m + kConsumerWarps * kRowTile;
    q8_stash<D>(acc[n], vref, r, rows, tid >> 5, tid & 31);
    group_bar(grp);
    for (int i = tid; i < rows * (D / 4); i += T) {
      const int h = i / (D / 4), c = 4 * (i - h * (D / 4)), at = n * kRowTile + h;
      float lse;
      const float4 x = q8_joined<D>(r, rows, h, c, &lse);
      if (d.slot < 0) {
        store4(out_of(at) + c, x);
      } else {
        const int64_t row = (int64_t)d.slot * a.rows + at;
        *reinterpret_cast<float4 *>(a.o_part + row * D + c) = times(x, kShareUnit);
        if (c == 0) a.lse_part[row] = lse;
      }
    }
  }
  if (d.slot < 0) return;
  // Whether this is the last of n ends that count on `counter` (then it is 0 again).
  auto last_of = [&](uint32_t *counter, int n) {
    group_bar(grp);
    if (tid == 0) {
      int last = 0;
      if (!*s_flag) last = dev::atomic_add_acq_rel(counter, 1u) + 1 == (unsigned)n;
      if (last) *counter = 0u;
      *s_last = last;
    }
    group_bar(grp);
    return *s_last != 0;  // (written again behind the next end's barriers)
  };
  // Joins the rows of parts p0, p0 + step, ..; into the output, or into the first one's place.
  auto join = [&](int p0, int step, int n, bool out) {
    int every = 1;  // lanes per item
    while (every < 32 && 2 * every * items <= T && 8 * every < n) every <<= 1;
    for (int i0 = 0; i0 < items; i0 += T / every) {  // uniform over the warp: q8_merge shuffles
      const int i = min(i0 + tid / every, items - 1);  // (the last item may be joined twice, alike)
      const int h = i / (D / 4), c = 4 * (i - h * (D / 4)), sub = tid & (every - 1);
      float lse;
      const float4 x = q8_merge<D>(a, d.share0, p0, step, n, h, c, sub, every, &lse);
      if (out) {
        if (sub == 0) store4(out_of(h) + c, times(x, 1.f / kShareUnit));
      } else {  // every other row of the run has been read when the barrier lets this one be
        group_bar(grp);
        const int64_t row = q8_row_of(a, d.share0, p0, h);
        if (sub == 0 && i0 + tid / every < items) {
          *reinterpret_cast<float4 *>(a.o_part + row * D + c) = x;
          if (c == 0) a.lse_part[row] = lse;
        }
        group_bar(grp);
      }
    }
  };
  if (d.parts > kOneJoin) {
    const int runs = (d.parts + kRunParts - 1) / kRunParts;
    const int p0 = ((d.slot >> 1) - d.share0) / kRunParts * kRunParts, n = min(kRunParts, d.parts - p0);
    if (n > 1) {  // (a run of one share has no counter: the next context's first run may have that one)
      if (!last_of(a.counters + kQ8MaxShares + d.share0 + p0, n)) return;
      join(p0, 1, n, false);
    }
    if (last_of(a.counters + d.share0, runs)) join(0, kRunParts, runs, true);
  } else if (last_of(a.counters + d.share0, d.parts)) {
    join(0, 1, d.parts, true);
  }
}

// The two pools' boxes at row y, by one copy: the map's third dimension leads from one pool to the other.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int32_t y, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(0), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const float *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival on `bar` when this thread's cp.asyncs so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// NT: tiles of rows.  LISTED: a.queries says whose the rows are, else row b of q is sequence b's one query.
template <int D, int KIND, int NT, bool LISTED>
__global__ void __launch_bounds__(q8_threads(D, NT), 1)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
                     const __grid_constant__ Q8Args a) {
  using SL = Q8Smem<D, NT>;
  constexpr int STAGES = SL::kStages, GROUPS = q8_groups(D, NT), WARPS = q8_threads(D, NT) / 32;
  constexpr int kFirstProducer = GROUPS * kConsumerWarps;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = dev::smem_addr(smem_raw);
  const uint32_t cta_base = (raw + 1023u) & ~1023u;
  uint8_t *const cta_ptr = smem_raw + (cta_base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool producer = warp >= kFirstProducer;
  const int grp = producer ? warp - kFirstProducer : warp / kConsumerWarps;
  const uint32_t base = cta_base + grp * SL::kGroup;
  uint8_t *const base_ptr = cta_ptr + grp * SL::kGroup;
  const uint32_t bar_full = base + SL::bars, bar_empty = bar_full + STAGES * 8;
  volatile int *const s_flag = reinterpret_cast<volatile int *>(base_ptr + SL::misc);
  volatile int *const s_last = s_flag + 1;
  volatile int *const s_issued = s_flag + 2;
  Q8Desc *const s_desc = reinterpret_cast<Q8Desc *>(base_ptr + SL::desc);
  int64_t *const s_sums = reinterpret_cast<int64_t *>(cta_ptr + SL::sums);
  int64_t *const s_incl = reinterpret_cast<int64_t *>(cta_ptr + SL::incl);

  if (!a.step) q8::await_stream();
  const int Hkv = a.num_kv_heads;
  const int cap = (int)min((int64_t)a.max_blocks * a.block_size, (int64_t)a.max_len);
  auto length = [&](int b) { return min(max(q8::ld(a.lens + b), 0), cap); };
  auto chunks_of = [](int L) { return (int)(((int64_t)L + kQ8Keys - 1) / kQ8Keys); };
  auto cost_of = [&](int L) { return L > 0 ? kChunkCost * (int64_t)chunks_of(L) + kEndCost : 0; };  // of a kv head
  auto shares_of = [&](int64_t w) { return min((int64_t)gridDim.x * GROUPS, max((int64_t)1, q8::quotient(w, kMinCost))); };
  // Shares 0 .. gridDim.x - 1 are the CTAs' first groups', so that a few lie on SMs of their own.
  const int share = grp * (int)gridDim.x + (int)blockIdx.x;
  // Entries of the block table, one a lane.
  auto entries = [&](int b, int at) {
    if (b >= a.num_seqs) return 0;
    const int seq = LISTED ? max(q8::ld(&a.queries[b].x), 0) : b;
    return at + lane < a.max_blocks ? q8::ld(a.tables + (int64_t)seq * a.max_blocks + at + lane) : 0;
  };

  // The table window of where this share would begin if all contexts had max_len keys: for equal
  // lengths its load is under way before the lengths are known.
  int guess_b = -1, guess_win = 0, guess_tb = 0;
  if (producer) {
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm0)) : "memory");
      if (!a.depth) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm1)) : "memory");
    }
    const int64_t n = cost_of(cap), all = n * Hkv * a.num_seqs, shares = shares_of(all);
    if (share < shares && all > 0) {
      const int64_t at = q8::quotient(all * share, shares), unit = q8::quotient(at, n);
      guess_b = (int)q8::quotient(unit, Hkv);
      guess_win = (int)((at - unit * n + kChunkCost - 1) / kChunkCost) * kQ8Keys >> a.log2_bs;
      guess_tb = entries(guess_b, guess_win);
    }
  }

  // ---- the list: the prefix of the sequences' chunks, a run of sequences per thread
  const int run = (a.num_seqs + WARPS * 32 - 1) / (WARPS * 32);
  const int b_lo = min((int)threadIdx.x * run, a.num_seqs), b_hi = min(b_lo + run, a.num_seqs);
  int64_t incl = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const int L0 = q8::ld(a.lens + b), L = min(max(L0, 0), cap);
    if (L != L0 && blockIdx.x == 0) raise_error(PKV_DEVERR_CONTEXT_LEN);
    incl += cost_of(L);
    if (L == 0 && b % (int)gridDim.x == (int)blockIdx.x) {  // empty: zeros
      int4 l = make_int4(b, b, 1, 0);
      if (LISTED) l = q8::ld(a.queries + b);
      uint2 *o = reinterpret_cast<uint2 *>(a.out + (int64_t)l.y * a.num_q_heads * D);
      for (int i = 0; i < l.z * a.num_q_heads * D / 4; ++i) o[i] = make_uint2(0u, 0u);
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_sums[warp] = incl;
  s_incl[threadIdx.x] = incl;
  if (producer && lane == 0) {
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      dev::mbar_init(bar_full + 8 * s, 33);  // lane 0's bytes, and every producer lane's scales
      dev::mbar_init(bar_empty + 8 * s, kConsumerWarps);
    }
    *s_flag = 0;
    *s_issued = 0;
    dev::fence_mbar_init();
  }
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) total += s_sums[w];
  const int64_t W = total * Hkv, N = shares_of(W);
  if (W == 0 || share >= N) {  // (no barrier of the whole CTA follows)
    if (a.step) q8::await_stream();  // the grid's end is the write's end, whoever has work
    return;
  }
  const int64_t lo = q8::quotient(W * share, N), hi = q8::quotient(W * (share + 1), N);
  auto timeout = [&] {
    if (lane == 0) {
      raise_error(PKV_DEVERR_TIMEOUT);
      *s_flag = 1;
    }
  };

  if (producer) {
    const uint64_t policy = dev::policy_evict_first();
    const int rb = a.box_rows;
    const uint32_t box_bytes = (uint32_t)(rb * D);
    const uint32_t q_bytes = (uint32_t)a.group * D * 2u;  // of a query
    // ---- the first chunk at or behind place lo: the thread whose run of sequences holds the place,
    // then the sequence, the kv head and the chunk
    int b, at_lane;
    int64_t at = 0, n;  // cost before; of the lane's sequence
    {
      int w = 0;
      while (w + 1 < WARPS && (at + s_sums[w]) * Hkv <= lo) at += s_sums[w++];
      const unsigned past = __ballot_sync(0xffffffffu, (at + s_incl[32 * w + lane]) * Hkv > lo);
      const int r = past ? __ffs(past) - 1 : 31;
      if (r > 0) at += s_incl[32 * w + r - 1];
      for (b = (32 * w + r) * run;; b += 32) {
        n = b + lane < a.num_seqs ? cost_of(length(b + lane)) : 0;
        int64_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, (at + inc) * Hkv > lo);
        if (hit || b + 32 >= a.num_seqs) {
          at_lane = hit ? __ffs(hit) - 1 : 0;
          at += __shfl_sync(0xffffffffu, inc - n, at_lane);
          break;
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
      }
      b += at_lane;
    }
    int64_t cost = max(__shfl_sync(0xffffffffu, n, at_lane), (int64_t)1);  // of a kv head of sequence b
    int nch = (int)max((cost - kEndCost) / kChunkCost, (int64_t)1), L = length(b);
    int g = (int)q8::quotient(lo - at * Hkv, cost);
    int64_t u0 = at * Hkv + g * cost;  // where the kv head begins in the list
    int c = (int)((lo - u0 + kChunkCost - 1) / kChunkCost);
    // Table entries are loaded ahead of their use: the current window of 32, the one after it, the
    // sequence's first, and the next sequence's length and first window.
    int win = (c * kQ8Keys) >> a.log2_bs;
    int tb = b == guess_b && win == guess_win ? guess_tb : entries(b, win);
    int tb_next = entries(b, win + 32), tb_first = win == 0 ? tb : entries(b, 0);
    int len_seq = b + 1 < a.num_seqs ? length(b + 1) : 0, tb_seq = entries(b + 1, 0);
    // The next kv head, or the next sequence that has keys (there is one: its place is below hi).
    auto next_head = [&] {
      c = 0;
      u0 += cost;
      if (++g == Hkv) {
        g = 0;
        do {
          ++b;
          L = len_seq;
          tb_first = tb_seq;
          len_seq = b + 1 < a.num_seqs ? length(b + 1) : 0;
          tb_seq = entries(b + 1, 0);
        } while (L == 0 && b + 1 < a.num_seqs);
        nch = chunks_of(L);
        cost = cost_of(L);
      }
      win = 0;
      tb = tb_first;
      tb_next = entries(b, 32);
    };
    if (c >= nch) next_head();  // lo lies at a kv head's end
    Q8Desc dsc = {};
    int4 listed = make_int4(0, 0, 1, 0);  // what sequence b is
    bool first = true, last = false;
    q8::await_stream();  // the step's write is done
    int i = 0;
    for (; !last; ++i) {
      const int s = i % STAGES;
      if (first) {
        const int64_t end = u0 + kChunkCost * (int64_t)(nch - 1);  // its last chunk's place
        if (LISTED)
          listed = q8::ld(a.queries + b);
        else
          listed.y = b;
        dsc.row0 = listed.y;
        dsc.g = g;
        dsc.slot = -1;
        dsc.share0 = share;
        dsc.parts = 1;
        if (u0 < lo || end >= hi) {  // cut: place x is in share floor(((x + 1) N - 1) / W)
          dsc.share0 = (int)q8::quotient((u0 + 1) * N - 1, W);
          dsc.parts = (int)q8::quotient((end + 1) * N - 1, W) - dsc.share0 + 1;
          dsc.slot = 2 * share + (dsc.share0 == share ? 1 : 0);
        }
      }
      if (i >= STAGES &&
          !__all_sync(0xffffffffu, wait_long(bar_empty + 8 * s, ((i / STAGES) - 1) & 1))) {
        timeout();
        break;
      }
      last = (c + 1 < nch ? u0 + kChunkCost * (int64_t)(c + 1) : u0 + cost) >= hi;
      const int k0 = c * kQ8Keys;
      const int nk = min(kQ8Keys, L - k0);
      const int nbox = (nk + rb - 1) >> a.log2_box;
      if ((k0 >> a.log2_bs) >= win + 32) {  // (a chunk's pages lie in one window)
        win += 32;
        tb = tb_next;
        tb_next = entries(b, win + 32);
      }
      const int key = k0 + lane * rb;
      int64_t phys = __shfl_sync(0xffffffffu, tb, min((key >> a.log2_bs) - win, 31));
      if (phys < 0 || phys >= a.num_blocks) {
        if (lane < nbox) raise_error(PKV_DEVERR_BLOCK_ID);
        phys = 0;
      }
      const int64_t unit = phys * Hkv + g;
      const int32_t row = (int32_t)((unit * a.block_size + (key & (a.block_size - 1))) * D / 128);
      if (lane == 0) {
        dsc.nkeys = nk;
        if (LISTED) dsc.seen = listed.w - k0;
        dsc.flags = (first ? kBegins : 0) | (c + 1 == nch || last ? kEnds : 0) | (last ? kLastOne : 0);
        if (LISTED) dsc.flags |= a.group * listed.z << 8;
        s_desc[s] = dsc;
        dev::mbar_arrive_expect_tx(bar_full + 8 * s, 2u * nbox * box_bytes + (first ? (LISTED ? listed.z : 1) * q_bytes : 0u));
        if (first)
          for (int i = 0; i < (LISTED ? listed.z : 1); ++i)
            dev::bulk_load(base + SL::q + s * SL::kQ + i * q_bytes,
                           a.q + ((int64_t)(listed.y + i) * a.num_q_heads + g * a.group) * D, q_bytes, bar_full + 8 * s);
      }
      __syncwarp();
      if (lane < nbox) {
        const uint32_t dst = base + s * SL::kStage + lane * 2 * box_bytes;
        if (a.depth) {
          tma_load_3d(dst, &tm0, row, bar_full + 8 * s, policy);
        } else {
          dev::tma_load_2d(dst, &tm0, 0, row, bar_full + 8 * s, policy);
          dev::tma_load_2d(dst + box_bytes, &tm1, 0, row, bar_full + 8 * s, policy);
        }
        const uint32_t ds = base + SL::scales + s * 128 + lane * 8;
        cp_async4(ds, a.k_scale + unit);
        cp_async4(ds + 4, a.v_scale + unit);
      }
      cp_async_arrive(bar_full + 8 * s);
      __syncwarp();
      first = false;
      if (++c == nch && !last) {
        first = true;
        next_head();
      }
    }
    if (lane == 0) *s_issued = i;
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ----------------------------------------------------------- consumer warps
    const int wg = warp - grp * kConsumerWarps, tid = (int)threadIdx.x - grp * kConsumers;
    const Q8Lane at = q8_lane<D, KIND>(wg, lane, a.log2_box, a.v_first);
    Q8Acc<D> acc[NT];
    Q8Ref ref = {};
    for (int i = 0;; ++i) {
      const int s = i % STAGES;
      if (!__all_sync(0xffffffffu, wait_long(bar_full + 8 * s, (i / STAGES) & 1))) {
        timeout();
        break;
      }
      const int2 info = *reinterpret_cast<const int2 *>(s_desc + s);  // keys, flags
      if (info.y & kBegins) {
        ref.vref = ref.vinv = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int row = n * kRowTile;
          load_q<D, KIND>(acc[n], base + SL::q + s * SL::kQ + row * D * 2, (LISTED ? info.y >> 8 : a.group) - row, lane,
                          a.scale_log2);
          if (LISTED) {
            acc[n].i0 = (row + 2 * (lane & 3)) / a.group;
            acc[n].i1 = (row + 2 * (lane & 3) + 1) / a.group;
          }
        }
      }
      const int nvalid = min(32, info.x - 32 * wg), seen = LISTED ? s_desc[s].seen - 32 * wg : nvalid;
      const float2 *const sc = reinterpret_cast<const float2 *>(base_ptr + SL::scales + s * 128);
      if (nvalid > 0) {
        if (!LISTED || (seen >= nvalid && (NT == 1 || nvalid == 32)))
          q8_tiles<D, KIND, NT, false>(acc, ref, base + s * SL::kStage, at, sc, a.log2_box, wg, lane, nvalid, seen);
        else
          q8_tiles<D, KIND, NT, LISTED>(acc, ref, base + s * SL::kStage, at, sc, a.log2_box, wg, lane, nvalid, seen);
      }
      if (info.y & kEnds) {
        const Q8Desc d = s_desc[s];
        q8_finish<D, NT, LISTED>(a, acc, ref.vref, reinterpret_cast<float *>(base_ptr + s * SL::kStage), d, grp, tid, s_flag,
                         s_last);
        dev::fence_proxy_async_smem();  // the results, ahead of the boxes that follow them
      }
      if (info.y & kLastOne) break;
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(bar_empty + 8 * s);
    }
    // ---- a timed-out wait leaves copies possibly in flight: wait for them (bounded), with what
    // the producer had issued when the flag was seen
    group_bar(grp);
    if (tid == 0 && *s_flag) {
      const uint64_t t0 = dev::globaltimer_ns();
      while (*s_issued == 0 && dev::globaltimer_ns() - t0 < 4000000000ull) {
      }
      const int issued = *s_issued;
      for (int s = 0; s < STAGES; ++s) {
        const int last = s + ((issued - 1 - s) / STAGES) * STAGES;  // last chunk on stage s
        if (last >= 0 && last < issued) (void)dev::mbar_wait(bar_full + 8 * s, (last / STAGES) & 1);
      }
    }
  }
}

bool g_q8_attr[kMaxDevices][2][2][3];  // kernel attributes set [head_dim][kind][NT - 1 + listed]

struct Q8Layout {
  size_t o_part, lse_part, total;
};

// The words that are zero between calls first, at the same place for every call; then the partial
// rows of as many shares as the GPU holds groups.
Q8Layout q8_layout(int part_rows, int d, int sms) {
  const size_t rows = (size_t)2 * std::min(sms * q8_groups(d, 1), kQ8MaxShares) * part_rows;
  Q8Layout l;
  l.o_part = 2 * kQ8MaxShares * sizeof(uint32_t);
  l.lse_part = l.o_part + rows * d * sizeof(float);
  l.total = (l.lse_part + rows * sizeof(float) + 255) & ~size_t(255);
  return l;
}

struct DecodeQ8 {
  const int4 *queries;
  int32_t most_queries;  // of a listed sequence
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

template <int D, int KIND, int NT, bool LISTED>
int launch_decode_q8(const DecodeQ8 &x, cudaStream_t stream, bool step) {
  const pkv_cache_desc &c = *x.desc;
  CUtensorMap tm0, tm1 = {};
  int sms = 0;
  auto *const kern = decode_q8_kernel<D, KIND, NT, LISTED>;
  const int box = std::min(c.block_size, kQ8Keys);
  // One map for both pools where they are whole rows apart (half the copies: 16 keys of head_dim 64
  // took the producer longer to issue than HBM to bring).
  const void *first = x.cache->k_cache, *second = x.cache->v_cache;
  const bool v_first = reinterpret_cast<uintptr_t>(second) < reinterpret_cast<uintptr_t>(first);
  if (v_first) std::swap(first, second);
  const size_t apart = reinterpret_cast<uintptr_t>(second) - reinterpret_cast<uintptr_t>(first);
  const bool depth = apart > 0 && apart % 128 == 0 && apart < (size_t(1) << 40);
  {
    std::lock_guard<std::mutex> lk(attn_mutex());
    int dev = 0, rc;
    if ((rc = current_device(&dev)) || (rc = device_sms(&sms)) ||
        (rc = codes_map(first, depth ? apart : 0, c, box, &tm0)) ||
        (!depth && (rc = codes_map(second, 0, c, box, &tm1))))
      return rc;
    bool *const attr = &g_q8_attr[dev][D == 64 ? 0 : 1][KIND][NT - 1 + LISTED];
    if (!*attr) {
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)q8_smem<D, NT>());
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
      if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute");
      *attr = true;
    }
  }
  const int part_rows = x.hq / c.num_kv_heads * (LISTED ? x.most_queries : 1);
  const Q8Layout l = q8_layout(part_rows, D, sms);
  char *const ws = static_cast<char *>(x.workspace);
  Q8Args a;
  a.q = x.q;
  a.out = x.out;
  a.tables = x.tables;
  a.lens = x.lens;
  a.queries = x.queries;
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
  a.rows = part_rows;
  a.block_size = c.block_size;
  a.log2_bs = ilog2(c.block_size);
  a.box_rows = box;
  a.log2_box = ilog2(box);
  a.depth = depth ? 1 : 0;
  a.v_first = v_first ? 1 : 0;
  a.step = step ? 1 : 0;
  a.scale_log2 = x.scale * kLog2e;
  // one CTA per SM; fewer where the batch cannot have that many shares
  const int64_t most =
      (((int64_t)x.max_len + kQ8Keys - 1) / kQ8Keys * kChunkCost + kEndCost) * x.num_seqs * c.num_kv_heads;
  const int64_t ctas = std::min(sms, kQ8MaxShares / q8_groups(D, NT));
  const int64_t grid = std::max<int64_t>(1, std::min(ctas, most / kMinCost));
  const cudaError_t e =
      q8::launch_early(kern, dim3((unsigned)grid), q8_threads(D, NT), q8_smem<D, NT>(), stream, tm0, tm1, a);
  if (e != cudaSuccess) return cuda_error(e, "decode_q8_kernel launch");
  return PKV_OK;
}

template <int NT, bool LISTED>
int launch_kinds_q8(const DecodeQ8 &x, cudaStream_t s, bool step) {
  const bool i8 = x.cache->kind == PKV_Q8_INT8;
  if (x.desc->head_dim == 64)
    return i8 ? launch_decode_q8<64, PKV_Q8_INT8, NT, LISTED>(x, s, step)
              : launch_decode_q8<64, PKV_Q8_E4M3, NT, LISTED>(x, s, step);
  return i8 ? launch_decode_q8<128, PKV_Q8_INT8, NT, LISTED>(x, s, step)
            : launch_decode_q8<128, PKV_Q8_E4M3, NT, LISTED>(x, s, step);
}

int launch_decode_q8(const DecodeQ8 &x, cudaStream_t s, bool step) {
  return x.num_seqs == 0 ? PKV_OK : launch_kinds_q8<1, false>(x, s, step);
}

// A few queries per sequence as a list for decode_q8_kernel, `each` queries to an entry, `per` entries to a
// sequence: query i of n sees the context's first L - n + i + 1 keys.  Also zeroes the decode's
// counters (this workspace keeps none).
struct ListArgs {
  const int32_t *start, *lens;
  int4 *queries;
  int32_t *seen;  // keys that an entry's last query sees
  uint32_t *counters;
  int32_t num_seqs, num_queries, max_new, cap, each, per;
};
__global__ void __launch_bounds__(256) list_queries_kernel(const ListArgs a) {
  q8::await_stream();
  q8::let_next_begin();
  const int i = blockIdx.x * 256 + threadIdx.x, b = i / a.per, first = (i - b * a.per) * a.each;
  if (i < 2 * kQ8MaxShares) a.counters[i] = 0u;
  if (b >= a.num_seqs) return;
  const int L = q8::ld(a.lens + b), s0 = q8::ld(a.start + b), e0 = q8::ld(a.start + b + 1);
  const int len = min(max(L, 0), a.cap), s = min(max(s0, 0), a.num_queries);
  const int n = min(max(min(e0, a.num_queries) - s, 0), a.max_new);
  if (first == 0 && (len != L || s != s0 || s + n != e0 || n > len)) raise_error(PKV_DEVERR_CONTEXT_LEN);
  const int count = min(n - first, a.each), sees = len - n + first + 1;
  a.queries[i] = count > 0 ? make_int4(b, s + first, count, sees) : make_int4(-1, 0, 0, 0);
  a.seen[i] = count > 0 ? max(sees + count - 1, 0) : 0;
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

// One tile of rows or two, whichever is less in all.  Times of a chunk as measured: 1.15 us of three groups' and
// 1.4 of two at head_dim 64 and 128 with one tile; with two 1.13 of two groups' and 2.8.
ListPlan list_plan(int32_t group, int32_t head_dim, int32_t max_query_len) {
  ListPlan best = {};
  for (int32_t tiles = 1; tiles <= 2; ++tiles) {
    const int32_t most = tiles * kRowTile / group, per = (max_query_len + most - 1) / most;
    const double chunk = head_dim == 64 ? (tiles == 1 ? 1.15 : 1.13) : tiles == 1 ? 1.4 : 2.8;
    const double block = chunk / q8_groups(head_dim, tiles);
    if (best.per == 0 || best.per > kMaxListPer || per * block <= best.per * best.block)
      best = {(max_query_len + per - 1) / per, per, tiles, block};
  }
  best.per = (max_query_len + best.each - 1) / best.each;  // (none of no queries)
  return best;
}

size_t list_q8_workspace(int64_t entries, int32_t d, int sms) {
  return q8_layout(2 * kRowTile, d, sms).total + (size_t)entries * (sizeof(int4) + sizeof(int32_t));
}

int launch_list_q8(const ChunkLaunch &l, const pkv_q8_cache &cache, const pkv_cache_desc &c,
                   const int32_t *block_tables, int32_t max_blocks, void *workspace, int sms, cudaStream_t stream) {
  const size_t decode = q8_layout(2 * kRowTile, c.head_dim, sms).total;
  ListArgs r;
  r.start = l.query_start;
  r.lens = l.context_lens;
  const ListPlan plan = list_plan(l.num_q_heads / l.num_kv_heads, l.head_dim, l.max_query_len);
  r.each = plan.each;
  r.per = plan.per;
  const int32_t entries = l.num_seqs * r.per;
  r.queries = reinterpret_cast<int4 *>(static_cast<char *>(workspace) + decode);
  r.seen = reinterpret_cast<int32_t *>(r.queries + entries);
  r.counters = static_cast<uint32_t *>(workspace);
  r.num_seqs = l.num_seqs;
  r.num_queries = (int32_t)l.num_queries;
  r.max_new = l.max_query_len;
  r.cap = l.max_context;
  const int threads = std::max(2 * kQ8MaxShares, (int)entries);
  const cudaError_t e =
      q8::launch_early(list_queries_kernel, dim3((unsigned)((threads + 255) / 256)), 256, 0, stream, r);
  if (e != cudaSuccess) return cuda_error(e, "list_queries_kernel launch");
  const DecodeQ8 x = {r.queries, r.each, l.out, l.q, &cache, block_tables, max_blocks, r.seen, l.max_context,
                      entries, l.num_q_heads, &c, l.scale, workspace, decode};
  return plan.tiles == 2 ? launch_kinds_q8<2, true>(x, stream, false) : launch_kinds_q8<1, true>(x, stream, false);
}

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
  const DecodeQ8 x = {nullptr, 1, out, q, cache, block_tables, max_blocks_per_seq, context_lens, max_context_len,
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
  const DecodeQ8 x = {nullptr, 1, out, q, cache, block_tables, max_blocks_per_seq, context_lens, max_context_len,
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
  const DecodeQ8 x = {nullptr, 1, out, q_out, cache, block_tables, max_blocks_per_seq, context_lens, max_context_len,
                      num_seqs, num_q_heads, desc, scale, workspace, workspace_bytes};
  return step_q8(w, x, static_cast<cudaStream_t>(stream), fn);
}
