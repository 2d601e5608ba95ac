// pkv_tiles.cu -- attention of many query rows that share keys, on the 5th-generation
// tensor cores: packed causal prompts (prompt_attention) and the shared prefixes of decode
// batches (the first half of paged_decode_shared_prefix_attention).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "attn_tc.cuh"
#include "q8_device.cuh"
#include "shared_device.cuh"

namespace pkv {

// ===========================================================================
// tile_kernel: a CTA works on one kv head's query rows -- (query token, head of the group)
// pairs -- as two tiles of up to 128 rows in ping-pong: while four softmax warps work on one
// tile's scores (one thread per row), the tensor core works on the other tile.
//   S_t = Q_t . K_j^T   tcgen05.mma M=128 N=128 K=D, both K-major in shared memory, S_t in TMEM
//   P_t = exp2(S_t * scale - m)  fp32, rounded to bf16 into TMEM over columns of S_t already read
//   O_t += P_t . V_j    P_t from TMEM, V_j MN-major in shared memory, O_t in TMEM
// The row's reference max m moves only when a block raises it by more than kTcRescale;
// then O_t and the row sum are rescaled.
// K and V stream through separate rings, each with its producer warp (the K producer loads the
// queries too); each tile's MMAs are issued by a thread of their own.
//
// Two ways of pairing:
//  * kPrompt: the tiles are consecutive query rows of one packed sequence and share every
//    K/V block (up to 256 rows per block staged).  Causal: a row of query i sees keys 0 .. i.
//    K and V rows come straight from the packed projections: one TMA box per block.
//    A CTA goes on to other work items, those of CTAs that have not started yet (cluster
//    launch control): its rings, queries and scores of the next item fill while the rows of
//    the last one are written, so that an item costs no launch, set-up and first-copy latency
//    of its own (about 9 us, the time of six key blocks).
//    Measured: 8192 tokens of 24 / 8 heads of 128 at 1565 TFLOP/s, the tensor pipe 67% busy
//    (a block pair takes 3080 cycles, 2080 of them MMAs; the exponentials and their rounding
//    are the rest); 8192 of 32 / 8 heads of 64 at 905, the tensor pipe 42% busy: half the MMAs
//    for the same softmax.  Short prompts end in what an item costs beside its blocks (an
//    epilogue of 2000 cycles, the last P.V, the first S: about 2.6 us).
//  * kPrefix: both tiles hold the same rows (queries of a group of sequences) and take
//    alternate key blocks, so that a few rows over a long prefix still overlap softmax and
//    tensor core.  The keys come from the pages of the group's first sequence; the CTA
//    covers one split of them, joins its tiles' results through shared memory and writes one
//    softmax-normalised fp32 row and log-sum-exp per query row.  (A cluster's splits joined
//    through distributed shared memory wrote a quarter of the rows, but took 3.5 us to read
//    them against 1 us to write them all.)  Bound by the copies: a box of 16 rows and 64 dims
//    takes the TMA unit 63 cycles and its bytes, 1.57 us per block of 128 keys at block_size
//    16 and head_dim 128, at which 152 CTAs draw 6.3 TB/s (16 sequences over 65536 tokens).
//  * kNewest: kPrompt for the newest tokens of sequences whose keys lie in packed rows of their own,
//    kv_rows to a sequence, in fp16 (the rows that an 8-bit cache is read back to): a query sees
//    `past` more keys than its place.  All operands are fp16: the queries are widened where their
//    tile was loaded, each row times a power of two; K's and V's rows are in units of a factor of
//    their (sequence, kv head); weights are taken with 2^7 at the reference.
enum { kPrompt = 0, kPrefix = 1, kNewest = 2 };
constexpr float kNewestTop = 7.f;  // weights reach 2^(kNewestTop + kTcRescale): fp16 ends at 65504

struct TileArgs {
  uint16_t *out;            // prompt
  int64_t out_stride;       // elements from one query token to the next
  const int32_t *start;     // [num + 1] first query row of each sequence / group
  int32_t num, total, max_len;   // sequences or groups, query tokens, longest sequence
  int32_t num_q_heads, num_kv_heads, group;
  int32_t tile_tokens;      // query tokens of a tile: 128 / group
  float scale_log2;
  const uint16_t *q, *k, *v;  // for the rows that are computed once more (row_by_keys)
  // prefix
  const int32_t *block_tables, *context_lens, *prefix_lens;
  int64_t num_blocks;
  int32_t box_rows;
  int32_t split_keys;       // keys per split (a multiple of kTcKeys)
  float *o_part, *lse_part; // [B][Hq][n_rows][D], [B][Hq][n_rows]; row s: the s-th split
  SharedCut cut;
  // newest tokens (and context_lens)
  int32_t kv_rows, max_context;    // packed rows of a sequence; the longest context
  const float *k_unit, *v_unit;    // [num][num_kv_heads]
  const int32_t *nan_from;         // [num][num_kv_heads] rows that see this key are NaN
  const int4 *order;               // [num] longest context first: a sequence, its first query row, its rows
};

// 8 softmax warps, the K and the V producer (two warps a ring measured neutral), an MMA warp per
// tile.  (Four more warps that write the output while the softmax warps go on to the next item:
// two documents of 7000 and 8192 tokens 1% faster, prompts of 336 tokens 6% slower, and 8% at
// head_dim 64: O_t has no second buffer in TMEM, so the next item's P.V waits all the same.)
constexpr int kTileThreads = 32 * 12;
constexpr int kItemReaders = 11;  // kPrompt's warps that read an item: all but the K producer

// One piece of work, handed from the K producer to the other warps.
struct TileItem {
  int32_t live;             // 0: no more items
  int32_t g, first;         // kv head, the sequence's (group's) first query token
  int32_t tok0, n;          // the tiles' first token and the token count, within the sequence
  int32_t key0, t_end;      // keys [key0, t_end) are staged, in blocks of kTcKeys
  int32_t nb0, nb1;         // blocks of each tile
  int32_t prefix;           // kPrefix: the whole pages of the group's prefix
  int32_t past, seq;        // kNewest: keys before the sequence's first query; its number
};

template <int D, int MODE>
struct TileSmem {
  // K and V ring stages.  kPrefix: even, so that a stage serves one tile alone (block j is
  // tile j & 1's): a waiter may trust a barrier's parity only if it saw the phase before,
  // and a tile's MMA thread sees the phases of its own blocks.
  static constexpr int KSK = D == 64 ? 4 : 2;
  static constexpr int KSV = D == 64 ? 4 : (MODE != kPrefix ? 2 : 4);
  static_assert(MODE != kPrefix || (KSK % 2 == 0 && KSV % 2 == 0), "one tile per stage");
  static constexpr uint32_t kSub = kTcKeys * 128;     // 128 rows x 128 B (64 dims)
  static constexpr uint32_t kTile = kSub * (D / 64);
  static constexpr int kQ = MODE != kPrefix ? 2 : 1;  // Q tiles
  static constexpr uint32_t k = 0;
  static constexpr uint32_t v = k + KSK * kTile;
  static constexpr uint32_t q = v + KSV * kTile;
  // head_dim 64: a [128 keys][64] tile of ones, read by P.V as 16 more columns of V, so that
  // the tensor core forms the row sums (O's columns are free in TMEM at 64, not at 128)
  static constexpr bool kOnes = D == 64;
  static constexpr uint32_t ones = q + kQ * kTile;
  // kPrompt: 32 dims of each softmax warp's 32 output rows, row r's 16-byte chunk c at
  // c ^ (r / 2 & 3)
  static constexpr uint32_t stage = ones + (kOnes ? kSub : 0);
  static constexpr uint32_t item = stage + (MODE != kPrefix ? 2 * kTcRows * 64 : 0);  // two items
  static constexpr uint32_t clc = item + 2 * sizeof(TileItem); // a launch-control answer, 16 B
  // kPrefix, once the rings are done with: the tiles' rows [2][128][D] fp32, row r's 16-byte
  // chunk c at c ^ (r & 7), where the rings begin; (max in base 2, sum) per row at their end
  static constexpr uint32_t rows = 0;
  static constexpr uint32_t ml = q - 2 * kTcRows * 8;
  static constexpr uint32_t bars = clc + 16;
  static_assert(MODE != kPrefix || rows + 2u * kTcRows * D * 4 <= ml, "the rows fit the rings");
  // the rings, then s_full, pv_done per tile, p_half per tile and half, q_full, q_free, o_free
  // per tile, item_full, item_empty per slot, clc_full, mma_done, tiles_done; kNewest: q_wide per tile
  static constexpr int kRings = 2 * KSK + 2 * KSV;
  static constexpr int kBars = kRings + (MODE == kNewest ? 23 : 21);
  static constexpr uint32_t tslot = bars + kBars * 8;
  static constexpr uint32_t flag = tslot + 8;
  static constexpr uint32_t turns = flag + 8;  // P.V batches issued, per tile
  static constexpr uint32_t total = turns + 8;
};
template <int D, int MODE>
constexpr size_t tile_smem() { return 1024 + TileSmem<D, MODE>::total; }
static_assert(tile_smem<64, kPrompt>() <= 227 * 1024 && tile_smem<128, kPrompt>() <= 227 * 1024 &&
                  tile_smem<64, kPrefix>() <= 227 * 1024 && tile_smem<128, kPrefix>() <= 227 * 1024,
              "the tiles fit a CTA");
static_assert(sizeof(TileItem) == 48, "items keep the answer 16-byte aligned");

// Cluster launch control: asks for a CTA of this grid that has not started; the answer (16
// bytes) completes on `bar`.  Then: whether there was one, and its blockIdx.x.
__device__ __forceinline__ void clc_try_cancel(uint32_t dst, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
      "r"(bar)
      : "memory");
}
__device__ __forceinline__ bool clc_answer(uint32_t src, uint32_t &ctaid) {
  uint32_t got;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(got), "=r"(ctaid)
      : "r"(src)
      : "memory");
  return got != 0;
}

// Where a search through the sequences stands: 32 of them from number `c`, one per lane, and
// what lies before them.
struct TileCursor {
  int c = -32, carry = 0, next_carry = 0;  // the furthest end before these, and with them
  int64_t before = 0;                      // pieces before these
  int s = 0, len = 0, mine = 0, upto = 0, prefix = 0;
  int seq = 0;                             // kNewest
};

// The sequence (or group) whose pieces of `tokens` query tokens hold piece number idx, its
// first query token, its length, the piece's place in it, its pieces and its prefix.  Whole
// warps; misplaced and over-long sequences are moved, cut and flagged.  The search goes on from
// where the last one ended (from the beginning, 512 sequences of 84 tokens took 15 us an item).
template <int MODE>
__device__ __forceinline__ bool locate_tile(const TileArgs &a, TileCursor &at, int64_t idx, int tokens,
                                            int lane, int &first, int &n, int &tile, int &ntiles,
                                            int &prefix, int &seq) {
  if (idx < at.before) at = TileCursor();
  while (true) {
    const int64_t total = at.before + __shfl_sync(0xffffffffu, at.upto, 31);
    if (idx < total) break;
    if (at.c + 32 >= a.num) return false;
    at.c += 32;
    at.before = total;
    at.carry = at.next_carry;
    at.prefix = a.prefix_lens && at.c + lane < a.num ? __ldg(a.prefix_lens + at.c + lane) : 0;
    if constexpr (MODE == kNewest) {
      const int4 o = at.c + lane < a.num ? q8::ld(a.order + at.c + lane) : make_int4(0, 0, 0, 0);
      at.seq = o.x;
      at.s = o.y;
      at.len = o.z;
    } else {
      disjoint_group(a.start, a.num, a.total, a.max_len, at.c, lane, at.next_carry, at.s, at.len);
    }
    at.mine = at.upto = (at.len + tokens - 1) / tokens;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at.upto, x);
      if (lane >= x) at.upto += y;
    }
  }
  const int l = __ffs(__ballot_sync(0xffffffffu, at.before + at.upto > idx)) - 1;
  prefix = __shfl_sync(0xffffffffu, at.prefix, l);
  seq = MODE == kNewest ? __shfl_sync(0xffffffffu, at.seq, l) : at.c + l;
  first = __shfl_sync(0xffffffffu, at.s, l);
  n = __shfl_sync(0xffffffffu, at.len, l);
  ntiles = __shfl_sync(0xffffffffu, at.mine, l);
  tile = (int)(idx - at.before - __shfl_sync(0xffffffffu, at.upto - at.mine, l));
  return true;
}

// The work of CTA (cta_x, cta_y), the same on every lane of the warp; false if it has none.
template <int MODE>
__device__ __forceinline__ bool make_item(const TileArgs &a, TileCursor &at, unsigned cta_x, unsigned cta_y,
                                          int lane, TileItem &it) {
  it.live = 1;
  it.g = (int)(cta_x % (unsigned)a.num_kv_heads);
  const int tokens = a.tile_tokens * (MODE != kPrefix ? 2 : 1);
  int tile, ntiles, prefix;
  if (!locate_tile<MODE>(a, at, cta_x / (unsigned)a.num_kv_heads, tokens, lane, it.first, it.n, tile, ntiles, prefix,
                   it.seq))
    return false;
  if constexpr (MODE == kNewest) {
    const int L = q8::ld(a.context_lens + it.seq), len = min(max(L, 0), a.max_context);
    if ((len != L || len < it.n) && lane == 0) raise_error(PKV_DEVERR_CONTEXT_LEN);
    it.past = len - it.n;  // (below 0: the first queries see no key, and give zeros)
    it.tok0 = (ntiles - 1 - tile) * tokens;
    const int e0 = min(it.tok0 + a.tile_tokens, it.n), e1 = min(it.tok0 + tokens, it.n);
    it.key0 = 0;
    it.t_end = max(it.past + e1, 1);
    it.nb0 = (max(it.past + e0, 1) + kTcKeys - 1) / kTcKeys;
    it.nb1 = e1 > e0 ? (it.t_end + kTcKeys - 1) / kTcKeys : 0;
  } else if constexpr (MODE == kPrompt) {
    it.tok0 = (ntiles - 1 - tile) * tokens;  // a sequence's last tiles see the most keys: first
    const int e0 = min(it.tok0 + a.tile_tokens, it.n), e1 = min(it.tok0 + tokens, it.n);
    it.key0 = 0;
    it.t_end = e1;
    it.nb0 = (e0 + kTcKeys - 1) / kTcKeys;
    it.nb1 = e1 > e0 ? (e1 + kTcKeys - 1) / kTcKeys : 0;
  } else {
    it.tok0 = tile * tokens;
    const int pages = shared_pages(a.cut, prefix);
    if ((prefix < 0 || prefix > min((int64_t)a.cut.max_blocks * a.cut.block_size, (int64_t)a.cut.max_prefix)) &&
        lane == 0)
      raise_error(PKV_DEVERR_CONTEXT_LEN);
    prefix = pages;
    it.prefix = prefix;
    it.key0 = (int)cta_y * a.split_keys;
    if (it.key0 >= prefix) return false;
    it.t_end = min(it.key0 + a.split_keys, prefix);
    const int nblk = (it.t_end - it.key0 + kTcKeys - 1) / kTcKeys;
    it.nb0 = (nblk + 1) / 2;
    it.nb1 = nblk / 2;
  }
  return true;
}

// Loads keys [k0, k0 + nk) of kv head g from the group's pages into a block tile
// [D/64][128][128 B], one TMA box of min(block_size, 64) rows and 64 dims per lane, completing
// on `bar`.
template <int D, uint32_t SUB>
__device__ __forceinline__ void load_paged_block(const CUtensorMap *tm, uint32_t dst, uint32_t bar,
                                                 int k0, int nk, int &win, int &tb,
                                                 const int32_t *trow, int lb_last,
                                                 const TileArgs &a, int g, int lane,
                                                 uint64_t policy) {
  constexpr int kH = D / 64;
  const int rb = a.box_rows;
  const int nbox = (nk + rb - 1) / rb;
  const int lb_hi = (k0 + (nbox - 1) * rb) >> a.cut.log2_bs;
  if (lb_hi >= win + 32 || (k0 >> a.cut.log2_bs) < win) {
    win = k0 >> a.cut.log2_bs;
    tb = (win + lane <= lb_last) ? __ldg(trow + win + lane) : 0;
  }
  const int bi = lane / kH, hh = lane % kH;
  const int key = k0 + bi * rb;
  const int src = min(max((key >> a.cut.log2_bs) - win, 0), 31);
  const int64_t phys_raw = __shfl_sync(0xffffffffu, tb, src);
  if (lane == 0) dev::mbar_arrive_expect_tx(bar, (uint32_t)nbox * rb * 128u * kH);
  __syncwarp();
  if (bi < nbox) {
    int64_t phys = phys_raw;
    if (phys < 0 || phys >= a.num_blocks) {
      raise_error(PKV_DEVERR_BLOCK_ID);
      phys = 0;
    }
    const int off = key & (a.cut.block_size - 1);
    const int32_t row = (int32_t)((phys * a.num_kv_heads + g) * a.cut.block_size + off);
    const uint32_t d = dst + (uint32_t)(bi * rb) * 128u;
    if constexpr (D == 64) {
      dev::tma_load_2d(d, tm, 0, row, bar, policy);
    } else {
      asm volatile(
          "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
          ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(d + hh * SUB),
          "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(hh), "r"(row), "r"(bar), "l"(policy)
          : "memory");
    }
  }
  __syncwarp();
}

// One whole block tile of packed rows [row, row + 128) of kv head g (rows past the tensor
// read as zeros): a single box {64 dims, 128 rows, D/64 halves, 1 head}.
__device__ __forceinline__ void load_packed_block(const CUtensorMap *tm, uint32_t dst, uint32_t bar,
                                                  uint32_t bytes, int row, int g, uint64_t policy) {
  dev::mbar_arrive_expect_tx(bar, bytes);
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(row), "r"(0), "r"(g), "r"(bar), "l"(policy)
      : "memory");
}

// dev::mbar_wait in as few instructions as it takes: the kernel waits in forty places, and
// with 90 KB of code its warps spent a quarter of their time waiting for instructions
// (128 prompts of 336 tokens, 217 us; with 57 KB 157 us).
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity) {
  uint64_t since = 0;
#pragma unroll 1
  while (!dev::mbar_try_wait(bar, parity)) {
    const uint64_t now = dev::globaltimer_ns();
    if (since == 0) since = now;
    if (now - since > 2000000000ull) return false;
  }
  return true;
}
// __syncthreads from more than one place of the code.
__device__ __forceinline__ void cta_sync() { asm volatile("bar.sync 0;" ::: "memory"); }
// The whole warp's: true on every lane, or on none.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, tile_wait(bar, parity));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// ---------------------------------------------------------------------------
// The softmax threads' work on one block, in two passes over the row's 128 columns of S_t,
// 32 at a time out of TMEM.  The second pass is a loop over the two 64-column halves (its
// straight-line form stalled on instruction fetches), and each half of P is published as
// soon as it is stored, so that its P.V runs under the other half's exponentials.

// A masked block's row sees the columns c <= lim; lo and hi are the least and the largest lim
// of the warp, so that 32 columns that all its rows see, or none, cost no compares, the
// latter no exponentials either (compares throughout: 512 prompts of 84
// tokens 124 against 119 us).
struct Limits {
  int lim, lo, hi;
};

// The largest of the row's columns (with kMask: of those it sees), unscaled; -inf if there is
// none.  Leaves columns 0 .. 31 in x0.
template <bool kMask>
__device__ __forceinline__ float row_max(uint32_t sb, const Limits &l, uint32_t (&x0)[32]) {
  float mx[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) mx[u] = -INFINITY;
  if constexpr (kMask) {
#pragma unroll 1
    for (int c0 = max(min(l.hi, kTcKeys - 1), 0) & ~31; c0 >= 0; c0 -= 32) {
      dev::tmem_ld32(sb + c0, x0);
      tmem_wait_ld_regs(x0);
      const int lim = l.lo >= c0 + 31 ? 31 : l.lim - c0;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        mx[e & 7] = fmax3(mx[e & 7], 2 * e <= lim ? __uint_as_float(x0[2 * e]) : -INFINITY,
                          2 * e + 1 <= lim ? __uint_as_float(x0[2 * e + 1]) : -INFINITY);
    }
    return fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(fmax3(mx[3], mx[4], mx[5]), mx[6], mx[7]));
  }
  uint32_t xb[32];
  dev::tmem_ld32(sb + 96, xb);
  tmem_wait_ld_regs(xb);
#pragma unroll
  for (int ch = 3; ch >= 0; --ch) {  // the buffers alternate; chunk 0 ends in x0
    uint32_t(&cur)[32] = (ch & 1) ? xb : x0;
    uint32_t(&nxt)[32] = (ch & 1) ? x0 : xb;
    if (ch > 0) dev::tmem_ld32(sb + (ch - 1) * 32, nxt);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      mx[e & 7] = fmax3(mx[e & 7], __uint_as_float(cur[2 * e]), __uint_as_float(cur[2 * e + 1]));
    }
    if (ch > 0) tmem_wait_ld_regs(nxt);
  }
  return fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(fmax3(mx[3], mx[4], mx[5]), mx[6], mx[7]));
}

__device__ __forceinline__ void add_f32x2(float &a0, float &a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

// P = exp2(S * scale - m) of the 32 columns x (columns c0 .. of the row) as bf16 (fp16) pairs, and
// their sum added to ls: of the weights as they are before the rounding, two to an add (the
// rounded ones, one to an add, measured 6% slower).  Rounding moves a weight by at most 2^-8
// of itself, and so the output by at most 2^-8 of sum p |v|.
template <bool kMask, bool kSum, bool kHalf>
__device__ __forceinline__ void chunk_exp(const uint32_t (&x)[32], int c0, int lim, float scale_log2,
                                          float m, uint32_t *pk, float (&ls)[4]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float a0, a1;
    fma_f32x2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]), scale_log2, -m, a0, a1);
    if constexpr (kMask) {
      a0 = c0 + 2 * e <= lim ? a0 : -INFINITY;
      a1 = c0 + 2 * e + 1 <= lim ? a1 : -INFINITY;
    }
    const float p0 = dev::ex2(a0), p1 = dev::ex2(a1);
    if constexpr (kHalf)
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk[e]) : "f"(p1), "f"(p0));
    else
      pk[e] = dev::pack_bf16x2(p0, p1);
    if constexpr (kSum) add_f32x2(ls[2 * (e & 1)], ls[2 * (e & 1) + 1], p0, p1);
  }
}

// ---------------------------------------------------------------------------
// A row that must not see a key gives it the weight 0, and in the product with V a NaN or an
// infinity of that key's v comes through all the same (0 * inf).  A masked row whose result is
// not finite is therefore computed once more, from its own keys alone, on the CUDA cores: by one
// warp, 32 keys at a time, a key's score per lane, D / 32 dims of the result per lane.  (Looking
// for such rows costs a call behind shared pages 0.1 to 0.3 us, 0.5 to 1%.)

template <int D>
struct RowSum {
  float m = -INFINITY, l = 0.f, acc[D / 32] = {};  // max (base 2), sum, unnormalised result
};

// The lane's dims of a row of bf16 values.
template <int D>
__device__ __forceinline__ void lane_dims(const uint16_t *row, int lane, float (&x)[D / 32]) {
  const uint32_t *const p = reinterpret_cast<const uint32_t *>(row) + lane * (D / 64);
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const uint32_t w = __ldg(p + i);
    x[2 * i] = dev::bf16lo_to_f32(w);
    x[2 * i + 1] = dev::bf16hi_to_f32(w);
  }
}

// Query row q over keys [n0, n1), key t's k and v at k_at(t) and v_at(t); stop(sum): no need to
// go on.  Whole warps.
template <int D, typename KAt, typename VAt, typename Stop>
__device__ __forceinline__ RowSum<D> row_by_keys(const uint16_t *q, int n0, int n1, float scale_log2, int lane,
                                                 KAt k_at, VAt v_at, Stop stop) {
  RowSum<D> r;
#pragma unroll 1
  for (int t0 = n0; t0 < n1; t0 += 32) {
    float x = -INFINITY;
    if (t0 + lane < n1) {
      const uint4 *const kr = reinterpret_cast<const uint4 *>(k_at(t0 + lane)), *const qr = reinterpret_cast<const uint4 *>(q);
      x = 0.f;
#pragma unroll 2
      for (int i = 0; i < D / 8; ++i) {
        const uint4 kk = __ldg(kr + i), qq = __ldg(qr + i);
        const uint32_t kw[4] = {kk.x, kk.y, kk.z, kk.w}, qw[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x = fmaf(dev::bf16lo_to_f32(qw[e]), dev::bf16lo_to_f32(kw[e]), x);
          x = fmaf(dev::bf16hi_to_f32(qw[e]), dev::bf16hi_to_f32(kw[e]), x);
        }
      }
      x *= scale_log2;
    }
    float m = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = fmaxf(m, r.m);
    const float ref = m == -INFINITY ? 0.f : m;  // no weight yet: all are 0
    const float f = dev::ex2(r.m - ref), p = dev::ex2(x - ref);
    float sum = p;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    r.m = m;
    r.l = r.l * f + sum;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) r.acc[d] *= f;
    const int nk = min(32, n1 - t0);
#pragma unroll 4
    for (int u = 0; u < nk; ++u) {
      const float w = __shfl_sync(0xffffffffu, p, u);
      float v[D / 32];
      lane_dims<D>(v_at(t0 + u), lane, v);
#pragma unroll
      for (int d = 0; d < D / 32; ++d) r.acc[d] = fmaf(w, v[d], r.acc[d]);
    }
    if (stop(r)) break;
  }
  return r;
}

// kPrefix: partial row `split` of query row `row` (b * Hq + h) once more, if it is not finite, from
// keys [key0, see) of the pages of sequence `first`.  Whole warps.
template <int D>
__device__ __noinline__ void prefix_row(const TileArgs &a, int row, int split, int first, int g, int key0,
                                        int see, int lane) {
  constexpr int VPL = D / 32;
  float *const dst = a.o_part + ((int64_t)row * a.cut.n_rows + split) * D + lane * VPL;
  bool bad = false;
#pragma unroll
  for (int d = 0; d < VPL; ++d) bad |= !isfinite(dst[d]);
  if (!__any_sync(0xffffffffu, bad)) return;
  const int32_t *const table = a.block_tables + (int64_t)first * a.cut.max_blocks;
  auto at = [&](int t) {
    int64_t phys = __ldg(table + (t >> a.cut.log2_bs));
    if (phys < 0 || phys >= a.num_blocks) phys = 0;  // (flagged where it was copied)
    return ((phys * a.num_kv_heads + g) * a.cut.block_size + (t & (a.cut.block_size - 1))) * D;
  };
  const RowSum<D> r = row_by_keys<D>(
      a.q + (int64_t)row * D, key0, see, a.scale_log2, lane, [&](int t) { return a.k + at(t); },
      [&](int t) { return a.v + at(t); }, [](const RowSum<D> &) { return false; });
#pragma unroll
  for (int d = 0; d < VPL; ++d) dst[d] = r.l == 0.f ? 0.f : r.acc[d] / r.l;
  if (lane == 0)
    a.lse_part[(int64_t)row * a.cut.n_rows + split] = r.l == 0.f ? -INFINITY : (r.m + log2f(r.l)) * kLn2;
}

// Row r of a query tile [D/64][128][128 B] from bf16 to fp16 in place, times 2^e (returned): for
// its largest value to be in [2^14, 2^15), as far as 2^e and its inverse are normal numbers.
template <int D, uint32_t SUB>
__device__ __forceinline__ int widen_row(uint8_t *tile, int r) {
  uint32_t m = 0;
#pragma unroll 1
  for (int c = 0; c < D / 8; ++c) {
    const uint4 x = *reinterpret_cast<const uint4 *>(tile + (c >> 3) * SUB + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x.x));
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x.y));
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x.z));
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x.w));
  }
  m &= 0x7fff7fffu;
  m = max(m & 0xffffu, m >> 16);
  const int e = min(max(14 - ((int)(m >> 7) - 127), -126), 126);
  const float up = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll 1
  for (int c = 0; c < D / 8; ++c) {
    uint4 *const p = reinterpret_cast<uint4 *>(tile + (c >> 3) * SUB + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    const uint4 x = *p;
    auto half2 = [&](uint32_t w) {
      uint32_t h;
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(dev::bf16hi_to_f32(w) * up), "f"(dev::bf16lo_to_f32(w) * up));
      return h;
    };
    *p = make_uint4(half2(x.x), half2(x.y), half2(x.z), half2(x.w));
  }
  return e;
}

template <int D, int MODE>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv, const __grid_constant__ TileArgs a) {
  using SL = TileSmem<D, MODE>;
  constexpr int KSK = SL::KSK, KSV = SL::KSV, kRings = SL::kRings;
  constexpr bool kPaged = MODE == kPrefix;     // keys from pages; partial outputs; one item
  constexpr bool kShareKeys = MODE != kPrefix; // both tiles take every block
  constexpr bool kHalf = MODE == kNewest;       // fp16 operands, scaled (else bf16)
  constexpr bool kOnes = SL::kOnes;
  constexpr int kON = D + (kOnes ? 16 : 0);    // O columns per tile (then the row sums)
  constexpr int kProducer = 8, kProducerV = 9, kMma = 10;  // kMma + t: tile t's MMA warp
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = dev::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *const bp = smem_raw + (base - raw);
  const uint32_t bars = base + SL::bars;
  auto k_full = [&](int s) { return bars + 8u * s; };
  auto k_empty = [&](int s) { return bars + 8u * (KSK + s); };
  auto v_full = [&](int s) { return bars + 8u * (2 * KSK + s); };
  auto v_empty = [&](int s) { return bars + 8u * (2 * KSK + KSV + s); };
  auto s_full = [&](int t) { return bars + 8u * (kRings + t); };
  auto pv_done = [&](int t) { return bars + 8u * (kRings + 2 + t); };
  auto p_half = [&](int t, int hf) { return bars + 8u * (kRings + 4 + 2 * t + hf); };
  auto q_full = [&](int t) { return bars + 8u * (kRings + 8 + t); };
  auto q_free = [&](int t) { return bars + 8u * (kRings + 10 + t); };
  auto o_free = [&](int t) { return bars + 8u * (kRings + 12 + t); };
  auto item_full = [&](int s) { return bars + 8u * (kRings + 14 + s); };
  auto item_empty = [&](int s) { return bars + 8u * (kRings + 16 + s); };
  const uint32_t clc_full = bars + 8u * (kRings + 18);
  const uint32_t mma_done = bars + 8u * (kRings + 19);
  const uint32_t tiles_done = bars + 8u * (kRings + 20);
  [[maybe_unused]] auto q_wide = [&](int t) { return bars + 8u * (kRings + 21 + t); };
  volatile int *const s_turn = reinterpret_cast<volatile int *>(bp + SL::turns);
  volatile uint32_t *const s_tmem = reinterpret_cast<volatile uint32_t *>(bp + SL::tslot);
  volatile int *const s_flag = reinterpret_cast<volatile int *>(bp + SL::flag);
  TileItem *const s_item = reinterpret_cast<TileItem *>(bp + SL::item);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.group, tile_rows = a.tile_tokens * G;
  // the decode kernel that merges may start its own part while this one runs
  if constexpr (kPaged) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (MODE == kNewest) q8::await_stream();
  auto blk = [&](int t, int i) { return kShareKeys ? i : 2 * i + t; };

  // kPrompt: the K producer looks for the first item while the others set up.
  TileItem it = {};
  TileCursor at;
  bool have = false;
  if (kPaged) {
    have = make_item<MODE>(a, at, blockIdx.x, blockIdx.y, lane, it);
    if (!have) return;
  }
  const TileItem first = it;  // kPrefix: the CTA's only one
  if (kPaged || warp != kProducer) {
    if (tid < SL::kBars) {
      const int i = tid, r = i - kRings;
      const uint32_t count = (i >= KSK && i < 2 * KSK) || (i >= 2 * KSK + KSV && i < kRings)
                                 ? (kShareKeys ? 2u : 1u)     // empty: both MMA threads, or one
                             : r >= 4 && r < 8 ? 4u           // p_half: one per softmax warp
                             : r == 12 || r == 13 ? 4u        // o_free: alike
                             : r == 16 || r == 17 ? (uint32_t)kItemReaders
                             : r == 19 ? 2u                   // mma_done: both MMA threads
                             : r == 20 ? 8u                   // tiles_done: every softmax warp
                             : r == 21 || r == 22 ? 4u        // q_wide: one per softmax warp
                                       : 1u;
      dev::mbar_init(bars + 8u * i, count);
      dev::fence_mbar_init();
    }
    if (tid == 0) {
      *s_flag = 0;
      s_turn[0] = s_turn[1] = 0;
    }
    if (kOnes && tid < 256) {  // 1.0 everywhere; read by the tensor core (async proxy)
      constexpr uint32_t kOne = kHalf ? 0x3C003C00u : 0x3F803F80u;
#pragma unroll 1
      for (int i = tid; i < (int)(SL::kSub / 16); i += 256)
        *reinterpret_cast<uint4 *>(bp + SL::ones + i * 16) =
            make_uint4(kOne, kOne, kOne, kOne);
    }
    // rows of the Q tiles past the last whole token are never loaded: zeros
    if (tid < 256) {
      const int pad = (kTcRows - tile_rows) * 8;  // 16-byte pieces
#pragma unroll 1
      for (int sub = 0; sub < SL::kQ * (D / 64); ++sub)
#pragma unroll 1
        for (int i = tid; i < pad; i += 256)
          *reinterpret_cast<uint4 *>(bp + SL::q + sub * SL::kSub + tile_rows * 128 + i * 16) =
              make_uint4(0u, 0u, 0u, 0u);
    }
    dev::fence_proxy_async_smem();
    if (warp == 0) dev::tmem_alloc(base + SL::tslot, 512);
    dev::tc_fence_before();
    cta_sync();
    dev::tc_fence_after();
  }
  const uint32_t tmem = *s_tmem;  // S_t at column 128 t, O_t at 256 + kON t

  auto fail = [&](bool ok) {
    if (!ok) {
      raise_error(PKV_DEVERR_TIMEOUT);
      *s_flag = 1;
    }
    return ok;
  };
  // Copies `it` number `items` (of the reading warp's count) out of its slot.
  auto next_item = [&](int items, TileItem &x) {
    if constexpr (kPaged) return items == 0 && have;  // every warp found its CTA's one item
    const int s = items & 1;
    if (!warp_wait(item_full(s), (items >> 1) & 1)) {
      if (lane == 0) fail(false);
      return false;
    }
    x = s_item[s];
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(item_empty(s));
    return x.live != 0;
  };
  int issued = 0, qn0 = 0, qn1 = 0;  // producers: blocks loaded, Q tiles of either tile
  [[maybe_unused]] int ends = 0;     // kPrefix's softmax warps: whether the row's context ends among the keys

  // Loads blocks [from, to) of the item's K or V into this warp's ring, each after
  // before(block); `issued` runs on.
  auto load_ring = [&](bool is_k, const TileItem &x, int from, int to, auto before) {
    const CUtensorMap *const tm = is_k ? &tmk : &tmv;
    const int ks = is_k ? KSK : KSV;
    // other CTAs read the same keys (kPrefix: only where the group has more than one tile of rows)
    const uint64_t policy = dev::policy_evict_last();
    const int32_t *const trow = kPaged ? a.block_tables + (int64_t)x.first * a.cut.max_blocks : nullptr;
    const int lb_last = kPaged ? (x.t_end - 1) >> a.cut.log2_bs : 0;
    [[maybe_unused]] int win = kPaged ? x.key0 >> a.cut.log2_bs : 0;
    [[maybe_unused]] int tb = kPaged && win + lane <= lb_last ? __ldg(trow + win + lane) : 0;
#pragma unroll 1
    for (int j = from; j < to; ++j, ++issued) {
      before(j);
      const int s = issued % ks;
      const uint32_t full = is_k ? k_full(s) : v_full(s), empty = is_k ? k_empty(s) : v_empty(s);
      if (issued >= ks && !warp_wait(empty, ((issued / ks) - 1) & 1)) return false;
      const uint32_t dst = base + (is_k ? SL::k : SL::v) + s * SL::kTile;
      if constexpr (kPaged)
        load_paged_block<D, SL::kSub>(tm, dst, full, x.key0 + j * kTcKeys,
                                      min(kTcKeys, x.t_end - x.key0 - j * kTcKeys), win, tb, trow,
                                      lb_last, a, x.g, lane, policy);
      else if (lane == 0)
        load_packed_block(tm, dst, full, SL::kTile, (MODE == kNewest ? x.seq * a.kv_rows : x.first) + j * kTcKeys, x.g, policy);
    }
    return true;
  };
  auto nothing = [](int) {};
  auto item_blocks = [](const TileItem &x) { return (x.t_end - x.key0 + kTcKeys - 1) / kTcKeys; };
  auto load_q = [&](int t, const TileItem &x) {  // one lane
    dev::mbar_arrive_expect_tx(q_full(t), (uint32_t)tile_rows * 128u * (D / 64));
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh)
      asm volatile(
          "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
          " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(base + SL::q + t * SL::kTile + hh * SL::kSub),
          "l"(reinterpret_cast<uint64_t>(&tmq)), "r"(hh * 64), "r"(x.g * G),
          "r"(x.first + x.tok0 + t * a.tile_tokens), "r"(q_full(t))
          : "memory");
  };

  if (warp < kProducer) {
    // --------------------------------------------- softmax warps of tile t: row r each
    const int t = warp >> 2, wq = warp & 3;
    const int r = 32 * wq + lane;
    [[maybe_unused]] const int tok = r / G, h = r - tok * G;  // the row's query token in the tile, its head
    const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
    const uint32_t sb = tmem + lane_base + 128u * t;
    const uint32_t ob = tmem + lane_base + 256u + (uint32_t)(kON * t);
    float scale_log2 = fabsf(a.scale_log2);
    int blocks = 0, sc = 0, on = 0;  // as in the MMA threads
    bool ok = true;
    for (int items = 0; ok && next_item(items, it); ++items) {
      const int nb = t ? it.nb1 : it.nb0;
      const int qi = it.tok0 + (kShareKeys ? t * a.tile_tokens : 0) + tok;  // in its sequence
      const bool valid = tok < a.tile_tokens && qi < it.n;
      const int64_t token = it.first + (valid ? qi : 0);
      // keys < see are this row's
      int see = it.t_end;
      if (kPaged && valid) see = min(max(__ldg(a.context_lens + token), 0), it.t_end);
      if (!kPaged) see = min((MODE == kNewest ? it.past : 0) + qi + 1, it.t_end);
      if (kPaged) ends = valid && see > it.key0 && see < it.t_end;
      [[maybe_unused]] float v_unit = 1.f;
      if constexpr (MODE == kNewest) {
        // The row's queries as fp16, times a power of two for the largest to be in [2^14, 2^15).
        const int64_t unit = (int64_t)it.seq * a.num_kv_heads + it.g;
        const float k_unit = q8::ld(a.k_unit + unit);
        v_unit = q8::ld(a.v_unit + unit);
        if (see > q8::ld(a.nan_from + unit)) v_unit = __int_as_float(0x7fc00000);
        if (nb > 0) {
          if (!(ok = warp_wait(q_full(t), on & 1))) {
            if (lane == 0) fail(false);
            break;
          }
          const int e = widen_row<D, SL::kSub>(bp + SL::q + t * SL::kTile, r);
          scale_log2 = fabsf(a.scale_log2) * k_unit * __uint_as_float((uint32_t)(127 - e) << 23);
          dev::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(q_wide(t));
        }
      }
      float m_ref = -INFINITY;
      float ls[4] = {0.f, 0.f, 0.f, 0.f};
      auto rescale_o = [&](float f) {  // O_t (and its row-sum column) and the row sum scale by f
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          dev::tmem_ld32(ob + ch * 32, o);
          dev::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          dev::tmem_st32(ob + ch * 32, o);
        }
        if constexpr (kOnes) {
          const uint32_t sm = tmem_ld1(ob + D);
          dev::tmem_wait_ld();
          tmem_st1(ob + D, __float_as_uint(__uint_as_float(sm) * f));
        }
        dev::tmem_wait_st();
#pragma unroll
        for (int u = 0; u < 4; ++u) ls[u] *= f;
      };
      for (int i = 0; i < nb && ok; ++i) {
        const int k0 = it.key0 + blk(t, i) * kTcKeys;
        const int lim = see - 1 - k0;  // columns c <= lim are seen
        if (!(ok = warp_wait(s_full(t), (sc + i) & 1))) break;
        dev::tc_fence_after();
        const Limits l{lim, __reduce_min_sync(0xffffffffu, lim), __reduce_max_sync(0xffffffffu, lim)};
        const bool masked = l.lo < kTcKeys - 1;
        uint32_t xa[32];
        const float mx = masked ? row_max<true>(sb, l, xa) : row_max<false>(sb, l, xa);
        const float bm = mx == -INFINITY ? -INFINITY : mx * scale_log2;
        if (i > 0) {
          // The reference moves only when the block raises it by more than kTcRescale.
          // PV_t(i-1) was issued before S_t(i) by the same thread, and s_full tracks every
          // MMA issued before its commit, so O_t is stable here.
          const bool need = bm > m_ref + kTcRescale;
          if (__any_sync(0xffffffffu, need)) {
            const float m_new = fmaxf(m_ref, bm);
            rescale_o(need ? dev::ex2(m_ref - m_new) : 1.f);
            if (need) m_ref = m_new;
          }
        } else {
          m_ref = bm;
        }
        // a row that has seen no key yet takes its weights, all masked to 0, against 0
        const float m = (m_ref == -INFINITY ? 0.f : m_ref) - (kHalf ? kNewestTop : 0.f);
        auto publish_half = [&](int hf) {
          dev::tmem_wait_st();
          dev::tc_fence_before();
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(p_half(t, hf));
        };
        if (masked) {
          // V rows past the prefix are stale, past the sequence another's
          const int nk = (kPaged ? it.t_end : MODE == kNewest ? max(it.past + it.n, 0) : it.n) - k0;
          if (nk < kTcKeys) {
            const int j = blocks + blk(t, i), s = j % KSV;
            if (!(ok = warp_wait(v_full(s), (j / KSV) & 1))) break;
            const uint32_t vt = SL::v + s * SL::kTile;
#pragma unroll 1
            for (int idx = r; idx < (kTcKeys - nk) * (D / 8); idx += kTcRows) {  // (nk >= 0: see the item)
              const int row = nk + idx / (D / 8), c = idx % (D / 8);
              *reinterpret_cast<uint4 *>(bp + vt + (c >> 3) * SL::kSub + row * 128 +
                                         (((c & 7) ^ (row & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
            dev::fence_proxy_async_smem();
          }
#pragma unroll 1
          for (int c0 = 0; c0 < kTcKeys; c0 += 32) {
            uint32_t pk[16];
            if (c0 > 0) {
              dev::tmem_ld32(sb + c0, xa);
              tmem_wait_ld_regs(xa);
            }
            if (l.lo >= c0 + 31) {
              chunk_exp<false, !kOnes, kHalf>(xa, 0, 0, scale_log2, m, pk, ls);
            } else if (l.hi < c0) {
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = 0u;
            } else {
              chunk_exp<true, !kOnes, kHalf>(xa, 0, l.lim - c0, scale_log2, m, pk, ls);
            }
            tmem_st16(sb + c0 / 2, pk);  // over columns this thread has read
            if (c0 & 32) publish_half(c0 >> 6);
          }
        } else {
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t xb[32], pk[32];
            dev::tmem_ld32(sb + 64 * hf + 32, xb);
            chunk_exp<false, !kOnes, kHalf>(xa, 0, 0, scale_log2, m, pk, ls);
            tmem_wait_ld_regs(xb);
            if (hf == 0) dev::tmem_ld32(sb + 64, xa);
            chunk_exp<false, !kOnes, kHalf>(xb, 0, 0, scale_log2, m, pk + 16, ls);
            if (hf == 0) tmem_wait_ld_regs(xa);
            dev::tmem_st32(sb + 32 * hf, pk);  // over columns this thread has read
            publish_half(hf);
          }
        }
      }
      if (ok && nb > 0) ok = warp_wait(pv_done(t), on & 1);
      if (!ok && lane == 0) fail(false);
      if (!ok && !kPaged) break;
      float lsum = (ls[0] + ls[1]) + (ls[2] + ls[3]);
      if (ok && nb > 0) {
        dev::tc_fence_after();
        if constexpr (kOnes) {
          lsum = __uint_as_float(tmem_ld1(ob + D));
          dev::tmem_wait_ld();
        }
      }
      if (!kPaged && nb > 0) {
        // through shared memory, so that 4 lanes write 64 bytes of a row (a row per lane, 16
        // bytes at a time, was a line per lane: 512 sequences of 84 tokens 167 against 124 us)
        const float inv = MODE == kNewest ? (lsum == 0.f ? 0.f : v_unit / lsum) : 1.f / lsum;
        const uint64_t dst = valid ? reinterpret_cast<uint64_t>(
                                         a.out + token * a.out_stride + (int64_t)(it.g * G + h) * D)
                                   : 0;  // the lane's row
        uint8_t *const stage = bp + SL::stage + warp * 2048;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          dev::tmem_ld32(ob + ch * 32, o);
          dev::tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t w4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w4[e] = dev::pack_bf16x2(__uint_as_float(o[8 * u + 2 * e]) * inv,
                                       __uint_as_float(o[8 * u + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4 *>(stage + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(w4[0], w4[1], w4[2], w4[3]);
          }
          if (ch == D / 32 - 1) dev::tc_fence_before();
          __syncwarp();
          // the next item's P.V may overwrite O_t
          if (ch == D / 32 - 1 && lane == 0) dev::mbar_arrive(o_free(t));
          uint4 x[4];  // all loads ahead of the stores, which they may not pass
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int row = 8 * u + (lane >> 2), c = lane & 3;
            x[u] = *reinterpret_cast<const uint4 *>(stage + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint64_t to = __shfl_sync(0xffffffffu, dst, 8 * u + (lane >> 2));
            if (to)
              asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(to + ch * 64 + (lane & 3) * 16),
                           "r"(x[u].x), "r"(x[u].y), "r"(x[u].z), "r"(x[u].w)
                           : "memory");
          }
          __syncwarp();  // read before it is overwritten
        }
      }
      if constexpr (kPaged) {
        // This tile's rows (max, sum, unnormalised O) into shared memory, to be joined with the
        // other's below: the rings are done with once both tiles' MMAs are.
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(tiles_done);
        ok = warp_wait(tiles_done, 0) && ok;
        if (!ok && lane == 0) fail(false);
        reinterpret_cast<float2 *>(bp + SL::ml)[t * kTcRows + r] =
            nb > 0 && ok ? make_float2(m_ref, lsum) : make_float2(-INFINITY, 0.f);
        float4 *const row_o = reinterpret_cast<float4 *>(bp + SL::rows + (t * kTcRows + r) * D * 4);
#pragma unroll 2
        for (int ch = 0; ch < D / 32 && nb > 0 && ok; ++ch) {
          uint32_t o[32];
          dev::tmem_ld32(ob + ch * 32, o);
          dev::tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 8; ++u)
            row_o[(ch * 8 + u) ^ (r & 7)] =
                make_float4(__uint_as_float(o[4 * u]), __uint_as_float(o[4 * u + 1]),
                            __uint_as_float(o[4 * u + 2]), __uint_as_float(o[4 * u + 3]));
        }
      }
      blocks += (it.t_end - it.key0 + kTcKeys - 1) / kTcKeys;
      sc += nb;
      on += nb > 0 ? 1 : 0;
    }
  } else {
    if (kPaged && warp < kMma) {
      // ----------------------------------------------- the Q tile, the K and V rings
      if (warp == kProducer) {
        if (lane == 0) load_q(0, it);
        ++qn0;
      }
      __syncwarp();
      if (!load_ring(warp == kProducer, it, 0, item_blocks(it), nothing) && lane == 0) fail(false);
    } else if (warp == kProducer) {
      // ----------------------------------------------- items, Q tiles and the K ring
      // The next item is asked for four blocks before this one's end and found two before it, so
      // that its queries follow this one's last scores.
      TileItem next = {};
      uint32_t cta = blockIdx.x;                     // the piece to look for next, if there is
      bool more = true, begun = false, found = false, ok = true;  // one; set up; looked for
      int items = 0, asks = 0, answers = 0;
      int j = 0, nblk = 0, split = 0;                // next block; blocks, those before `next`
      auto publish = [&](const TileItem &x) {
        const int s = items & 1;
        if (items >= 2 && !warp_wait(item_empty(s), ((items >> 1) - 1) & 1)) return false;
        if (lane == 0) {
          s_item[s] = x;
          dev::mbar_arrive(item_full(s));
        }
        ++items;
        return true;
      };
      auto ask = [&] {
        ++asks;
        if (lane == 0) {
          dev::fence_proxy_async_smem();
          dev::mbar_arrive_expect_tx(clc_full, 16);
          clc_try_cancel(base + SL::clc, clc_full);
        }
      };
      while (true) {
        const int stop = found ? nblk : split;
        ok = load_ring(true, it, j, stop, [&](int b) {
          if (b == max(nblk - 4, 0)) ask();
        });
        if (!ok) break;
        j = stop;
        if (!found) {
          if (begun) {
            if (!(ok = warp_wait(clc_full, answers & 1))) break;
            ++answers;
            more = clc_answer(base + SL::clc, cta);
          }
          have = more && make_item<MODE>(a, at, cta, 0, lane, next);
          __syncwarp();  // every lane has read the answer: it may be overwritten
          if (!begun) cta_sync();
          begun = found = true;
          continue;
        }
        if (!more) break;
        found = false;
        j = nblk = split = 0;
        if (!have) {  // past the last sequence's
          ask();
          continue;
        }
        it = next;
        if (!(ok = publish(it))) break;
#pragma unroll 1
        for (int t = 0; ok && t < 2; ++t) {
          if ((t ? it.nb1 : it.nb0) == 0) continue;
          const int n = t ? qn1 : qn0;
          if (n > 0 && !(ok = warp_wait(q_free(t), (n - 1) & 1))) break;
          (t ? qn1 : qn0) = n + 1;
          if (lane == 0) load_q(t, it);
        }
        if (!ok) break;
        nblk = item_blocks(it);
        split = min(nblk, max(nblk - 2, KSK));       // the ring's free stages first
      }
      if (asks > answers) ok = warp_wait(clc_full, answers & 1) && ok;  // before the CTA may leave
      it.live = 0;
      ok = publish(it) && ok;
      if (!ok && lane == 0) fail(false);
    } else if (warp == kProducerV) {
      // ----------------------------------------------- the V ring
      bool ok = true;
      for (int items = 0; ok && next_item(items, it); ++items)
        ok = load_ring(false, it, 0, item_blocks(it), nothing);
      if (!ok && lane == 0) fail(false);
    } else {
      // ----------------------------------- tensor-core issue, one thread for each tile:
      // what one of them does between its MMAs (waits, commits) runs under the other's.  They
      // take turns, P.V and the next S of one tile at a time: left to interleave, both tiles'
      // scores came at the same moment and both softmaxes ran against each other while the
      // tensor core idled (4011 against 3080 cycles per block pair at head_dim 128).
      const int t = warp - kMma;
      constexpr uint32_t kTypes = kHalf ? 1u << 7 | 1u << 10 : 0u;  // A and B: fp16 is 0, bf16 1
      // a negative scale negates the queries instead, so that the softmax sees none
      const uint32_t id_s =
          (dev::idesc_bf16_f32(kTcRows, kTcKeys, 0) & ~kTypes) | (a.scale_log2 < 0.f ? 1u << 13 : 0u);
      constexpr uint32_t id_o = dev::idesc_bf16_f32(kTcRows, kON, 1) & ~kTypes;
      const uint64_t dq = dev::smem_desc(base + SL::q + (kShareKeys ? t * SL::kTile : 0u), 16, 1024);
      const uint64_t dk0 = dev::smem_desc(base + SL::k, 16, 1024);
      // V stage s as the MN-major B operand: the next 64 columns are V's other half
      // (head_dim 128) or the tile of ones, `lbo` bytes further on
      auto dv = [&](int s) {
        const uint32_t vs = SL::v + s * SL::kTile;
        return dev::smem_desc(base + vs, kOnes ? SL::ones - vs : SL::kSub, 1024);
      };
      const uint32_t s_tm = tmem + 128u * t, o_tm = tmem + 256u + (uint32_t)(kON * t);
      // Running counts over the items: blocks staged before this one (`blocks`), this tile's
      // score blocks (sc) and live items (on), both tiles' P.V batches (b0, b1).  Every ring
      // phase is seen by both threads of a prompt, in order.
      int blocks = 0, sc = 0, on = 0, b0 = 0, b1 = 0;
      bool ok = true;
      for (int items = 0; ok && next_item(items, it); ++items) {
        const int nblk = item_blocks(it);
        const int nb = t ? it.nb1 : it.nb0, nb0 = it.nb0, nb1 = it.nb1;
        if (lane == 0) {
          // Until the other tile has issued this many batches.  Only a matter of order, so it
          // counts (no phase to mistake) and, past its limit, goes on.
          auto await_turn = [&](int batches) {
            if (s_turn[t ^ 1] >= batches) return;
            const uint64_t t0 = dev::globaltimer_ns();
            for (uint32_t n = 1; s_turn[t ^ 1] < batches; ++n)
              if ((n & 255u) == 0 && dev::globaltimer_ns() - t0 > 2000000000ull) return;
          };
          auto wait_k = [&](int i) {
            const int j = blocks + blk(t, i);
            return tile_wait(k_full(j % KSK), (j / KSK) & 1);
          };
          auto issue_s = [&](int i) {
            const int s = (blocks + blk(t, i)) % KSK;
            issue_qk<D>(s_tm, dq, desc_add(dk0, s * SL::kTile), SL::kSub, id_s);
            if (i > 0) s_turn[t] = (t ? b1 : b0) + i;
            dev::umma_commit(s_full(t));
            dev::umma_commit(k_empty(s));
            if (kShareKeys && i + 1 == nb) dev::umma_commit(q_free(t));
          };
          if (nb > 0) {
            ok = tile_wait(kHalf ? q_wide(t) : q_full(kShareKeys ? t : 0), on & 1) && wait_k(0);
            if (ok) {
              dev::tc_fence_after();
              issue_s(0);
            }
          }
          for (int i = 0; ok && i < nb; ++i) {
            const int j = blocks + blk(t, i), s = j % KSV, ph = (sc + i) & 1;
            // every wait but one ahead of the turn, so that the turn is MMAs back to back
            if (!(ok = tile_wait(v_full(s), (j / KSV) & 1))) break;
            if (i + 1 < nb && !(ok = wait_k(i + 1))) break;
            // the last item's O has been read
            if (i == 0 && on > 0 && !(ok = tile_wait(o_free(t), (on - 1) & 1))) break;
            if (!(ok = tile_wait(p_half(t, 0), ph))) break;
            // after the other tile's turn: tile 1's i-1st, or tile 0's i-th, if it has one
            await_turn(t ? b0 + min(i + 1, nb0) : b1 + min(i, nb1));
            dev::tc_fence_after();
            const uint64_t vd = dv(s), vh = desc_add(vd, 4 * 2048u);
            // keys 0-63, then 64-127 of the block (waiting for both halves of P ahead of the
            // turn measured 9% slower)
            umma4_ts(o_tm, s_tm, s_tm + 8, s_tm + 16, s_tm + 24, vd, desc_add(vd, 2048),
                     desc_add(vd, 4096), desc_add(vd, 6144), id_o, i > 0 ? 1u : 0u);
            if (!(ok = tile_wait(p_half(t, 1), ph))) break;
            dev::tc_fence_after();
            umma4_ts(o_tm, s_tm + 32, s_tm + 40, s_tm + 48, s_tm + 56, vh, desc_add(vh, 2048),
                     desc_add(vh, 4096), desc_add(vh, 6144), id_o, 1u);
            // S_t(i+1) over S_t(i) and P_t(i), after the P.V that reads P_t(i): the MMAs of
            // one thread run in issue order
            if (i + 1 < nb) {
              issue_s(i + 1);
            } else {
              s_turn[t] = (t ? b1 : b0) + nb;
              dev::umma_commit(pv_done(t));
            }
            dev::umma_commit(v_empty(s));
          }
          // blocks of the other tile alone: seen, and let go of unread
#pragma unroll 1
          for (int i = nb; kShareKeys && ok && i < nblk; ++i) {
            const int j = blocks + i;
            if (!(ok = tile_wait(k_full(j % KSK), (j / KSK) & 1))) break;
            dev::mbar_arrive(k_empty(j % KSK));
            if (!(ok = tile_wait(v_full(j % KSV), (j / KSV) & 1))) break;
            dev::mbar_arrive(v_empty(j % KSV));
          }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        blocks += nblk;
        sc += nb;
        on += nb > 0 ? 1 : 0;
        b0 += nb0;
        b1 += nb1;
      }
      if (lane == 0) {
        if (!ok) fail(false);
        dev::umma_commit(mma_done);
      }
    }
  }

  // ---- teardown: no tensor-core op or copy may still be in flight when TMEM is freed
  if (tid == 0) (void)tile_wait(mma_done, 0);
  __syncthreads();
  if constexpr (kPaged) {
    // Both tiles' rows of a query row joined and written: the weights and the place of each row
    // first, then 16 bytes per thread.
    const int toks = min(a.tile_tokens, first.n - first.tok0), nrows = toks * G;  // tokens: sequences
    const int c16 = tid % (D / 4), r_first = tid / (D / 4);
    constexpr int kStep = kTileThreads / (D / 4);
    const float2 *const s_ml = reinterpret_cast<const float2 *>(bp + SL::ml);
    const float4 *const s_rows = reinterpret_cast<const float4 *>(bp + SL::rows);
    float2 *const s_join = reinterpret_cast<float2 *>(bp + SL::q);                 // per row: the tiles' weights
    int *const s_row = reinterpret_cast<int *>(bp + SL::q + kTcRows * 8);          // per row: b * Hq + h
    if (tid < nrows) {
      const int tok = tid / G;
      const int row = (first.first + first.tok0 + tok) * a.num_q_heads + first.g * G + (tid - tok * G);
      const float2 a0 = s_ml[tid], a1 = s_ml[kTcRows + tid];
      // a tile without keys wrote no row (weight -1 below); no key at all gives zeros and -inf
      const bool any0 = a0.x != -INFINITY || a0.y != 0.f, any1 = a1.x != -INFINITY || a1.y != 0.f;
      const float m = fmaxf(a0.x, a1.x);
      const float w0 = any0 ? dev::ex2(a0.x - m) : 0.f, w1 = any1 ? dev::ex2(a1.x - m) : 0.f;
      const float l = (any0 ? w0 * a0.y : 0.f) + (any1 ? w1 * a1.y : 0.f);
      s_join[tid] = make_float2(any0 ? w0 / l : -1.f, any1 ? w1 / l : -1.f);
      s_row[tid] = row;
      a.lse_part[(int64_t)row * a.cut.n_rows + blockIdx.y] =
          any0 || any1 ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
    const int any_ends = __syncthreads_or(ends);
#pragma unroll 4
    for (int r = r_first; r < nrows; r += kStep) {
      const float2 w = s_join[r];
      const int at = r * (D / 4) + (c16 ^ (r & 7));
      const float4 x0 = s_rows[at], x1 = s_rows[kTcRows * (D / 4) + at];
      auto join = [&](float u, float v) { return (w.x == -1.f ? 0.f : w.x * u) + (w.y == -1.f ? 0.f : w.y * v); };
      reinterpret_cast<float4 *>(a.o_part + ((int64_t)s_row[r] * a.cut.n_rows + blockIdx.y) * D)[c16] =
          make_float4(join(x0.x, x1.x), join(x0.y, x1.y), join(x0.z, x1.z), join(x0.w, x1.w));
    }
    if (any_ends) {
      __syncthreads();  // the rows are written
      for (int r = warp; r < nrows; r += kTileThreads / 32) {
        const int see = __ldg(a.context_lens + first.first + first.tok0 + r / G);
        if (see > first.key0 && see < first.t_end)
          prefix_row<D>(a, s_row[r], blockIdx.y, first.first, first.g, first.key0, see, lane);
      }
    }
  }
  // a wait that gave up leaves copies possibly in flight: waited for (bounded)
  if (warp >= kProducer && warp < kMma && lane == 0 && *s_flag) {
    if (qn0 > 0) (void)tile_wait(q_full(0), (qn0 - 1) & 1);
    if (qn1 > 0) (void)tile_wait(q_full(1), (qn1 - 1) & 1);
    const int ks = warp < kProducerV ? KSK : KSV;
    for (int s = 0; s < ks; ++s) {
      const int last = s + ((issued - 1 - s) / ks) * ks;  // the last block on stage s
      if (last >= 0 && last < issued)
        (void)tile_wait(warp < kProducerV ? k_full(s) : v_full(s), (last / ks) & 1);
    }
  }
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  if (warp == 0) dev::tmem_dealloc(tmem, 512);
}

cudaError_t read_tile_errors(uint32_t *flags, int clear) { return read_tu_errors(flags, clear); }

namespace {

bool g_tile_attr[kMaxDevices][2][3];  // dynamic smem attribute set: [D 64/128][mode]

template <int D, int MODE>
int prepare_tile_kernel() {
  std::lock_guard<std::mutex> lk(attn_mutex());
  int dev = 0;
  const int rc = current_device(&dev);
  if (rc) return rc;
  bool &set = g_tile_attr[dev][D == 64 ? 0 : 1][MODE];
  if (!set) {
    cudaError_t e = cudaFuncSetAttribute(tile_kernel<D, MODE>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)tile_smem<D, MODE>());
    if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute");
    set = true;
  }
  return PKV_OK;
}

template <int D, int MODE>
int launch_prompt(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                  const TileArgs &a, unsigned grid, cudaStream_t stream) {
  const int rc = prepare_tile_kernel<D, MODE>();
  if (rc) return rc;
  cudaError_t e;
  if constexpr (MODE == kNewest) {
    e = q8::launch_early(tile_kernel<D, MODE>, dim3(grid), kTileThreads, tile_smem<D, MODE>(), stream, tmq, tmk, tmv, a);
  } else {
    tile_kernel<D, MODE><<<grid, kTileThreads, tile_smem<D, MODE>(), stream>>>(tmq, tmk, tmv, a);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? PKV_OK : cuda_error(e, "tile_kernel launch");
}

template <int D>
int launch_prefix_tiles(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                        const TileArgs &a, dim3 grid, cudaStream_t stream) {
  const int rc = prepare_tile_kernel<D, kPrefix>();
  if (rc) return rc;
  tile_kernel<D, kPrefix><<<grid, kTileThreads, tile_smem<D, kPrefix>(), stream>>>(tmq, tmk, tmv, a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PKV_OK : cuda_error(e, "tile_kernel launch");
}

}  // namespace

int launch_prefix(const CUtensorMap &tmk, const CUtensorMap &tmv, const pkv_cache_desc &c,
                  const PrefixLaunch &l, cudaStream_t stream) {
  TileArgs a = {};
  a.start = l.group_start;
  a.num = l.num_groups;
  a.total = l.num_seqs;
  a.max_len = l.num_seqs;
  a.num_q_heads = l.num_q_heads;
  a.num_kv_heads = c.num_kv_heads;
  a.group = l.num_q_heads / c.num_kv_heads;
  a.tile_tokens = kTileRows / a.group;
  a.scale_log2 = l.scale * kLog2e;
  a.q = l.q;
  a.k = l.k_cache;
  a.v = l.v_cache;
  a.block_tables = l.block_tables;
  a.context_lens = l.context_lens;
  a.prefix_lens = l.prefix_lens;
  a.num_blocks = c.num_blocks;
  a.box_rows = std::min(c.block_size, (int32_t)kChunk);
  a.split_keys = l.split_keys;
  a.o_part = l.o_part;
  a.lse_part = l.lse_part;
  a.cut = *l.cut;
  if (l.tiles * c.num_kv_heads > 0x7fffffffLL || l.splits > 65535)
    return set_error(PKV_ERR_UNSUPPORTED, "shared prefix: too many tiles");
  CUtensorMap tmq;
  {
    std::lock_guard<std::mutex> lk(attn_mutex());
    const int rc = query_map(l.q, l.num_seqs, l.num_q_heads, c.head_dim,
                             (int64_t)l.num_q_heads * c.head_dim, a.group, a.tile_tokens, &tmq);
    if (rc) return rc;
  }
  const dim3 grid((unsigned)(l.tiles * c.num_kv_heads), (unsigned)l.splits);
  return c.head_dim == 64 ? launch_prefix_tiles<64>(tmq, tmk, tmv, a, grid, stream)
                          : launch_prefix_tiles<128>(tmq, tmk, tmv, a, grid, stream);
}

int launch_chunk(const ChunkLaunch &l, cudaStream_t stream) {
  TileArgs a = {};
  a.out = l.out;
  a.out_stride = (int64_t)l.num_q_heads * l.head_dim;
  a.start = l.query_start;
  a.num = l.num_seqs;
  a.total = (int32_t)l.num_queries;
  a.max_len = l.max_query_len;
  a.num_q_heads = l.num_q_heads;
  a.num_kv_heads = l.num_kv_heads;
  a.group = l.num_q_heads / l.num_kv_heads;
  a.tile_tokens = kTileRows / a.group;
  a.scale_log2 = l.scale * kLog2e;
  a.context_lens = l.context_lens;
  a.kv_rows = l.kv_rows;
  a.max_context = l.max_context;
  a.k_unit = l.k_unit;
  a.v_unit = l.v_unit;
  a.nan_from = l.nan_from;
  a.order = l.order;
  const int64_t tiles = l.num_queries / (2 * a.tile_tokens) + std::min<int64_t>(l.num_seqs, l.num_queries);
  if (l.num_queries > 0x7fffff00LL || tiles > 0x7fffffffLL / l.num_kv_heads)
    return set_error(PKV_ERR_UNSUPPORTED, "paged_prefill_attention_q8: too many query rows");
  const int64_t rows = (int64_t)l.num_seqs * l.kv_rows, kw = (int64_t)l.num_kv_heads * l.head_dim;
  CUtensorMap tmq, tmk, tmv;
  {
    std::lock_guard<std::mutex> lk(attn_mutex());
    int rc = query_map(l.q, l.num_queries, l.num_q_heads, l.head_dim, a.out_stride, a.group, a.tile_tokens, &tmq);
    if (!rc) rc = packed_map(l.k, rows, l.num_kv_heads, l.head_dim, kw, kTcKeys, &tmk);
    if (!rc) rc = packed_map(l.v, rows, l.num_kv_heads, l.head_dim, kw, kTcKeys, &tmv);
    if (rc) return rc;
  }
  const unsigned grid = (unsigned)(tiles * l.num_kv_heads);
  return l.head_dim == 64 ? launch_prompt<64, kNewest>(tmq, tmk, tmv, a, grid, stream)
                          : launch_prompt<128, kNewest>(tmq, tmk, tmv, a, grid, stream);
}

}  // namespace pkv

using namespace pkv;

PKV_API int prompt_attention(pkv_bf16 *out, const pkv_bf16 *q, const pkv_bf16 *k,
                             const pkv_bf16 *v, int64_t out_stride, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, const int32_t *query_start,
                             int64_t num_tokens, int32_t max_query_len, int32_t num_seqs,
                             int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                             float scale, void *stream) {
  const char *const fn = "prompt_attention";
  if (num_seqs < 0 || num_tokens < 0 || max_query_len < 0 || num_q_heads <= 0 || num_kv_heads <= 0)
    return set_error(PKV_ERR_SHAPE, "%s: bad sizes", fn);
  if (num_q_heads % num_kv_heads != 0)
    return set_error(PKV_ERR_SHAPE, "%s: num_q_heads %d is not a multiple of num_kv_heads %d", fn,
                     num_q_heads, num_kv_heads);
  if (num_q_heads / num_kv_heads > kTileRows)
    return set_error(PKV_ERR_UNSUPPORTED, "%s: query group %d > %d", fn, num_q_heads / num_kv_heads,
                     kTileRows);
  if (head_dim != 64 && head_dim != 128)
    return set_error(PKV_ERR_UNSUPPORTED, "%s: head_dim %d (built: 64, 128)", fn, head_dim);
  if (num_tokens > 0x7fffff00LL) return set_error(PKV_ERR_UNSUPPORTED, "%s: num_tokens over 2^31", fn);
  const int64_t qw = (int64_t)num_q_heads * head_dim, kw = (int64_t)num_kv_heads * head_dim;
  if (q_stride < qw || out_stride < qw || k_stride < kw || v_stride < kw)
    return set_error(PKV_ERR_SHAPE, "%s: a token stride is shorter than the token's heads", fn);
  if (q_stride % 8 || out_stride % 8 || k_stride % 8 || v_stride % 8)
    return set_error(PKV_ERR_ALIGN, "%s: token strides must be multiples of 8 elements", fn);
  if (q_stride > (1LL << 38) || out_stride > (1LL << 38) || k_stride > (1LL << 38) ||
      v_stride > (1LL << 38))
    return set_error(PKV_ERR_UNSUPPORTED, "%s: a token stride is too long", fn);
  if (num_seqs == 0 || num_tokens == 0 || max_query_len == 0) {
    clear_error();
    return PKV_OK;
  }
  if (!out || !q || !k || !v || !query_start) return set_error(PKV_ERR_NULL, "%s: NULL pointer", fn);
  if (!aligned16(out) || !aligned16(q) || !aligned16(k) || !aligned16(v))
    return set_error(PKV_ERR_ALIGN, "%s: out, q, k and v must be 16-byte aligned", fn);
  if (reinterpret_cast<uintptr_t>(query_start) & 3u)
    return set_error(PKV_ERR_ALIGN, "%s: query_start must be 4-byte aligned", fn);
  TileArgs a = {};
  a.out = out;
  a.out_stride = out_stride;
  a.start = query_start;
  a.num = num_seqs;
  a.total = (int32_t)num_tokens;
  a.max_len = max_query_len;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.group = num_q_heads / num_kv_heads;
  a.tile_tokens = kTileRows / a.group;
  a.scale_log2 = scale * kLog2e;
  // tiles of all sequences: at most the packed tokens' plus one partial tile per sequence
  const int64_t tiles = num_tokens / (2 * a.tile_tokens) + std::min<int64_t>(num_seqs, num_tokens);
  if (tiles > 0x7fffffffLL / num_kv_heads) return set_error(PKV_ERR_UNSUPPORTED, "%s: too many query rows", fn);
  CUtensorMap tmq, tmk, tmv;
  int rc;
  {
    std::lock_guard<std::mutex> lk(attn_mutex());
    rc = query_map(q, num_tokens, num_q_heads, head_dim, q_stride, a.group, a.tile_tokens, &tmq);
    if (!rc) rc = packed_map(k, num_tokens, num_kv_heads, head_dim, k_stride, kTcKeys, &tmk);
    if (!rc) rc = packed_map(v, num_tokens, num_kv_heads, head_dim, v_stride, kTcKeys, &tmv);
  }
  if (rc) return rc;
  const unsigned grid = (unsigned)(tiles * num_kv_heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = head_dim == 64 ? launch_prompt<64, kPrompt>(tmq, tmk, tmv, a, grid, s)
                      : launch_prompt<128, kPrompt>(tmq, tmk, tmv, a, grid, s);
  if (!rc) clear_error();
  return rc;
}
