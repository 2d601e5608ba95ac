// pkv_q8.cu -- the 8-bit paged cache: the quantising write (with or without rotary embedding),
// the reading back, chunked prefill over it, and its pages' copies.
//
// A page of one kv head is block_size rows of head_dim codes and one fp32 scale s; a code c
// stands for c * s.  The write gives each page that it touches the scale its rows need,
//   s = max(old s, max |x| / top),     top = 127 (int8) or 448 (e4m3),
// and the codes round(x / s); where s grew, the rows that the page held before are rounded
// anew, round((c * old s) / s).  The new rows of a page are known to one group of threads, since
// the call names sequences and not slots, so that nothing is shared between groups: no atomics,
// the same bits every time.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "attn_device.cuh"
#include "q8_device.cuh"

namespace pkv {
namespace {

constexpr int kQ8Threads = 128;   // of a CTA; a write's may have two or four times as many
constexpr int64_t kReadWide = 1 << 18;  // vectors of a call
constexpr int kHeldVecs = 4;  // of 16 held codes, a thread's loads in flight while they are rounded anew
constexpr int kRotateHeads = 4;  // q heads a thread rotates with one position's cosines and sines

// What names the tokens of a call: sequence b's newest n of context_lens[b], its rows in the
// packed tensors from row0 on.
struct Span {
  const int32_t *tables, *lens, *start;
  int64_t num_blocks, num_tokens;
  int32_t max_blocks, num_seqs, max_new, num_kv_heads, block_size, log2_bs;
};
struct Tokens {
  int32_t begin, end;  // positions; begin == end where there are none, or they do not fit
  int64_t row0;        // packed row of position `begin`
};

// The tokens of sequence b.  Without `start` one token for each sequence that has any, packed row
// b.  Lengths that do not fit the tables, the packed rows or max_new: none, and *bad is set.
__device__ __forceinline__ Tokens tokens_of(const Span &s, int b, bool *bad) {
  const int L = q8::ld(s.lens + b);
  int64_t row0 = b, n = L > 0 ? 1 : 0;
  if (s.start) {
    row0 = q8::ld(s.start + b);
    n = (int64_t)q8::ld(s.start + b + 1) - row0;
  }
  *bad = L < 0 || (int64_t)L > (int64_t)s.max_blocks * s.block_size || n < 0 || n > s.max_new || n > L ||
         row0 < 0 || row0 + n > s.num_tokens;
  Tokens t;
  t.end = *bad ? 0 : L;
  t.begin = *bad ? 0 : L - (int)n;
  t.row0 = row0;
  return t;
}

// Whether a chunk may have queries of sequence b.  (Of one that has none no page is looked at: its tables may
// be old.)
__device__ __forceinline__ bool has_queries(const Span &s, int b) { return q8::ld(s.start + b + 1) > q8::ld(s.start + b); }

// ---------------------------------------------------------------------------
// Rotary embedding of 8 coordinates: products and sums in fp32, each rounded once, then bf16.

struct Rope {
  const float *cos_sin;      // [max_position][r]: the cosine of pair i at i, its sine at r/2 + i
  const int64_t *positions;  // of the packed rows; NULL: a token's position in its sequence
  int64_t max_position;
  int32_t r, neox;
};

__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
  const float4 a = q8::ld(reinterpret_cast<const float4 *>(p)), b = q8::ld(reinterpret_cast<const float4 *>(p) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// The cosines and sines of vector c (coordinates 8c .. 8c+7, below r), of the position's row cs.
struct Angles {
  float c[8], s[8];  // neox: of the vector's pairs (e, e + r/2); else of its 4 pairs (2i, 2i + 1)
};
__device__ __forceinline__ Angles angles_of(const float *cs, int c, const Rope &p) {
  Angles a;
  if (p.neox) {
    const int e = c < p.r / 16 ? c : c - p.r / 16;
    load8(cs + 8 * e, a.c);
    load8(cs + p.r / 2 + 8 * e, a.s);
  } else {
    const float4 c4 = q8::ld(reinterpret_cast<const float4 *>(cs + 4 * c));
    const float4 s4 = q8::ld(reinterpret_cast<const float4 *>(cs + p.r / 2 + 4 * c));
    a.c[0] = c4.x, a.c[1] = c4.y, a.c[2] = c4.z, a.c[3] = c4.w;
    a.s[0] = s4.x, a.s[1] = s4.y, a.s[2] = s4.z, a.s[3] = s4.w;
  }
  return a;
}
// neox: x rotated, y being the partners' vector; lo: x holds the pairs' first coordinates.
__device__ __forceinline__ uint4 rotate_neox(const uint4 &x, const uint4 &y, const Angles &a, bool lo) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float f[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float own = __fmul_rn(k ? dev::bf16hi_to_f32(w[j]) : dev::bf16lo_to_f32(w[j]), a.c[2 * j + k]);
      const float other = __fmul_rn(k ? dev::bf16hi_to_f32(v[j]) : dev::bf16lo_to_f32(v[j]), a.s[2 * j + k]);
      f[k] = lo ? __fsub_rn(own, other) : __fadd_rn(own, other);
    }
    o[j] = dev::pack_bf16x2(f[0], f[1]);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 rotate_pairs(const uint4 &x, const Angles &a) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float e = dev::bf16lo_to_f32(w[j]), f = dev::bf16hi_to_f32(w[j]);
    o[j] = dev::pack_bf16x2(__fsub_rn(__fmul_rn(e, a.c[j]), __fmul_rn(f, a.s[j])),
                            __fadd_rn(__fmul_rn(f, a.c[j]), __fmul_rn(e, a.s[j])));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// ---------------------------------------------------------------------------
// The write.  One group of 2^log2_group threads (a warp to the whole CTA) per (sequence, touched
// page, K or V, kv head): it holds the page's new rows in registers between finding their largest
// value and rounding them, U 16-byte vectors a thread (where k is rotated, rows that do not fit are read
// a second time).
// Bound by its instructions (two thirds of the issue slots; widening, two products and two
// conversions for each pair of codes) and by HBM: 35000 tokens of 8 heads of 128 take 47 us, 4.6
// TB/s; with k rotated 80, with 24 heads of q besides 144.  256 tokens of a step: 3.2 us, and 2 more where
// pages of 16 all grow (30 more with pages of 256).

struct WriteArgs {
  Span s;
  const uint4 *k, *v;           // rows of head_dim, heads contiguous
  int64_t k_stride, v_stride;   // vectors from one token to the next
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;     // [num_blocks][num_kv_heads]
  int32_t pages;                // touched pages of a sequence, at most
  int32_t log2_group;
  uint32_t item_ctas;           // CTAs of a sequence's K (or V) groups; the ones behind rotate q
  Rope rope;
  const uint4 *q;
  uint4 *q_out;
  int64_t q_stride, q_out_stride;
  int32_t num_q_heads, q_ctas;  // CTAs (of both halves) per sequence that rotate its q rows
};

__device__ __forceinline__ uint32_t absmax(uint32_t m, const uint4 &x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)  // magnitudes compared (the sign is left over), NaN on top
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[k]));
  return m;
}

// The q rows of one sequence: a thread owns two vectors (of a rotation, both partners, so that q_out
// may be q) of kRotateHeads heads.
template <int D>
__device__ __forceinline__ void rotate_q(const WriteArgs &a, const Tokens &t, uint32_t part) {
  constexpr int V = D / 8;
  const int half = a.rope.neox ? a.rope.r / 16 : 0;
  const int runs = (a.num_q_heads + kRotateHeads - 1) / kRotateHeads;
  const int64_t n = (int64_t)(t.end - t.begin) * runs * (V / 2);
  for (int64_t i = (int64_t)part * blockDim.x + threadIdx.x; i < n; i += (int64_t)a.q_ctas * blockDim.x) {
    const int c = (int)(i % (V / 2)), ca = c < half ? c : 2 * c, cb = c < half ? c + half : 2 * c + 1;
    const int64_t run = i / (V / 2), tok = q8::quotient(run, runs);
    const int h0 = (int)(run - tok * runs) * kRotateHeads, heads = min(a.num_q_heads - h0, kRotateHeads);
    const int64_t at = t.row0 + tok;
    const int64_t pos = a.rope.positions ? q8::ld(a.rope.positions + at) : t.begin + tok;
    if (pos < 0 || pos >= a.rope.max_position) continue;  // reported by the k rows
    const uint4 *const src = a.q + at * a.q_stride + h0 * V;
    uint4 *const dst = a.q_out + at * a.q_out_stride + h0 * V;
    uint4 x[kRotateHeads], y[kRotateHeads];
#pragma unroll
    for (int h = 0; h < kRotateHeads; ++h)
      if (h < heads) {
        x[h] = src[h * V + ca];
        y[h] = src[h * V + cb];
      }
    if (8 * ca < a.rope.r) {
      const float *const cs = a.rope.cos_sin + pos * a.rope.r;
      const Angles g = angles_of(cs, ca, a.rope);
      if (half) {
#pragma unroll
        for (int h = 0; h < kRotateHeads; ++h) {
          const uint4 z = x[h];
          x[h] = rotate_neox(z, y[h], g, true);
          y[h] = rotate_neox(y[h], z, g, false);
        }
      } else {
        const Angles g2 = angles_of(cs, cb, a.rope);
#pragma unroll
        for (int h = 0; h < kRotateHeads; ++h) {
          x[h] = rotate_pairs(x[h], g);
          y[h] = rotate_pairs(y[h], g2);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < kRotateHeads; ++h)
      if (h < heads) {
        dst[h * V + ca] = x[h];
        dst[h * V + cb] = y[h];
      }
  }
}

template <int D, int KIND, bool ROPE, int U>
__global__ void __launch_bounds__(ROPE ? 2 * kQ8Threads : 4 * kQ8Threads, ROPE ? 3 : 2)
    write_q8_kernel(const __grid_constant__ WriteArgs a) {
  constexpr int V = D / 8;  // vectors of a row: 8 bf16 in, 8 codes out
  q8::await_stream();
  q8::let_next_begin();  // a step's decode: its set-up
  const int b = blockIdx.z;
  const bool is_v = blockIdx.y;
  bool bad;
  const Tokens t = tokens_of(a.s, b, &bad);
  if constexpr (ROPE) {
    if (blockIdx.x >= a.item_ctas) {
      rotate_q<D>(a, t, 2 * (blockIdx.x - a.item_ctas) + blockIdx.y);
      return;
    }
  }
  __shared__ uint32_t s_max[4 * kQ8Threads / 32];
  __shared__ alignas(8) uint8_t s_again[4 * kQ8Threads / 32][256];
  const int tid = threadIdx.x, group = 1 << a.log2_group, gt = tid & (group - 1);
  const uint32_t item = blockIdx.x * (blockDim.x >> a.log2_group) + (tid >> a.log2_group);
  const int j = (int)(item / (uint32_t)a.s.num_kv_heads), h = (int)(item - (uint32_t)j * a.s.num_kv_heads);
  bool live = j < a.pages;
  if (bad) {
    if (live && gt == 0) raise_error(PKV_DEVERR_CONTEXT_LEN);
    return;  // (the whole CTA, as below)
  }
  {  // the CTA's first group is the one of the earliest page
    const int64_t earliest = (t.begin >> a.s.log2_bs) +
                             (blockIdx.x * (blockDim.x >> a.log2_group)) / (uint32_t)a.s.num_kv_heads;
    if (t.begin == t.end || earliest << a.s.log2_bs >= t.end) return;
  }
  const int page = (t.begin >> a.s.log2_bs) + j;
  const int64_t lo = (int64_t)page << a.s.log2_bs;  // the page's first position
  const int r0 = max(t.begin - (int)min(lo, (int64_t)t.end), 0);
  const int r1 = (int)min((int64_t)t.end - lo, (int64_t)a.s.block_size);
  live = live && r1 > r0;  // rows r0 .. r1-1 are new, rows before r0 are held
  int64_t phys = live ? q8::ld(a.s.tables + (int64_t)b * a.s.max_blocks + page) : 0;
  if (phys < 0 || phys >= a.s.num_blocks) {
    if (gt == 0) raise_error(PKV_DEVERR_BLOCK_ID);
    live = false;
    phys = 0;
  }
  const int64_t unit = phys * a.s.num_kv_heads + h;
  float *const scale = (is_v ? a.v_scale : a.k_scale) + unit;
  uint8_t *const rows = (is_v ? a.v_cache : a.k_cache) + unit * a.s.block_size * D;
  const float old = live && r0 > 0 ? *scale : 0.f;  // a page that begins here has none

  // A thread's vectors are P columns of every (group / (V / P))-th row: where k is rotated, the two of
  // a rotation.
  constexpr int P = ROPE ? 2 : 1, S = U / P;
  const int c = gt % (V / P), half = ROPE && !is_v && a.rope.neox ? a.rope.r / 16 : 0;
  const int col[2] = {c < half ? c : P * c, c < half ? c + half : P * c + 1};
  const bool turns = ROPE && !is_v && 8 * col[0] < a.rope.r;
  const int64_t row0 = t.row0 + (lo + r0 - t.begin), stride = is_v ? a.v_stride : a.k_stride;
  const int rows_apart = group / (V / P), first = gt / (V / P), count = live ? r1 - r0 : 0;
  const uint4 *const src = (is_v ? a.v : a.k) + (row0 + first) * stride + h * V;
  const int64_t apart = rows_apart * stride;
  // The columns of row first + u * rows_apart.
  auto load = [&](int u, uint4 *x) {
#pragma unroll
    for (int p = 0; p < P; ++p) x[p] = q8::ld(src + u * apart + col[p]);
  };
  // The same, rotated; false, and zeros, where the row's position has no angles.
  auto turn = [&](int u, uint4 *x) {
    if (!ROPE || is_v) return true;
    const int r = first + u * rows_apart;
    const int64_t pos = a.rope.positions ? q8::ld(a.rope.positions + row0 + r) : lo + r0 + r;
    if (pos < 0 || pos >= a.rope.max_position) {
      raise_error(PKV_DEVERR_POSITION);
      x[0] = x[P - 1] = make_uint4(0, 0, 0, 0);
      return false;
    }
    if (!turns) return true;
    const float *const cs = a.rope.cos_sin + pos * a.rope.r;
    const Angles g = angles_of(cs, col[0], a.rope);
    if (half) {
      const uint4 y = x[0];
      x[0] = rotate_neox(y, x[P - 1], g, true);
      x[P - 1] = rotate_neox(x[P - 1], y, g, false);
    } else {
      x[0] = rotate_pairs(x[0], g);
      x[P - 1] = rotate_pairs(x[P - 1], angles_of(cs, col[1], a.rope));
    }
    return true;
  };
  uint4 x[U];
  uint32_t m = 0, skip = 0;
#pragma unroll
  for (int u = 0; u < S; ++u) {
#pragma unroll
    for (int p = 0; p < P; ++p) x[P * u + p] = make_uint4(0, 0, 0, 0);
    if (first + u * rows_apart < count) load(u, x + P * u);
  }
  if constexpr (ROPE) {
#pragma unroll
    for (int u = 0; u < S; ++u)
      if (first + u * rows_apart < count && !turn(u, x + P * u)) skip |= 1u << u;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) m = absmax(m, x[u]);
  if constexpr (ROPE) {  // (without a rotation there are threads enough: write_threads)
    for (int u = S; first + u * rows_apart < count; ++u) {
      uint4 y[P];
      load(u, y);
      turn(u, y);
#pragma unroll
      for (int p = 0; p < P; ++p) m = absmax(m, y[p]);
    }
  }
  m &= 0x7fff7fffu;
  m = max(m & 0xffffu, m >> 16);  // bf16 patterns order as whole numbers, infinity and NaN on top
  m = __reduce_max_sync(0xffffffffu, m);
  if (group > 32) {  // uniform over the grid
    if ((tid & 31) == 0) s_max[tid >> 5] = m;
    __syncthreads();
    for (int w = 0; w < group / 32; ++w) m = max(m, s_max[((tid >> a.log2_group) << (a.log2_group - 5)) + w]);
  } else {
    __syncwarp();  // every lane has read the old scale
  }
  if (!live) return;
  constexpr float kTop = q8::top<KIND>();
  float to = old;
  if (m >= 0x7f80u || old != old) {
    to = __int_as_float(0x7fc00000);  // what is not finite has no place under a shared scale
  } else if (m > 0u) {
    to = fmaxf(old, fmaxf(__fdiv_rn(__uint_as_float(m << 16), kTop), 1.17549435e-38f));
  }
  if (gt == 0 && !(to == old && r0 > 0)) *scale = to;
  const q8::Inverse by = q8::inverse_of(to == 0.f ? 1.f : to);
  uint2 *const dst = reinterpret_cast<uint2 *>(rows + (int64_t)(r0 + first) * D);
  // The rare rows next to a border between codes are noted and divided at the end, from their loads on
  // (with the divisions behind every vector the code left the instruction cache: 56 us, 49 without).
  auto store = [&](int u, const uint4 *x, bool exact) {
    bool all = true;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      bool sure = true;
      dst[u * rows_apart * V + col[p]] = exact ? q8::divided8<KIND>(x[p], by.s) : q8::encode8<KIND>(x[p], by, &sure);
      all = all && sure;
    }
    return all;
  };
  uint32_t again = 0;
#pragma unroll
  for (int u = 0; u < S; ++u)
    if (first + u * rows_apart < count && !(skip >> u & 1u) && !store(u, x + P * u, false)) again |= 1u << u;
#pragma unroll 1
  for (int u = again ? __ffs(again) - 1 : S; ROPE ? first + u * rows_apart < count : u < S; ++u) {
    if (u < S && !(again >> u & 1u)) continue;
    uint4 y[P];
    load(u, y);
    if (turn(u, y) && (u < S || !store(u, y, false))) store(u, y, true);
  }
  if (to > old && r0 > 0) {  // the rows held before, in units of the new scale
    // A code's new one goes by the code alone: each warp divides for the 256 there are.  (Divided element by
    // element, 256 sequences of one token whose pages of 16 all grew took 24 us, of 256 rows 200.)
    uint8_t *const map = s_again[tid >> 5];
    uint2 w = make_uint2(0x03020100u + 0x08080808u * (tid & 31), 0x07060504u + 0x08080808u * (tid & 31));
    auto anew = [&](uint32_t c) {
      const uint32_t z = q8::prep<KIND>(c);
      const float2 f = q8::f16x2_to_f32(q8::pair<KIND, 0>(z)), g = q8::f16x2_to_f32(q8::pair<KIND, 1>(z));
      return q8::encode4<KIND>(__fdiv_rn(__fmul_rn(f.x, old), to), __fdiv_rn(__fmul_rn(f.y, old), to),
                               __fdiv_rn(__fmul_rn(g.x, old), to), __fdiv_rn(__fmul_rn(g.y, old), to));
    };
    w.x = anew(w.x);
    w.y = anew(w.y);
    reinterpret_cast<uint2 *>(map)[tid & 31] = w;
    __syncwarp();
    auto mapped = [&](uint32_t c) {
      return map[c & 255] | map[c >> 8 & 255] << 8 | map[c >> 16 & 255] << 16 | (uint32_t)map[c >> 24] << 24;
    };
    const int vecs = r0 * (D / 16);
    for (int e = gt; e < vecs; e += kHeldVecs * group) {
      uint4 v[kHeldVecs];
#pragma unroll
      for (int u = 0; u < kHeldVecs; ++u)
        if (e + u * group < vecs) v[u] = reinterpret_cast<const uint4 *>(rows)[e + u * group];
#pragma unroll
      for (int u = 0; u < kHeldVecs; ++u)
        if (e + u * group < vecs)
          reinterpret_cast<uint4 *>(rows)[e + u * group] =
              make_uint4(mapped(v[u].x), mapped(v[u].y), mapped(v[u].z), mapped(v[u].w));
    }
  }
}

// ---------------------------------------------------------------------------
// Reading back: bf16(code * scale).  One group of threads per (sequence, page, K or V, run of kv
// heads), up to 16 loads of a thread in flight.  Bound by HBM, which takes two bytes for each one
// read: 16 contexts of 1 to 8192 tokens, 8 heads of 128, 31.5 us, 5.0 TB/s (27.6 with 256-token pages).
// For the prefill, whole contexts of the sequences with queries as fp16 rows, row seq * out_rows + t
// being token t's: code * (scale / unit) for the largest scale of the (sequence, kv head) as unit, so
// that codes keep 11 bits (bf16 rows, of 8, doubled the error of the output).

struct ReadArgs {
  Span s;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  uint4 *k_out, *v_out;
  int64_t k_stride, v_stride;  // packed rows: vectors from one token to the next
  int32_t out_rows;            // whole contexts in fp16; 0: bf16 rows of the newest tokens
  const float *k_unit, *v_unit;
  int32_t pages;
  int32_t log2_heads, runs;    // kv heads of an item: a power of two; items of a page
  int32_t log2_group;
};

// The units: the largest scale of each (sequence, kv head)'s pages.  One CTA per sequence; thread
// (page % rows, kv head), joined through shared memory.  And the sequence's place in the order of the
// tiles, longest contexts first (the tiles of 4 chunks over 1600 to 5800 tokens took 174 us in the
// batch's order, whose last was not the shortest), with its query rows: moved behind those of every
// sequence before it, cut and flagged where they do not fit (as in disjoint_group).
struct UnitArgs {
  Span s;
  const float *k_scale, *v_scale;
  float *k_unit, *v_unit;
  int32_t *nan_from;  // the first key of a page whose scale is NaN
  int4 *order;
  int32_t num_queries, max_query_len;
  int32_t ahead;  // sequences of earlier groups: theirs are the entries of s.start below 0
};
constexpr int kUnitThreads = 1024;
__global__ void __launch_bounds__(kUnitThreads) units_q8_kernel(const __grid_constant__ UnitArgs a) {
  static_assert(kUnitThreads == 32 * 32, "a warp joins the warps' results");
  q8::await_stream();
  __shared__ float s_k[kUnitThreads], s_v[kUnitThreads];
  __shared__ int s_before[32], s_rank[32], s_nan[kUnitThreads];
  const int b = blockIdx.x, H = a.s.num_kv_heads, tid = threadIdx.x;
  const int cap = (int)min((int64_t)a.s.max_blocks * a.s.block_size, (int64_t)a.s.max_new);
  const int L = min(max(q8::ld(a.s.lens + b), 0), cap);
  const int pages = has_queries(a.s, b) ? (int)(((int64_t)L + a.s.block_size - 1) >> a.s.log2_bs) : 0;
  const int32_t *const row = a.s.tables + (int64_t)b * a.s.max_blocks;
  int before = 0, rank = 0;  // the furthest end of the sequences before b; how many are taken before b
  for (int i = tid - a.ahead; i < 0; i += kUnitThreads)
    before = max(before, min(max(q8::ld(a.s.start + i + 1), 0), a.num_queries));
  for (int i = tid; i < a.s.num_seqs; i += kUnitThreads) {
    if (i < b) before = max(before, min(max(q8::ld(a.s.start + i + 1), 0), a.num_queries));
    const int Li = min(max(q8::ld(a.s.lens + i), 0), cap);
    rank += Li > L || (Li == L && i < b);
  }
  before = __reduce_max_sync(0xffffffffu, before);
  rank = __reduce_add_sync(0xffffffffu, rank);
  if ((tid & 31) == 0) {
    s_before[tid >> 5] = before;
    s_rank[tid >> 5] = rank;
  }
  __syncthreads();
  if (tid < 32) {
    before = __reduce_max_sync(0xffffffffu, s_before[tid]);
    rank = __reduce_add_sync(0xffffffffu, s_rank[tid]);
    if (tid == 0) {
      const int s0 = q8::ld(a.s.start + b), e0 = q8::ld(a.s.start + b + 1), e = min(max(e0, 0), a.num_queries);
      const int s = min(max(max(s0, 0), before), a.num_queries), n = min(max(e - s, 0), a.max_query_len);
      if (s != s0 || s + n != e0) raise_error(PKV_DEVERR_CONTEXT_LEN);
      a.order[rank] = make_int4(b, s, n, 0);
    }
  }
  for (int h0 = 0; h0 < H; h0 += kUnitThreads) {  // (heads past 1024 in further rounds)
    const int wide = min(H - h0, kUnitThreads), rows = kUnitThreads / wide;
    const int h = tid % wide, r = tid / wide;
    float k = 0.f, v = 0.f;
    int bad = pages;  // the first page of scale NaN
    if (r < rows)
#pragma unroll 4
      for (int p = r; p < pages; p += rows) {
        int64_t phys = q8::ld(row + p);
        if (phys < 0 || phys >= a.s.num_blocks) phys = 0;  // (flagged by the reading)
        const float ks = q8::ld(a.k_scale + phys * H + h0 + h), vs = q8::ld(a.v_scale + phys * H + h0 + h);
        if (ks != ks || vs != vs) bad = min(bad, p);
        k = fmaxf(k, ks);
        v = fmaxf(v, vs);
      }
    s_k[tid] = k;
    s_v[tid] = v;
    s_nan[tid] = bad;
    __syncthreads();
    int half = 1;
    while (2 * half < rows) half *= 2;
    for (; half > 0 && rows > 1; half /= 2) {
      if (r < half && r + half < rows) {
        s_k[tid] = k = fmaxf(k, s_k[tid + half * wide]);
        s_v[tid] = v = fmaxf(v, s_v[tid + half * wide]);
        s_nan[tid] = bad = min(bad, s_nan[tid + half * wide]);
      }
      __syncthreads();
    }
    if (tid < wide) {
      a.k_unit[(int64_t)b * H + h0 + tid] = k;
      a.v_unit[(int64_t)b * H + h0 + tid] = v;
      a.nan_from[(int64_t)b * H + h0 + tid] = (int32_t)min((int64_t)bad << a.s.log2_bs, (int64_t)0x7fffffff);
    }
    __syncthreads();
  }
}

template <int D, int KIND, bool WHOLE, int U>
__global__ void __launch_bounds__(kQ8Threads, U == 16 ? 5 : 8) read_q8_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int V = D / 8;  // vectors of a row: 8 codes in, 8 bf16 out
  q8::await_stream();
  const int tid = threadIdx.x, lane = tid & 31, group = 1 << a.log2_group, gt = tid & (group - 1);
  const int b = blockIdx.z;
  const bool is_v = blockIdx.y;
  const uint32_t item = blockIdx.x * (blockDim.x >> a.log2_group) + (tid >> a.log2_group);
  const int j = (int)(item / (uint32_t)a.runs), h0 = (int)(item - (uint32_t)j * a.runs) << a.log2_heads;
  if (j >= a.pages) return;  // (whole warps, here and below)
  Tokens t;
  if constexpr (WHOLE) {  // lengths past the tables are cut, as the attention does
    if (!has_queries(a.s, b)) return;
    const int cap = (int)min((int64_t)a.s.max_blocks * a.s.block_size, (int64_t)a.s.max_new);
    t.begin = 0;
    t.end = min(max(q8::ld(a.s.lens + b), 0), cap);
    t.row0 = (int64_t)b * a.out_rows;
  } else {
    bool bad;
    t = tokens_of(a.s, b, &bad);
    if (bad && gt == 0) raise_error(PKV_DEVERR_CONTEXT_LEN);
  }
  const int page = (t.begin >> a.s.log2_bs) + j;
  const int64_t lo = (int64_t)page << a.s.log2_bs;
  const int r0 = max(t.begin - (int)min(lo, (int64_t)t.end), 0);
  const int r1 = (int)min((int64_t)t.end - lo, (int64_t)a.s.block_size);
  if (r1 <= r0) return;
  const int64_t phys = q8::ld(a.s.tables + (int64_t)b * a.s.max_blocks + page);
  int64_t from = phys;
  if (phys < 0 || phys >= a.s.num_blocks) {
    if (gt == 0) raise_error(PKV_DEVERR_BLOCK_ID);
    from = 0;
  }
  const int heads = min(1 << a.log2_heads, a.s.num_kv_heads - h0);
  const int64_t unit = from * a.s.num_kv_heads + h0;
  float scale = 0.f;  // lane l: head h0 + l's
  if (lane < heads) {
    scale = q8::ld((is_v ? a.v_scale : a.k_scale) + unit + lane);
    if constexpr (WHOLE) {
      const float of = q8::ld((is_v ? a.v_unit : a.k_unit) + (int64_t)b * a.s.num_kv_heads + h0 + lane);
      scale = of > 0.f ? __fdiv_rn(scale, of) : scale * 0.f;
    }
  }
  const uint2 *const src = reinterpret_cast<const uint2 *>((is_v ? a.v_cache : a.k_cache) + unit * a.s.block_size * D) + gt % V;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  uint4 *const dst = (is_v ? a.v_out : a.k_out) + (t.row0 + lo - t.begin) * stride + h0 * V + gt % V;
  // The heads' pages are one run of rows; a thread's vectors are one column of every (group / V)-th.
  const int rows_apart = group / V, rows = heads << a.s.log2_bs;
  auto run = [&](auto whole, int r) {  // whole: every row of them is wanted
    constexpr bool kAll = decltype(whole)::value;
    uint2 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = r + u * rows_apart, in = at & (a.s.block_size - 1);
      if (kAll || (at < rows && in >= r0 && in < r1)) x[u] = __ldcs(src + at * V);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = r + u * rows_apart, in = at & (a.s.block_size - 1), h = at >> a.s.log2_bs;
      const float s = __shfl_sync(0xffffffffu, scale, h & 31);  // (a warp's rows are of one head)
      if (!kAll && (at >= rows || in < r0 || in >= r1)) continue;
      // (zeros for a page of scale NaN: a NaN among the keys would reach rows that do not see it)
      const bool none = WHOLE && s != s;
      const uint64_t s2 = none ? 0u : q8::f32x2(s, s);
      const uint32_t w[2] = {none ? 0u : x[u].x, none ? 0u : x[u].y};
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t z = q8::prep<KIND>(w[k]);
        const float2 f = q8::f16x2_to_f32(q8::pair<KIND, 0>(z)), g = q8::f16x2_to_f32(q8::pair<KIND, 1>(z));
        const float2 p = q8::split(q8::mul2(q8::f32x2(f.x, f.y), s2));
        const float2 q = q8::split(q8::mul2(q8::f32x2(g.x, g.y), s2));
        o[2 * k] = WHOLE ? q8::pack_f16x2(p.x, p.y) : dev::pack_bf16x2(p.x, p.y);
        o[2 * k + 1] = WHOLE ? q8::pack_f16x2(q.x, q.y) : dev::pack_bf16x2(q.x, q.y);
      }
      uint4 *const to = dst + in * stride + h * V;
      if (WHOLE)  // (the tiles read it next)
        *to = make_uint4(o[0], o[1], o[2], o[3]);
      else
        __stcs(to, make_uint4(o[0], o[1], o[2], o[3]));
    }
  };
  for (int r = gt / V; r < rows; r += U * rows_apart) {
    if (r1 - r0 == a.s.block_size && r - gt / V + U * rows_apart <= rows)
      run(std::true_type{}, r);
    else
      run(std::false_type{}, r);
  }
}

int log2_group_of(int64_t vectors, int per_thread, int threads) {  // of one item's threads: a warp to a CTA
  int r = 5;
  while (r < ilog2(threads) && ((int64_t)per_thread << r) < vectors) ++r;
  return r;
}

// pick(head_dim, kind), with both as constants.
template <typename F>
auto of_kinds(int32_t d, int32_t kind, F pick) {
  using std::integral_constant;
  constexpr integral_constant<int, 64> d64{};
  constexpr integral_constant<int, 128> d128{};
  constexpr integral_constant<int, PKV_Q8_INT8> i8{};
  constexpr integral_constant<int, PKV_Q8_E4M3> e4{};
  if (d == 64) return kind == PKV_Q8_INT8 ? pick(d64, i8) : pick(d64, e4);
  return kind == PKV_Q8_INT8 ? pick(d128, i8) : pick(d128, e4);
}

// Pages that `n` consecutive tokens touch, at most.
int64_t touched(int64_t n, int bs) { return n <= 0 ? 0 : (n + bs - 2) / bs + 1; }

Span span_of(const int32_t *tables, int32_t max_blocks, const int32_t *lens, const int32_t *start,
             int32_t max_new, int32_t num_seqs, int64_t num_tokens, const pkv_cache_desc &c) {
  Span s;
  s.tables = tables;
  s.lens = lens;
  s.start = start;
  s.num_blocks = c.num_blocks;
  s.num_tokens = num_tokens;
  s.max_blocks = max_blocks;
  s.num_seqs = num_seqs;
  s.max_new = max_new;
  s.num_kv_heads = c.num_kv_heads;
  s.block_size = c.block_size;
  s.log2_bs = ilog2(c.block_size);
  return s;
}

bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// What the write and the reading back check alike: x, y are the packed tensors.
int check_span(const void *x, const void *y, int64_t x_stride, int64_t y_stride, const int32_t *start,
               int64_t num_tokens, int32_t max_new, const int32_t *tables, int32_t max_blocks,
               const int32_t *lens, int32_t num_seqs, const pkv_q8_cache *q, const pkv_cache_desc *c,
               const char *fn) {
  int rc = check_q8(q, c, num_seqs, fn);
  if (rc) return rc;
  if (num_seqs < 0 || num_tokens < 0 || max_new < 0)
    return set_error(PKV_ERR_SHAPE, "%s: negative count", fn);
  if (max_blocks <= 0) return set_error(PKV_ERR_SHAPE, "%s: max_blocks_per_seq must be positive", fn);
  if (!start && max_new > 1)
    return set_error(PKV_ERR_SHAPE, "%s: more than one token a sequence needs query_start", fn);
  if (!start && num_tokens < num_seqs)
    return set_error(PKV_ERR_SHAPE, "%s: fewer rows than sequences, and no query_start", fn);
  const int64_t row = (int64_t)c->num_kv_heads * c->head_dim;
  if (num_tokens > 1 && (x_stride < row || y_stride < row))
    return set_error(PKV_ERR_SHAPE, "%s: a token stride is under num_kv_heads * head_dim", fn);
  if (num_seqs == 0 || num_tokens == 0 || max_new == 0) return PKV_OK;
  if (x_stride % 8 || y_stride % 8)
    return set_error(PKV_ERR_ALIGN, "%s: token strides must be multiples of 8 elements", fn);
  if (!x || !y || !tables || !lens) return set_error(PKV_ERR_NULL, "%s: NULL tensor pointer", fn);
  if (!aligned16(x) || !aligned16(y)) return set_error(PKV_ERR_ALIGN, "%s: k and v must be 16-byte aligned", fn);
  if (misaligned4(tables) || misaligned4(lens) || misaligned4(start))
    return set_error(PKV_ERR_ALIGN, "%s: int32 tensors must be 4-byte aligned", fn);
  const int64_t pages = std::min<int64_t>(touched(max_new, c->block_size), max_blocks);
  if (pages * num_seqs > 0x7fffffffLL / (2 * c->num_kv_heads))
    return set_error(PKV_ERR_UNSUPPORTED, "%s: more than 2^31-1 pages of heads", fn);
  return PKV_OK;
}

// out_rows > 0: whole contexts in fp16, units at k_unit and v_unit.
int launch_read(const Span &s, const pkv_q8_cache &q, const pkv_cache_desc &c, void *k_out, void *v_out,
                int64_t k_stride, int64_t v_stride, int32_t out_rows, const float *k_unit, const float *v_unit,
                int64_t pages, cudaStream_t stream) {
  ReadArgs a = {};
  a.s = s;
  a.k_cache = static_cast<const uint8_t *>(q.k_cache);
  a.v_cache = static_cast<const uint8_t *>(q.v_cache);
  a.k_scale = q.k_scale;
  a.v_scale = q.v_scale;
  a.k_out = static_cast<uint4 *>(k_out);
  a.v_out = static_cast<uint4 *>(v_out);
  a.k_stride = k_stride / 8;
  a.v_stride = v_stride / 8;
  a.out_rows = out_rows;
  a.k_unit = k_unit;
  a.v_unit = v_unit;
  a.pages = (int32_t)pages;
  // 16 vectors a thread, of several heads where a page of one has fewer; 4 where the call is too short for
  // that to fill the GPU (8 heads of 128, pages of 16: one context of 100 tokens 3.3 us by 16 and 2.6 by
  // 4, 16 of 300 5.4 and 6.4, 16 of 8192 at most 34 and 47).  With registers for 8 or 4 where all heads
  // together have fewer.
  const int64_t page_vecs = (int64_t)s.block_size * c.head_dim / 8;
  int per_thread = pages * s.num_seqs * 2 * c.num_kv_heads * page_vecs >= kReadWide ? 16 : 4;
  while ((page_vecs << (a.log2_heads + 1)) <= 32 * per_thread && (1 << a.log2_heads) < c.num_kv_heads) ++a.log2_heads;
  while (per_thread > 4 && (page_vecs << a.log2_heads) <= 16 * per_thread) per_thread /= 2;
  a.runs = (c.num_kv_heads + (1 << a.log2_heads) - 1) >> a.log2_heads;
  a.log2_group = log2_group_of(page_vecs << a.log2_heads, per_thread, kQ8Threads);
  const int per = kQ8Threads >> a.log2_group;
  const dim3 ctas((unsigned)((pages * a.runs + per - 1) / per), 2, (unsigned)s.num_seqs);
  auto pick = [&](auto d, auto kind) -> void (*)(const ReadArgs) {
    if (out_rows)
      return per_thread == 16  ? read_q8_kernel<d(), kind(), true, 16>
             : per_thread == 8 ? read_q8_kernel<d(), kind(), true, 8>
                               : read_q8_kernel<d(), kind(), true, 4>;
    return per_thread == 16  ? read_q8_kernel<d(), kind(), false, 16>
           : per_thread == 8 ? read_q8_kernel<d(), kind(), false, 8>
                             : read_q8_kernel<d(), kind(), false, 4>;
  };
  void (*const kern)(const ReadArgs) = of_kinds(c.head_dim, q.kind, pick);
  const cudaError_t e = q8::launch_early(kern, ctas, kQ8Threads, 0, stream, a);
  if (e != cudaSuccess) return cuda_error(e, "read_q8_kernel launch");
  return PKV_OK;
}

}  // namespace

cudaError_t read_q8_errors(uint32_t *flags, int clear) { return read_tu_errors(flags, clear); }

int check_q8_sizes(const pkv_cache_desc *c, const char *fn) {
  if (c->num_blocks <= 0 || c->num_kv_heads <= 0 || c->block_size <= 0 || c->head_dim <= 0)
    return set_error(PKV_ERR_SHAPE, "%s: cache sizes must be positive", fn);
  if (c->head_dim != 64 && c->head_dim != 128)
    return set_error(PKV_ERR_UNSUPPORTED, "%s: head_dim %d (built: 64, 128)", fn, c->head_dim);
  if (c->block_size < 8 || c->block_size > 256 || (c->block_size & (c->block_size - 1)))
    return set_error(PKV_ERR_UNSUPPORTED, "%s: block_size %d (built: powers of two 8..256)", fn, c->block_size);
  if (c->num_blocks > 0x7fffffffLL / ((int64_t)c->num_kv_heads * c->block_size))
    return set_error(PKV_ERR_UNSUPPORTED, "%s: pool has more than 2^31-1 rows", fn);
  return PKV_OK;
}

int check_q8(const pkv_q8_cache *q, const pkv_cache_desc *c, int32_t num_seqs, const char *fn) {
  if (!q || !c) return set_error(PKV_ERR_NULL, "%s: cache descriptor is NULL", fn);
  if (q->kind != PKV_Q8_E4M3 && q->kind != PKV_Q8_INT8)
    return set_error(PKV_ERR_UNSUPPORTED, "%s: unknown kind of codes %d", fn, q->kind);
  const int rc = check_q8_sizes(c, fn);
  if (rc) return rc;
  if (num_seqs > 65535) return set_error(PKV_ERR_UNSUPPORTED, "%s: num_seqs > 65535", fn);
  if (num_seqs <= 0) return PKV_OK;
  if (!q->k_cache || !q->v_cache || !q->k_scale || !q->v_scale)
    return set_error(PKV_ERR_NULL, "%s: NULL cache or scale pointer", fn);
  if (!aligned16(q->k_cache) || !aligned16(q->v_cache) || misaligned4(q->k_scale) || misaligned4(q->v_scale))
    return set_error(PKV_ERR_ALIGN, "%s: caches must be 16-byte, scales 4-byte aligned", fn);
  return PKV_OK;
}

int check_write_q8(const WriteQ8 &w, const char *fn) {
  int rc = check_span(w.k, w.v, w.k_stride, w.v_stride, w.query_start, w.num_tokens, w.max_query_len,
                      w.block_tables, w.max_blocks, w.context_lens, w.num_seqs, w.cache, w.desc, fn);
  if (rc || !w.rope) return rc;
  if (w.rotary_dim <= 0 || w.rotary_dim % 16 != 0 || w.rotary_dim > w.desc->head_dim)
    return set_error(PKV_ERR_UNSUPPORTED, "%s: rotary_dim %d must be a positive multiple of 16 <= head_dim", fn,
                     w.rotary_dim);
  if (w.max_position <= 0) return set_error(PKV_ERR_SHAPE, "%s: max_position <= 0", fn);
  if (w.q && w.num_q_heads <= 0) return set_error(PKV_ERR_SHAPE, "%s: num_q_heads <= 0", fn);
  if (w.q && w.num_tokens > 1 && (w.q_stride < (int64_t)w.num_q_heads * w.desc->head_dim ||
                                  w.q_out_stride < (int64_t)w.num_q_heads * w.desc->head_dim))
    return set_error(PKV_ERR_SHAPE, "%s: a token stride of q is under num_q_heads * head_dim", fn);
  if (w.num_tokens == 0 || w.num_seqs == 0 || w.max_query_len == 0) return PKV_OK;
  if (!w.cos_sin || (w.q && !w.q_out)) return set_error(PKV_ERR_NULL, "%s: NULL cos_sin/q_out", fn);
  if (!aligned16(w.cos_sin) || !aligned16(w.q) || !aligned16(w.q_out) ||
      (reinterpret_cast<uintptr_t>(w.positions) & 7u))
    return set_error(PKV_ERR_ALIGN, "%s: cos_sin and q 16-byte, positions 8-byte aligned", fn);
  if (w.q && (w.q_stride % 8 || w.q_out_stride % 8))
    return set_error(PKV_ERR_ALIGN, "%s: token strides must be multiples of 8 elements", fn);
  return PKV_OK;
}

// Threads of a write's CTA: as many as hold an item's vectors, 8 each; with a rotation (80 registers, not 64)
// up to 256, whose rows past those are read twice.
static int write_threads(int64_t vecs, bool rope) {
  return vecs <= 8 * kQ8Threads ? kQ8Threads : vecs <= 16 * kQ8Threads || rope ? 2 * kQ8Threads : 4 * kQ8Threads;
}

int launch_write_q8(const WriteQ8 &w, cudaStream_t stream) {
  if (w.num_tokens == 0 || w.num_seqs == 0 || w.max_query_len == 0) return PKV_OK;
  const pkv_cache_desc &c = *w.desc;
  WriteArgs a = {};
  a.s = span_of(w.block_tables, w.max_blocks, w.context_lens, w.query_start, w.max_query_len, w.num_seqs,
                w.num_tokens, c);
  a.k = reinterpret_cast<const uint4 *>(w.k);
  a.v = reinterpret_cast<const uint4 *>(w.v);
  a.k_stride = w.k_stride / 8;
  a.v_stride = w.v_stride / 8;
  a.k_cache = static_cast<uint8_t *>(w.cache->k_cache);
  a.v_cache = static_cast<uint8_t *>(w.cache->v_cache);
  a.k_scale = w.cache->k_scale;
  a.v_scale = w.cache->v_scale;
  a.pages = (int32_t)std::min<int64_t>(touched(w.max_query_len, c.block_size), w.max_blocks);
  const int64_t vecs = (int64_t)std::min(c.block_size, w.max_query_len) * c.head_dim / 8;  // of an item
  const int per_thread = vecs <= 32 ? 1 : vecs <= 128 ? 4 : 8;
  const int threads = write_threads(vecs, w.rope);
  a.log2_group = log2_group_of(vecs, per_thread, threads);
  const int per = threads >> a.log2_group;
  a.item_ctas = (uint32_t)(((int64_t)a.pages * c.num_kv_heads + per - 1) / per);
  uint32_t ctas = a.item_ctas;
  if (w.rope) {
    a.rope.cos_sin = w.cos_sin;
    a.rope.positions = w.positions;
    a.rope.max_position = w.max_position;
    a.rope.r = w.rotary_dim;
    a.rope.neox = w.neox_style ? 1 : 0;
    if (w.q) {
      a.q = reinterpret_cast<const uint4 *>(w.q);
      a.q_out = reinterpret_cast<uint4 *>(w.q_out);
      a.q_stride = w.q_stride / 8;
      a.q_out_stride = w.q_out_stride / 8;
      a.num_q_heads = w.num_q_heads;
      const int64_t units =
          (int64_t)w.max_query_len * ((w.num_q_heads + kRotateHeads - 1) / kRotateHeads) * (c.head_dim / 16);
      a.q_ctas = 2 * (int32_t)std::min<int64_t>((units + 2 * threads - 1) / (2 * threads), 16384);
      ctas += (uint32_t)a.q_ctas / 2;
    }
  }
  auto pick = [&](auto d, auto kind) -> void (*)(const WriteArgs) {
    if (w.rope)
      return per_thread == 1   ? write_q8_kernel<d(), kind(), true, 2>
             : per_thread == 4 ? write_q8_kernel<d(), kind(), true, 4>
                               : write_q8_kernel<d(), kind(), true, 8>;
    return per_thread == 1   ? write_q8_kernel<d(), kind(), false, 1>
           : per_thread == 4 ? write_q8_kernel<d(), kind(), false, 4>
                             : write_q8_kernel<d(), kind(), false, 8>;
  };
  void (*const kern)(const WriteArgs) = of_kinds(c.head_dim, w.cache->kind, pick);
  const cudaError_t e = q8::launch_early(kern, dim3(ctas, 2, (unsigned)w.num_seqs), threads, 0, stream, a);
  if (e != cudaSuccess) return cuda_error(e, "write_q8_kernel launch");
  return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

PKV_API int paged_kv_write_q8(const pkv_bf16 *k, const pkv_bf16 *v, int64_t k_stride, int64_t v_stride,
                              const int32_t *query_start, int64_t num_tokens, int32_t max_query_len,
                              const int32_t *block_tables, int32_t max_blocks_per_seq,
                              const int32_t *context_lens, int32_t num_seqs, const pkv_q8_cache *cache,
                              const pkv_cache_desc *desc, void *stream) {
  WriteQ8 w = {};
  w.k = k, w.v = v, w.k_stride = k_stride, w.v_stride = v_stride;
  w.query_start = query_start, w.num_tokens = num_tokens, w.max_query_len = max_query_len;
  w.block_tables = block_tables, w.max_blocks = max_blocks_per_seq, w.context_lens = context_lens;
  w.num_seqs = num_seqs, w.cache = cache, w.desc = desc;
  int rc = check_write_q8(w, "paged_kv_write_q8");
  if (!rc) rc = launch_write_q8(w, static_cast<cudaStream_t>(stream));
  if (!rc) clear_error();
  return rc;
}

PKV_API int paged_kv_write_rope_q8(const pkv_bf16 *k, const pkv_bf16 *v, int64_t k_stride, int64_t v_stride,
                                   const pkv_bf16 *q, pkv_bf16 *q_out, int64_t q_stride, int64_t q_out_stride,
                                   int32_t num_q_heads, const int64_t *positions, const float *cos_sin,
                                   int64_t max_position, int32_t rotary_dim, int32_t neox_style,
                                   const int32_t *query_start, int64_t num_tokens, int32_t max_query_len,
                                   const int32_t *block_tables, int32_t max_blocks_per_seq,
                                   const int32_t *context_lens, int32_t num_seqs, const pkv_q8_cache *cache,
                                   const pkv_cache_desc *desc, void *stream) {
  WriteQ8 w = {};
  w.k = k, w.v = v, w.k_stride = k_stride, w.v_stride = v_stride;
  w.query_start = query_start, w.num_tokens = num_tokens, w.max_query_len = max_query_len;
  w.block_tables = block_tables, w.max_blocks = max_blocks_per_seq, w.context_lens = context_lens;
  w.num_seqs = num_seqs, w.cache = cache, w.desc = desc;
  w.rope = true;
  w.q = q, w.q_out = q_out, w.q_stride = q_stride, w.q_out_stride = q_out_stride, w.num_q_heads = num_q_heads;
  w.positions = positions, w.cos_sin = cos_sin, w.max_position = max_position;
  w.rotary_dim = rotary_dim, w.neox_style = neox_style;
  int rc = check_write_q8(w, "paged_kv_write_rope_q8");
  if (!rc) rc = launch_write_q8(w, static_cast<cudaStream_t>(stream));
  if (!rc) clear_error();
  return rc;
}

PKV_API int paged_kv_read_q8(pkv_bf16 *k_out, pkv_bf16 *v_out, int64_t k_stride, int64_t v_stride,
                             const int32_t *query_start, int64_t num_tokens, int32_t max_query_len,
                             const int32_t *block_tables, int32_t max_blocks_per_seq,
                             const int32_t *context_lens, int32_t num_seqs, const pkv_q8_cache *cache,
                             const pkv_cache_desc *desc, void *stream) {
  int rc = check_span(k_out, v_out, k_stride, v_stride, query_start, num_tokens, max_query_len, block_tables,
                      max_blocks_per_seq, context_lens, num_seqs, cache, desc, "paged_kv_read_q8");
  if (!rc && num_seqs > 0 && num_tokens > 0 && max_query_len > 0) {
    const Span s = span_of(block_tables, max_blocks_per_seq, context_lens, query_start, max_query_len, num_seqs,
                           num_tokens, *desc);
    rc = launch_read(s, *cache, *desc, k_out, v_out, k_stride, v_stride, 0, nullptr, nullptr,
                     std::min<int64_t>(touched(max_query_len, desc->block_size), max_blocks_per_seq),
                     static_cast<cudaStream_t>(stream));
  }
  if (!rc) clear_error();
  return rc;
}

// ---------------------------------------------------------------------------
// Chunked prefill.  A few queries per sequence (draft tokens to check) are rows of the decode kernel, up
// to 16 of a kv head for each pass over the codes as they are; more of them take the tensor-core
// tiles of the packed prompts: the contexts are read back into fp16 rows in the workspace, and the tensor-core
// tiles of the packed prompts run over those.  (Widening the codes where the tiles stage them would
// be done once for every 256 query rows that see them, on the warps that the softmax waits for; the
// reading back costs 5 bytes of traffic a code once.)

namespace {

struct PrefillLayout {
  int32_t rows;  // packed rows of a sequence
  size_t k, v, k_unit, v_unit, nan_from, order, total;
};
constexpr int kMaxListed = 32, kMaxEntries = 65535;  // queries of a sequence, entries of a call's list

// Whether the queries fit a list for the decode kernel.
bool list_fits(int32_t max_query_len, int32_t num_seqs, int32_t group, int32_t d) {
  return max_query_len <= kMaxListed && (int64_t)num_seqs * list_plan(group, d, max_query_len).per <= kMaxEntries;
}

// Whether such a list is the shorter way, by the longest context: it reads that once for each entry, spread
// over the GPU; the tiles read it once (and once more back), but the CTAs of one (sequence, kv head) take
// its blocks of 128 keys one after another.  Times as measured: list_plan's, 10 us besides; 1.3 us of a
// tile's block, 6 TB/s for the reading back, 12 us besides.  With 8 kv heads of 4 x 64: 8 sequences of 2
// queries over 4000 tokens 16 us by a list, 67 by tiles, of 8 queries 28 and 67, of 32 75 and 68; 64 of 8
// 143 and 291, of 16 276 and 291, of 32 539 and 292.
bool list_pays(int64_t num_queries, int32_t max_query_len, int32_t num_seqs, int32_t hq, int32_t hkv, int32_t d,
               int32_t max_len, int sms) {
  const int32_t group = hq / hkv;
  const ListPlan plan = list_plan(group, d, max_query_len);
  const double blocks = (max_len - 1) / 128 + 1, heads = hkv;
  const double list = (double)num_seqs * plan.per * heads * (blocks + 1) / sms * plan.block + 10;  // (an end as a block)
  const double ctas = (num_queries / (2. * (128 / group)) + num_seqs) * heads;
  const double tiles = (ctas > sms ? ctas / sms : 1) * blocks * 1.3 + 12 + num_seqs * heads * d * max_len * 6. / 6e6;
  return list < tiles;
}

size_t up(size_t x) { return (x + 255) & ~size_t(255); }

// The tiles' workspace; false: more rows than they count.
bool prefill_layout(int32_t num_seqs, int32_t hkv, int32_t d, int32_t max_len, PrefillLayout *p) {
  if ((int64_t)max_len * num_seqs > 0x7fffff00LL / hkv) return false;
  p->rows = max_len;
  const size_t rows = up((size_t)max_len * num_seqs * hkv * d * 2), units = up((size_t)num_seqs * hkv * 4);
  p->k = 0;
  p->v = rows;
  p->k_unit = 2 * rows;
  p->v_unit = p->k_unit + units;
  p->nan_from = p->v_unit + units;
  p->order = p->nan_from + units;
  p->total = p->order + up((size_t)num_seqs * sizeof(int4));
  return true;
}
// The list's, however many queries a sequence has.
size_t list_bytes(int32_t num_seqs, int32_t d, int sms) {
  return up(list_q8_workspace(std::min((int64_t)num_seqs * kMaxListPer, (int64_t)kMaxEntries), d, sms));
}

// The tiles take the sequences in groups, as many at a time as the workspace has rows for.  How many, evenly
// (0: none), and a group's layout.
int32_t seqs_at_once(int32_t num_seqs, int32_t hkv, int32_t d, int32_t max_len, size_t bytes, PrefillLayout *p) {
  const size_t one = (size_t)max_len * hkv * d * 4;
  int32_t n = (int32_t)std::min<size_t>({(size_t)num_seqs, bytes / one, 0x7fffff00ull / hkv / max_len});
  while (n > 0 && !(prefill_layout(n, hkv, d, max_len, p) && p->total <= bytes)) --n;  // (the rest is small)
  if (n == 0) return 0;
  const int32_t groups = (num_seqs + n - 1) / n;
  n = (num_seqs + groups - 1) / groups;
  prefill_layout(n, hkv, d, max_len, p);
  return n;
}
// So much is asked for at most, where one context's rows are not more: 3 % of the GPU's memory.  (Groups cost
// launches that do not fill the GPU: 64 chunks of 40 to 200, one over 32768 tokens and the others over up to 4000,
// take 0.66 ms at once, in 8.6 GB, and 1.16 in 0.9; 16 of 512 over 32768 each 2.97 in 2.1 GB and 3.50 in 0.8.)
constexpr size_t kRowsPlenty = size_t(1) << 33;

// The way that a call takes; the workspace that it is best given, 0 bytes where no way can be.
struct PrefillWay {
  bool list;
  size_t bytes;
};
PrefillWay prefill_way(int64_t num_queries, int32_t max_query_len, int32_t num_seqs, int32_t hq, int32_t hkv, int32_t d,
                       int32_t max_len, int sms) {
  PrefillWay w = {};
  PrefillLayout p;
  const bool rows = prefill_layout(1, hkv, d, max_len, &p);
  w.list = list_fits(max_query_len, num_seqs, hq / hkv, d) &&
           (!rows || list_pays(num_queries, max_query_len, num_seqs, hq, hkv, d, max_len, sms));
  if (w.list)
    w.bytes = list_bytes(num_seqs, d, sms);
  else if (rows && seqs_at_once(num_seqs, hkv, d, max_len, std::max(kRowsPlenty, p.total), &p) > 0)
    w.bytes = p.total;
  return w;
}

// The current device's SMs; without a device (the checks that need none still stand) `otherwise`.
int sms_or(int otherwise) {
  std::lock_guard<std::mutex> lk(attn_mutex());
  int sms = 0;
  return device_sms(&sms) == PKV_OK && sms > 0 ? sms : otherwise;
}

}  // namespace

PKV_API size_t paged_prefill_q8_workspace_size(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim,
                                               int32_t max_context_len) {
  PrefillLayout p;
  if (num_seqs <= 0 || num_kv_heads <= 0 || max_context_len <= 0 || (head_dim != 64 && head_dim != 128) ||
      !prefill_layout(num_seqs, num_kv_heads, head_dim, max_context_len, &p))
    return 0;
  return std::max(p.total, list_bytes(num_seqs, head_dim, sms_or(152)));
}

PKV_API size_t paged_prefill_q8_workspace_size_for(int64_t num_queries, int32_t max_query_len, int32_t num_seqs,
                                                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                                   int32_t max_context_len) {
  if (num_queries <= 0 || max_query_len <= 0 || num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > kMaxGroup || (head_dim != 64 && head_dim != 128) ||
      max_context_len < max_query_len)
    return 0;
  return prefill_way(num_queries, max_query_len, num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                     sms_or(152)).bytes;
}

PKV_API int paged_prefill_attention_q8(pkv_bf16 *out, const pkv_bf16 *q, int64_t num_queries,
                                       const pkv_q8_cache *cache, const int32_t *block_tables,
                                       int32_t max_blocks_per_seq, const int32_t *context_lens,
                                       int32_t max_context_len, const int32_t *query_start, int32_t max_query_len,
                                       int32_t num_seqs, int32_t num_q_heads, const pkv_cache_desc *desc, float scale,
                                       void *workspace, size_t workspace_bytes, void *stream) {
  const char *const fn = "paged_prefill_attention_q8";
  int rc = check_q8(cache, desc, num_seqs, fn);
  if (!rc)
    rc = check_decode(q, cache->k_cache, cache->v_cache, block_tables, max_blocks_per_seq, context_lens,
                      max_context_len, num_queries > 0 ? num_seqs : 0, num_q_heads, desc, fn);
  if (rc) return rc;
  if (num_queries < 0 || max_query_len < 0 || max_query_len > max_context_len)
    return set_error(PKV_ERR_SHAPE, "%s: need num_queries >= 0, 0 <= max_query_len <= max_context_len", fn);
  if (num_seqs == 0 || max_query_len == 0 || num_queries == 0) {
    clear_error();
    return PKV_OK;
  }
  if (!out || !query_start) return set_error(PKV_ERR_NULL, "%s: NULL out/query_start", fn);
  if (num_queries > 0x7fffff00LL) return set_error(PKV_ERR_UNSUPPORTED, "%s: num_queries over 2^31", fn);
  if (!aligned16(out)) return set_error(PKV_ERR_ALIGN, "%s: out must be 16-byte aligned", fn);
  if (misaligned4(query_start) || misaligned4(block_tables) || misaligned4(context_lens))
    return set_error(PKV_ERR_ALIGN, "%s: int32 tensors must be 4-byte aligned", fn);
  const int sms = sms_or(152);
  const PrefillWay way = prefill_way(num_queries, max_query_len, num_seqs, num_q_heads, desc->num_kv_heads, desc->head_dim,
                                     max_context_len, sms);
  if (way.bytes == 0)
    return set_error(PKV_ERR_UNSUPPORTED, "%s: a context has more than 2^31 rows of heads", fn);
  PrefillLayout p;
  int32_t at_once = num_seqs;
  size_t least = way.bytes;
  if (!way.list) {
    prefill_layout(1, desc->num_kv_heads, desc->head_dim, max_context_len, &p);
    least = p.total;
    at_once = seqs_at_once(num_seqs, desc->num_kv_heads, desc->head_dim, max_context_len, workspace_bytes, &p);
  }
  if (!workspace || workspace_bytes < least || at_once == 0)
    return set_error(PKV_ERR_WORKSPACE, "%s: workspace %zu bytes < %zu needed", fn, workspace_bytes, least);
  if (!aligned16(workspace)) return set_error(PKV_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char *const ws = static_cast<char *>(workspace);
  ChunkLaunch l = {};
  l.out = out;
  l.q = q;
  l.query_start = query_start;
  l.context_lens = context_lens;
  l.num_queries = num_queries;
  l.max_query_len = max_query_len;
  l.max_context = (int32_t)std::min<int64_t>((int64_t)max_blocks_per_seq * desc->block_size, max_context_len);
  l.num_seqs = num_seqs;
  l.num_q_heads = num_q_heads;
  l.num_kv_heads = desc->num_kv_heads;
  l.head_dim = desc->head_dim;
  l.scale = scale;
  if (way.list) {
    rc = launch_list_q8(l, *cache, *desc, block_tables, max_blocks_per_seq, workspace, sms, s);
    if (!rc) clear_error();
    return rc;
  }
  const int64_t stride = (int64_t)desc->num_kv_heads * desc->head_dim;
  for (int32_t b0 = 0; !rc && b0 < num_seqs; b0 += at_once) {
    const int32_t n = std::min(at_once, num_seqs - b0);
    const Span span = span_of(block_tables + (int64_t)b0 * max_blocks_per_seq, max_blocks_per_seq, context_lens + b0,
                              query_start + b0, max_context_len, n, 0, *desc);
    UnitArgs u;
    u.s = span;
    u.k_scale = cache->k_scale;
    u.v_scale = cache->v_scale;
    u.k_unit = reinterpret_cast<float *>(ws + p.k_unit);
    u.v_unit = reinterpret_cast<float *>(ws + p.v_unit);
    u.nan_from = reinterpret_cast<int32_t *>(ws + p.nan_from);
    u.order = reinterpret_cast<int4 *>(ws + p.order);
    u.num_queries = (int32_t)num_queries;
    u.max_query_len = max_query_len;
    u.ahead = b0;
    const cudaError_t e = q8::launch_early(units_q8_kernel, dim3((unsigned)n), kUnitThreads, 0, s, u);
    if (e != cudaSuccess) return cuda_error(e, "units_q8_kernel launch");
    rc = launch_read(span, *cache, *desc, ws + p.k, ws + p.v, stride, stride, p.rows, u.k_unit, u.v_unit,
                     ((int64_t)max_context_len + desc->block_size - 1) / desc->block_size, s);
    if (rc) return rc;
    l.query_start = span.start;
    l.context_lens = span.lens;
    l.num_seqs = n;
    l.kv_rows = p.rows;
    l.k = reinterpret_cast<const uint16_t *>(ws + p.k);
    l.v = reinterpret_cast<const uint16_t *>(ws + p.v);
    l.k_unit = u.k_unit;
    l.v_unit = u.v_unit;
    l.nan_from = u.nan_from;
    l.order = u.order;
    rc = launch_chunk(l, s);
  }
  if (!rc) clear_error();
  return rc;
}
