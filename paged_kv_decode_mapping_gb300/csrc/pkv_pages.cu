// pkv_pages.cu -- whole-page operations on the paged cache: pages copied to other pages
// (the copy-on-write of forked sequences), and compaction (pages moved into free pages,
// block tables rewritten), for every layer's caches in one launch.
//
// A page is one contiguous run of num_kv_heads * block_size * head_dim elements.  There is
// no arithmetic: each byte is read once and written once, so a launch is bound by HBM
// (2 bytes of traffic per byte copied), and the small ones by the launch itself.  16 KB of a
// page per CTA, four 16-byte loads in flight per thread before the first store.  Measured: 256
// pages of 28 layers (939 MB) 128 us, 7.3 TB/s; 2900 pages of 4 layers (381 MB) 58 us, 6.6
// TB/s; 5 pages of 16 layers 2.6 us.  Pages of 8 KB and over; smaller ones, a CTA each with less
// than a vector per thread and load, were not timed.
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_device.cuh"

namespace pkv {

constexpr int kPageLayers = 64;   // layers whose pointers one launch carries
constexpr int kPageThreads = 256;
constexpr int kPageUnroll = 4;    // 16-byte vectors a thread keeps in flight

struct PageArgs {
  uint4 *k[kPageLayers], *v[kPageLayers];
  const int2 *pairs;        // (source, destination)
  const int32_t *rows;      // tokens to copy per pair, or NULL: whole pages
  int64_t num_blocks;
  uint32_t page_vecs;       // 16-byte vectors of a page
  uint32_t head_vecs;       // ... of one kv head's block_size rows
  uint32_t row_vecs;        // ... of one row
  uint32_t block_size;
  uint32_t chunks;          // CTAs per page
  int32_t planes;           // 2 * layers: plane 2l is layer l's K, 2l + 1 its V
  int32_t *tables;          // compaction: entries to rewrite (from plane `planes` on), or NULL
  int64_t entries;
  const int32_t *block_map;
};

// Grid: x = (pair, chunk of its page), chunk fastest; y = plane.  With `tables`, the rows of CTAs
// past the planes rewrite the block-table entries, grid-stride: as many rows as the entries
// need (in one row, a single moved page of one chunk left the whole table to one CTA: tables of
// 256 x 512 took 115 us, now 1.8; of 64 x 8192 455, now 2.7).
__global__ void __launch_bounds__(kPageThreads) copy_pages_kernel(const __grid_constant__ PageArgs a) {
  const int tid = threadIdx.x, plane = blockIdx.y;
  if (plane >= a.planes) {
    const int64_t cta = (int64_t)(plane - a.planes) * gridDim.x + blockIdx.x;
    const int64_t ctas = (int64_t)(gridDim.y - a.planes) * gridDim.x;
    for (int64_t i = cta * kPageThreads + tid; i < a.entries; i += ctas * kPageThreads) {
      const int32_t x = a.tables[i];
      if (x < 0) continue;  // unused entry
      int32_t y = -1;
      if (x < a.num_blocks) y = __ldg(a.block_map + x);
      if (y < 0 || y >= a.num_blocks) {
        raise_error(PKV_DEVERR_BLOCK_ID);
        continue;
      }
      if (y != x) a.tables[i] = y;
    }
    return;
  }
  const uint32_t pair = blockIdx.x / a.chunks, chunk = blockIdx.x - pair * a.chunks;
  const int2 p = __ldg(a.pairs + pair);
  if (p.x < 0 || p.x >= a.num_blocks || p.y < 0 || p.y >= a.num_blocks) {
    if (tid == 0) raise_error(PKV_DEVERR_BLOCK_ID);
    return;
  }
  if (p.x == p.y) return;
  uint32_t limit = a.head_vecs;  // vectors of each head's rows to copy
  if (a.rows) {
    int32_t r = __ldg(a.rows + pair);
    if (r < 0 || r > (int32_t)a.block_size) {
      if (tid == 0) raise_error(PKV_DEVERR_CONTEXT_LEN);
      r = r < 0 ? 0 : (int32_t)a.block_size;
    }
    limit = (uint32_t)r * a.row_vecs;
  }
  uint4 *const pool = (plane & 1) ? a.v[plane >> 1] : a.k[plane >> 1];
  const uint4 *const src = pool + (int64_t)p.x * a.page_vecs;
  uint4 *const dst = pool + (int64_t)p.y * a.page_vecs;
  const uint32_t i0 = chunk * (kPageThreads * kPageUnroll) + tid;
  uint4 x[kPageUnroll];
  bool take[kPageUnroll];
#pragma unroll
  for (int u = 0; u < kPageUnroll; ++u) {
    const uint32_t i = i0 + u * kPageThreads;
    take[u] = i < a.page_vecs && (limit == a.head_vecs || i % a.head_vecs < limit);
    if (take[u]) x[u] = __ldcs(src + i);
  }
#pragma unroll
  for (int u = 0; u < kPageUnroll; ++u)
    if (take[u]) __stcs(dst + i0 + u * kPageThreads, x[u]);
}

// The 8-bit cache's scales of the copied pages: plane 2l is layer l's K, 2l + 1 its V.  A pair of which
// no row is copied leaves its destination's scales too.
struct ScaleArgs {
  float *k[kPageLayers], *v[kPageLayers];
  const int2 *pairs;
  const int32_t *rows;
  int64_t num_blocks, num_pairs;
  uint32_t heads;
};
__global__ void __launch_bounds__(kPageThreads) copy_scales_kernel(const __grid_constant__ ScaleArgs a) {
  const int plane = blockIdx.y;
  const int64_t i = (int64_t)blockIdx.x * kPageThreads + threadIdx.x;
  const int64_t pair = i / a.heads;
  if (pair >= a.num_pairs) return;
  const int2 p = __ldg(a.pairs + pair);
  // (flagged by the rows' copy)
  if (p.x < 0 || p.x >= a.num_blocks || p.y < 0 || p.y >= a.num_blocks || p.x == p.y) return;
  if (a.rows && __ldg(a.rows + pair) <= 0) return;
  float *const pool = (plane & 1) ? a.v[plane >> 1] : a.k[plane >> 1];
  const uint32_t h = (uint32_t)(i - pair * a.heads);
  pool[(int64_t)p.y * a.heads + h] = pool[(int64_t)p.x * a.heads + h];
}

cudaError_t read_page_errors(uint32_t *flags, int clear) { return read_tu_errors(flags, clear); }

namespace {

int check_pages(pkv_bf16 *const *k_caches, pkv_bf16 *const *v_caches, int32_t num_layers,
                const int32_t *pairs, int64_t num_pairs, const pkv_cache_desc *c, const char *fn) {
  if (!c) return set_error(PKV_ERR_NULL, "%s: cache descriptor is NULL", fn);
  if (num_layers < 0 || num_pairs < 0) return set_error(PKV_ERR_SHAPE, "%s: negative count", fn);
  if (c->num_blocks <= 0 || c->block_size <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0)
    return set_error(PKV_ERR_SHAPE, "%s: cache sizes must be positive", fn);
  if (c->num_blocks > 0x7fffffffLL)
    return set_error(PKV_ERR_UNSUPPORTED, "%s: more than 2^31-1 blocks", fn);
  if (c->head_dim % 8 != 0)
    return set_error(PKV_ERR_UNSUPPORTED, "%s: head_dim %d is not a multiple of 8", fn, c->head_dim);
  const int64_t half = (int64_t)c->num_kv_heads * c->block_size;
  if (half > (1LL << 40) / c->head_dim || half * c->head_dim / 8 > (1 << 28))
    return set_error(PKV_ERR_UNSUPPORTED, "%s: a page has more than 4 GB", fn);
  if (num_layers == 0) return PKV_OK;
  if (!k_caches || !v_caches) return set_error(PKV_ERR_NULL, "%s: NULL cache array", fn);
  for (int32_t l = 0; l < num_layers; ++l) {
    if (!k_caches[l] || !v_caches[l]) return set_error(PKV_ERR_NULL, "%s: NULL cache of layer %d", fn, l);
    if (!aligned16(k_caches[l]) || !aligned16(v_caches[l]))
      return set_error(PKV_ERR_ALIGN, "%s: the caches must be 16-byte aligned", fn);
  }
  if (num_pairs > 0 && !pairs) return set_error(PKV_ERR_NULL, "%s: NULL block pairs", fn);
  if (num_pairs > 0 && (reinterpret_cast<uintptr_t>(pairs) & 7u))
    return set_error(PKV_ERR_ALIGN, "%s: the block pairs must be 8-byte aligned", fn);
  const int64_t vecs = half * (c->head_dim / 8);
  const int64_t chunks = (vecs + kPageThreads * kPageUnroll - 1) / (kPageThreads * kPageUnroll);
  if (num_pairs > 0x7fffffffLL / chunks) return set_error(PKV_ERR_UNSUPPORTED, "%s: too many pairs", fn);
  return PKV_OK;
}

int launch_pages(pkv_bf16 *const *k_caches, pkv_bf16 *const *v_caches, int32_t num_layers,
                 const int32_t *pairs, const int32_t *rows, int64_t num_pairs, int32_t *tables,
                 int64_t entries, const int32_t *block_map, const pkv_cache_desc &c,
                 cudaStream_t stream) {
  PageArgs a = {};
  a.pairs = reinterpret_cast<const int2 *>(pairs);
  a.rows = rows;
  a.num_blocks = c.num_blocks;
  a.row_vecs = (uint32_t)(c.head_dim / 8);
  a.head_vecs = a.row_vecs * (uint32_t)c.block_size;
  a.page_vecs = a.head_vecs * (uint32_t)c.num_kv_heads;
  a.block_size = (uint32_t)c.block_size;
  a.chunks = (a.page_vecs + kPageThreads * kPageUnroll - 1) / (kPageThreads * kPageUnroll);
  if (num_pairs == 0) num_layers = 0;  // tables only
  int32_t l0 = 0;
  do {
    const int32_t n = std::min(num_layers - l0, (int32_t)kPageLayers);
    for (int32_t l = 0; l < n; ++l) {
      a.k[l] = reinterpret_cast<uint4 *>(k_caches[l0 + l]);
      a.v[l] = reinterpret_cast<uint4 *>(v_caches[l0 + l]);
    }
    a.planes = 2 * n;
    const bool remap = l0 == 0 && entries > 0;
    a.tables = remap ? tables : nullptr;
    a.entries = remap ? entries : 0;
    a.block_map = block_map;
    const int64_t table_ctas = remap ? std::min<int64_t>((entries + kPageThreads - 1) / kPageThreads, 4096) : 0;
    int64_t x = num_layers > 0 ? num_pairs * a.chunks : 0;
    if (x == 0) x = table_ctas;
    const unsigned y = (unsigned)(a.planes + (remap ? (table_ctas + x - 1) / x : 0));
    if (y > 0) {
      copy_pages_kernel<<<dim3((unsigned)x, y, 1), kPageThreads, 0, stream>>>(a);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return cuda_error(e, "copy_pages_kernel launch");
    }
    l0 += n;
  } while (l0 < num_layers);
  return PKV_OK;
}

// The layers' 8-bit caches checked; the rows as ones of head_dim / 2 16-bit elements.
int check_q8_pages(const pkv_q8_cache *caches, int32_t num_layers, const pkv_cache_desc *c, const char *fn) {
  if (!c || (num_layers > 0 && !caches)) return set_error(PKV_ERR_NULL, "%s: NULL caches or descriptor", fn);
  if (num_layers < 0) return set_error(PKV_ERR_SHAPE, "%s: negative count", fn);
  int rc = check_q8_sizes(c, fn);  // (of no layers too: tables alone)
  for (int32_t l = 0; !rc && l < num_layers; ++l) rc = check_q8(caches + l, c, 1, fn);
  return rc;
}

int copy_q8_pages(const pkv_q8_cache *caches, int32_t num_layers, const int32_t *pairs, const int32_t *rows,
                  int64_t num_pairs, int32_t *tables, int64_t entries, const int32_t *block_map,
                  const pkv_cache_desc &c, cudaStream_t stream) {
  pkv_cache_desc half = c;
  half.head_dim = c.head_dim / 2;
  int32_t l0 = 0;
  do {
    const int32_t n = std::min(num_layers - l0, (int32_t)kPageLayers);
    pkv_bf16 *k[kPageLayers], *v[kPageLayers];
    ScaleArgs a = {};
    for (int32_t l = 0; l < n; ++l) {
      const pkv_q8_cache &q = caches[l0 + l];
      k[l] = static_cast<pkv_bf16 *>(q.k_cache);
      v[l] = static_cast<pkv_bf16 *>(q.v_cache);
      a.k[l] = q.k_scale;
      a.v[l] = q.v_scale;
    }
    const bool remap = l0 == 0;
    const int rc = launch_pages(k, v, n, pairs, rows, num_pairs, remap ? tables : nullptr, remap ? entries : 0,
                                block_map, half, stream);
    if (rc) return rc;
    if (n > 0 && num_pairs > 0) {
      a.pairs = reinterpret_cast<const int2 *>(pairs);
      a.rows = rows;
      a.num_blocks = c.num_blocks;
      a.num_pairs = num_pairs;
      a.heads = (uint32_t)c.num_kv_heads;
      const int64_t ctas = (num_pairs * c.num_kv_heads + kPageThreads - 1) / kPageThreads;
      copy_scales_kernel<<<dim3((unsigned)ctas, (unsigned)(2 * n)), kPageThreads, 0, stream>>>(a);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return cuda_error(e, "copy_scales_kernel launch");
    }
    l0 += n;
  } while (l0 < num_layers);
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

PKV_API int paged_kv_copy_blocks(pkv_bf16 *const *k_caches, pkv_bf16 *const *v_caches,
                                 int32_t num_layers, const int32_t *block_pairs,
                                 const int32_t *num_tokens, int64_t num_pairs,
                                 const pkv_cache_desc *cache, void *stream) {
  int rc = check_pages(k_caches, v_caches, num_layers, block_pairs, num_pairs, cache,
                       "paged_kv_copy_blocks");
  if (!rc && num_tokens && (reinterpret_cast<uintptr_t>(num_tokens) & 3u))
    rc = set_error(PKV_ERR_ALIGN, "paged_kv_copy_blocks: num_tokens must be 4-byte aligned");
  if (!rc && num_pairs > 0 && num_layers > 0)
    rc = launch_pages(k_caches, v_caches, num_layers, block_pairs, num_tokens, num_pairs, nullptr, 0,
                      nullptr, *cache, static_cast<cudaStream_t>(stream));
  if (!rc) clear_error();
  return rc;
}

PKV_API int paged_kv_compact(pkv_bf16 *const *k_caches, pkv_bf16 *const *v_caches,
                             int32_t num_layers, const int32_t *block_moves, int64_t num_moves,
                             int32_t *block_tables, int64_t num_seqs, int32_t max_blocks_per_seq,
                             const int32_t *block_map, const pkv_cache_desc *cache, void *stream) {
  const char *const fn = "paged_kv_compact";
  int rc = check_pages(k_caches, v_caches, num_layers, block_moves, num_moves, cache, fn);
  if (rc) return rc;
  if (num_seqs < 0 || max_blocks_per_seq < 0)
    return set_error(PKV_ERR_SHAPE, "%s: negative block table size", fn);
  if (num_seqs > 0 && max_blocks_per_seq > 0) {
    if (num_seqs > 0x7fffffffLL) return set_error(PKV_ERR_UNSUPPORTED, "%s: num_seqs > 2^31-1", fn);
    if (!block_tables || !block_map) return set_error(PKV_ERR_NULL, "%s: NULL block_tables/block_map", fn);
    if ((reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(block_map) & 3u))
      return set_error(PKV_ERR_ALIGN, "%s: block_tables and block_map must be 4-byte aligned", fn);
  }
  const int64_t entries = num_seqs * max_blocks_per_seq;
  if ((num_moves > 0 && num_layers > 0) || entries > 0)
    rc = launch_pages(k_caches, v_caches, num_layers, block_moves, nullptr, num_moves, block_tables,
                      entries, block_map, *cache, static_cast<cudaStream_t>(stream));
  if (!rc) clear_error();
  return rc;
}

PKV_API int paged_kv_copy_blocks_q8(const pkv_q8_cache *caches, int32_t num_layers, const int32_t *block_pairs,
                                    const int32_t *num_tokens, int64_t num_pairs, const pkv_cache_desc *desc,
                                    void *stream) {
  return paged_kv_compact_q8(caches, num_layers, block_pairs, num_tokens, num_pairs, nullptr, 0, 0, nullptr, desc,
                             stream);
}

PKV_API int paged_kv_compact_q8(const pkv_q8_cache *caches, int32_t num_layers, const int32_t *block_moves,
                                const int32_t *num_tokens, int64_t num_moves, int32_t *block_tables,
                                int64_t num_seqs, int32_t max_blocks_per_seq, const int32_t *block_map,
                                const pkv_cache_desc *desc, void *stream) {
  const char *const fn = "paged_kv_copy_blocks_q8/compact_q8";
  int rc = check_q8_pages(caches, num_layers, desc, fn);
  if (rc) return rc;
  if (num_moves < 0 || num_seqs < 0 || max_blocks_per_seq < 0) return set_error(PKV_ERR_SHAPE, "%s: negative count", fn);
  if (num_moves > 0 && !block_moves) return set_error(PKV_ERR_NULL, "%s: NULL block pairs", fn);
  if ((reinterpret_cast<uintptr_t>(block_moves) & 7u) || (reinterpret_cast<uintptr_t>(num_tokens) & 3u) ||
      (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(block_map) & 3u))
    return set_error(PKV_ERR_ALIGN, "%s: block pairs must be 8-byte, other int32 arrays 4-byte aligned", fn);
  if (num_moves > 0x3fffffffLL / desc->num_kv_heads / desc->block_size)
    return set_error(PKV_ERR_UNSUPPORTED, "%s: too many pairs", fn);
  const int64_t entries = num_seqs > 0x7fffffffLL ? -1 : num_seqs * max_blocks_per_seq;
  if (entries < 0) return set_error(PKV_ERR_UNSUPPORTED, "%s: num_seqs > 2^31-1", fn);
  if (entries > 0 && (!block_tables || !block_map))
    return set_error(PKV_ERR_NULL, "%s: NULL block_tables/block_map", fn);
  if ((num_moves > 0 && num_layers > 0) || entries > 0)
    rc = copy_q8_pages(caches, num_layers, block_moves, num_tokens, num_moves, block_tables, entries, block_map, *desc,
                       static_cast<cudaStream_t>(stream));
  if (!rc) clear_error();
  return rc;
}
