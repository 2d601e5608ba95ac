// pkv_q8_call.cpp -- the 8-bit cache's calls with their arguments as 64-bit words.  A foreign-function
// interface converts each argument of a call by itself (ctypes: 14 of them 1 us of a call's 9); words are
// packed at once.
#include "pkv_internal.h"

#include <cstring>

namespace {

struct Words {
  const int64_t *p;
  template <typename T>
  T *pointer() { return reinterpret_cast<T *>(static_cast<uintptr_t>(*p++)); }
  int64_t wide() { return *p++; }
  int32_t count() {  // a value that does not fit is refused as one that is negative
    const int64_t x = *p++;
    return x < -1 || x > 0x7fffffff ? -1 : (int32_t)x;
  }
  float real() {
    double x;
    std::memcpy(&x, p++, sizeof x);
    return (float)x;
  }
};

}  // namespace

PKV_API int pkv_call_q8(int32_t call, const int64_t *words) {
  if (!words) return pkv::set_error(PKV_ERR_NULL, "pkv_call_q8: NULL words");
  Words w = {words};
  pkv_q8_cache cache;
  cache.k_cache = w.pointer<void>();
  cache.v_cache = w.pointer<void>();
  cache.k_scale = w.pointer<float>();
  cache.v_scale = w.pointer<float>();
  cache.kind = w.count();
  pkv_cache_desc d;
  d.num_blocks = w.wide();
  d.block_size = w.count();
  d.num_kv_heads = w.count();
  d.head_dim = w.count();
  const int32_t *const tables = w.pointer<const int32_t>();
  const int32_t max_blocks = w.count();
  const int32_t *const lens = w.pointer<const int32_t>();
  const int32_t num_seqs = w.count();
  void *const stream = w.pointer<void>();
  if (call == PKV_CALL_WRITE_Q8 || call == PKV_CALL_READ_Q8 || call == PKV_CALL_WRITE_ROPE_Q8) {
    pkv_bf16 *const k = w.pointer<pkv_bf16>(), *const v = w.pointer<pkv_bf16>();
    const int64_t k_stride = w.wide(), v_stride = w.wide();
    const int32_t *const start = w.pointer<const int32_t>();
    const int64_t num_tokens = w.wide();
    const int32_t max_query_len = w.count();
    if (call == PKV_CALL_WRITE_Q8)
      return paged_kv_write_q8(k, v, k_stride, v_stride, start, num_tokens, max_query_len, tables, max_blocks, lens,
                               num_seqs, &cache, &d, stream);
    if (call == PKV_CALL_READ_Q8)
      return paged_kv_read_q8(k, v, k_stride, v_stride, start, num_tokens, max_query_len, tables, max_blocks, lens,
                              num_seqs, &cache, &d, stream);
    const pkv_bf16 *const q = w.pointer<const pkv_bf16>();
    pkv_bf16 *const q_out = w.pointer<pkv_bf16>();
    const int64_t q_stride = w.wide(), q_out_stride = w.wide();
    const int32_t num_q_heads = w.count();
    const int64_t *const positions = w.pointer<const int64_t>();
    const float *const cos_sin = w.pointer<const float>();
    const int64_t max_position = w.wide();
    const int32_t rotary_dim = w.count(), neox_style = w.count();
    return paged_kv_write_rope_q8(k, v, k_stride, v_stride, q, q_out, q_stride, q_out_stride, num_q_heads, positions,
                                  cos_sin, max_position, rotary_dim, neox_style, start, num_tokens, max_query_len,
                                  tables, max_blocks, lens, num_seqs, &cache, &d, stream);
  }
  if (call == PKV_CALL_DECODE_Q8 || call == PKV_CALL_PREFILL_Q8 || call == PKV_CALL_STEP_Q8 ||
      call == PKV_CALL_STEP_ROPE_Q8) {
    pkv_bf16 *const out = w.pointer<pkv_bf16>();
    const pkv_bf16 *const q = w.pointer<const pkv_bf16>();
    const int32_t max_len = w.count(), num_q_heads = w.count();
    const float scale = w.real();
    void *const workspace = w.pointer<void>();
    const size_t bytes = (size_t)w.wide();
    if (call == PKV_CALL_DECODE_Q8)
      return paged_decode_attention_q8(out, q, &cache, tables, max_blocks, lens, max_len, num_seqs, num_q_heads, &d, scale,
                                       workspace, bytes, stream);
    if (call == PKV_CALL_PREFILL_Q8) {
      const int64_t num_queries = w.wide();
      const int32_t *const start = w.pointer<const int32_t>();
      const int32_t max_query_len = w.count();
      return paged_prefill_attention_q8(out, q, num_queries, &cache, tables, max_blocks, lens, max_len, start,
                                        max_query_len, num_seqs, num_q_heads, &d, scale, workspace, bytes, stream);
    }
    const pkv_bf16 *const k = w.pointer<const pkv_bf16>(), *const v = w.pointer<const pkv_bf16>();
    const int64_t k_stride = w.wide(), v_stride = w.wide();
    if (call == PKV_CALL_STEP_Q8)
      return paged_decode_step_q8(out, q, k, v, k_stride, v_stride, &cache, tables, max_blocks, lens, max_len, num_seqs,
                                  num_q_heads, &d, scale, workspace, bytes, stream);
    const int64_t q_stride = w.wide();
    pkv_bf16 *const q_out = w.pointer<pkv_bf16>();
    const int64_t *const positions = w.pointer<const int64_t>();
    const float *const cos_sin = w.pointer<const float>();
    const int64_t max_position = w.wide();
    const int32_t rotary_dim = w.count(), neox_style = w.count();
    return paged_decode_step_rope_q8(out, q, q_stride, q_out, k, v, k_stride, v_stride, positions, cos_sin, max_position,
                                     rotary_dim, neox_style, &cache, tables, max_blocks, lens, max_len, num_seqs,
                                     num_q_heads, &d, scale, workspace, bytes, stream);
  }
  return pkv::set_error(PKV_ERR_UNSUPPORTED, "pkv_call_q8: unknown call %d", call);
}
