// pkv_block_manager.cpp -- host-side KV block allocator: the part of the scheduler that
// produces the block tables and slot mappings the kernels consume.
//
// "mini-vLLM" LLM-Inference-Engine README (architecture diagram and milestone M4): a
// Block Manager allocates physical blocks out of a fixed pool and keeps a block table
// per sequence; under memory pressure the most recently admitted sequence is preempted
// (LIFO).  "vLLM-Style Llama Inference Engine", How it works: the scheduler allocates
// physical KV-cache blocks, and finished requests release their blocks.
//
// Design: a LIFO stack of free block ids (a block freed last is handed out first), a
// hash map from sequence id to {length, blocks}, and the admission order for LIFO
// preemption.  Appending a token to a sequence allocates a new block only when the
// sequence's last block is full.  Forked sequences share blocks: every block counts the
// sequences that hold it, is copied before one of them writes into it (copy-on-write: the
// caller copies the pages), and is free again when the last of them lets go.  All
// operations are O(blocks touched), a compaction O(pool); one mutex makes the manager safe
// to share between threads.  No exception crosses the C boundary.
#include <algorithm>
#include <cstdint>
#include <exception>
#include <mutex>
#include <new>
#include <unordered_map>
#include <vector>

#include "pkv_internal.h"

struct pkv_block_manager {
  struct Seq {
    int64_t len = 0;
    std::vector<int32_t> blocks;
    uint64_t order = 0;  // admission stamp (larger = more recent)
  };
  int64_t num_blocks = 0;
  int32_t block_size = 0;
  std::vector<int32_t> free_stack;  // top = back()
  std::vector<int32_t> refs;        // per block: the sequences that hold it
  std::unordered_map<int64_t, Seq> seqs;
  uint64_t stamp = 0;
  std::mutex mu;

  // Blocks a sequence of `len` tokens occupies.
  int64_t blocks_for(int64_t len) const { return (len + block_size - 1) / block_size; }

  // The free stack holds num_blocks entries from the start, so push_back never allocates.
  int32_t take() {
    const int32_t b = free_stack.back();
    free_stack.pop_back();
    refs[(size_t)b] = 1;
    return b;
  }
  void drop(int32_t b) {
    if (--refs[(size_t)b] == 0) free_stack.push_back(b);
  }
  // Lets go of the sequence's blocks past the first `keep`.
  void release(Seq &s, size_t keep = 0) {
    while (s.blocks.size() > keep) {
      drop(s.blocks.back());
      s.blocks.pop_back();
    }
  }
};

using pkv::set_error;

namespace {

// Runs a call's body; a C++ exception (host memory ran out) becomes an error code.
template <typename F>
int guarded(const char *fn, F body) {
  try {
    return body();
  } catch (const std::exception &e) {
    return set_error(PKV_ERR_NOSPACE, "%s: %s", fn, e.what());
  }
}

}  // namespace

PKV_API pkv_block_manager *pkv_bm_create(int64_t num_blocks, int32_t block_size) {
  if (num_blocks <= 0 || num_blocks > 0x7fffffffLL || block_size <= 0) {
    set_error(PKV_ERR_SHAPE, "pkv_bm_create: need 0 < num_blocks < 2^31 and block_size > 0");
    return nullptr;
  }
  pkv_block_manager *m = new (std::nothrow) pkv_block_manager();
  if (!m) {
    set_error(PKV_ERR_NOSPACE, "pkv_bm_create: out of host memory");
    return nullptr;
  }
  m->num_blocks = num_blocks;
  m->block_size = block_size;
  const int rc = guarded("pkv_bm_create", [&]() -> int {
    m->free_stack.reserve((size_t)num_blocks);
    m->refs.assign((size_t)num_blocks, 0);
    return PKV_OK;
  });
  if (rc) {
    delete m;
    return nullptr;
  }
  for (int64_t b = num_blocks - 1; b >= 0; --b) m->free_stack.push_back((int32_t)b);  // 0 first
  pkv::clear_error();
  return m;
}

PKV_API void pkv_bm_destroy(pkv_block_manager *m) { delete m; }

PKV_API int64_t pkv_bm_num_free_blocks(pkv_block_manager *m) {
  if (!m) return set_error(PKV_ERR_NULL, "pkv_bm_num_free_blocks: NULL manager");
  std::lock_guard<std::mutex> lk(m->mu);
  return (int64_t)m->free_stack.size();
}

PKV_API int pkv_bm_add_sequence(pkv_block_manager *m, int64_t seq_id, int64_t num_tokens) {
  if (!m) return set_error(PKV_ERR_NULL, "pkv_bm_add_sequence: NULL manager");
  if (num_tokens < 0) return set_error(PKV_ERR_SHAPE, "pkv_bm_add_sequence: num_tokens < 0");
  std::lock_guard<std::mutex> lk(m->mu);
  if (m->seqs.count(seq_id))
    return set_error(PKV_ERR_SHAPE, "pkv_bm_add_sequence: sequence %lld already present",
                     (long long)seq_id);
  const int64_t need = m->blocks_for(num_tokens);
  if (need > (int64_t)m->free_stack.size())
    return set_error(PKV_ERR_NOSPACE, "pkv_bm_add_sequence: %lld blocks needed, %zu free",
                     (long long)need, m->free_stack.size());
  return guarded("pkv_bm_add_sequence", [&]() -> int {
    std::vector<int32_t> blocks;
    blocks.reserve((size_t)need);
    pkv_block_manager::Seq &s = m->seqs[seq_id];
    s.blocks.swap(blocks);
    s.len = num_tokens;
    s.order = ++m->stamp;
    for (int64_t i = 0; i < need; ++i) s.blocks.push_back(m->take());
    pkv::clear_error();
    return PKV_OK;
  });
}

PKV_API int pkv_bm_fork(pkv_block_manager *m, int64_t parent_id, int64_t child_id) {
  if (!m) return set_error(PKV_ERR_NULL, "pkv_bm_fork: NULL manager");
  std::lock_guard<std::mutex> lk(m->mu);
  auto parent = m->seqs.find(parent_id);
  if (parent == m->seqs.end())
    return set_error(PKV_ERR_SHAPE, "pkv_bm_fork: unknown sequence %lld", (long long)parent_id);
  if (m->seqs.count(child_id))
    return set_error(PKV_ERR_SHAPE, "pkv_bm_fork: sequence %lld already present",
                     (long long)child_id);
  return guarded("pkv_bm_fork", [&]() -> int {
    pkv_block_manager::Seq s = parent->second;  // copied first: the insertion may rehash
    s.order = ++m->stamp;
    const auto child = m->seqs.emplace(child_id, std::move(s)).first;
    for (int32_t b : child->second.blocks) ++m->refs[(size_t)b];
    pkv::clear_error();
    return PKV_OK;
  });
}

namespace {

// Appends one token to each listed sequence.  With `pairs`, a shared last block that a
// token goes into is replaced by a new one (copy-on-write); without, it is refused.
int append(pkv_block_manager *m, const int64_t *seq_ids, int32_t n, int64_t *slot_mapping,
           int32_t *pairs, int32_t *rows, int32_t *num_pairs, const char *fn) {
  // all-or-nothing: check every sequence and count the new blocks first
  int64_t new_blocks = 0;
  std::unordered_map<int64_t, int64_t> extra;    // appends per sequence in this call
  std::unordered_map<int32_t, int32_t> leaving;  // sequences that let go of a block
  std::vector<pkv_block_manager::Seq *> where((size_t)n);
  for (int32_t i = 0; i < n; ++i) {
    auto it = m->seqs.find(seq_ids[i]);
    if (it == m->seqs.end())
      return set_error(PKV_ERR_SHAPE, "%s: unknown sequence %lld", fn, (long long)seq_ids[i]);
    pkv_block_manager::Seq &s = it->second;
    where[(size_t)i] = &s;
    const int64_t before = extra[seq_ids[i]]++, pos = s.len + before;
    const int64_t lb = pos / m->block_size;
    if (lb >= (int64_t)s.blocks.size()) {
      if (pos % m->block_size == 0) ++new_blocks;
      if ((size_t)lb >= s.blocks.capacity()) s.blocks.reserve(2 * (size_t)lb + 1);
    } else if (before == 0) {
      const int32_t b = s.blocks[(size_t)lb];
      // (a block of this sequence alone makes no entry: one for each took half the call's time)
      if (m->refs[(size_t)b] > 1 && m->refs[(size_t)b] - leaving[b] > 1) {
        if (!pairs)
          return set_error(PKV_ERR_UNSUPPORTED,
                           "%s: sequence %lld shares its last block %d; append with "
                           "pkv_bm_append_slots_cow",
                           fn, (long long)seq_ids[i], b);
        ++leaving[b];
        ++new_blocks;
      }
    }
  }
  if (new_blocks > (int64_t)m->free_stack.size())
    return set_error(PKV_ERR_NOSPACE, "%s: %lld new blocks needed, %zu free", fn,
                     (long long)new_blocks, m->free_stack.size());
  int32_t np = 0;
  for (int32_t i = 0; i < n; ++i) {
    pkv_block_manager::Seq &s = *where[(size_t)i];
    const int64_t pos = s.len++;
    const int64_t lb = pos / m->block_size;
    if (lb >= (int64_t)s.blocks.size()) {
      s.blocks.push_back(m->take());
    } else if (m->refs[(size_t)s.blocks[(size_t)lb]] > 1) {
      const int32_t old = s.blocks[(size_t)lb], own = m->take();
      m->drop(old);
      s.blocks[(size_t)lb] = own;
      pairs[2 * np] = old;
      pairs[2 * np + 1] = own;
      rows[np++] = (int32_t)(pos % m->block_size);
    }
    slot_mapping[i] = (int64_t)s.blocks[(size_t)lb] * m->block_size + pos % m->block_size;
  }
  if (num_pairs) *num_pairs = np;
  pkv::clear_error();
  return PKV_OK;
}

}  // namespace

PKV_API int pkv_bm_append_slots(pkv_block_manager *m, const int64_t *seq_ids, int32_t n,
                                int64_t *slot_mapping) {
  if (!m || (n > 0 && (!seq_ids || !slot_mapping)))
    return set_error(PKV_ERR_NULL, "pkv_bm_append_slots: NULL argument");
  if (n < 0) return set_error(PKV_ERR_SHAPE, "pkv_bm_append_slots: n < 0");
  std::lock_guard<std::mutex> lk(m->mu);
  return guarded("pkv_bm_append_slots", [&]() -> int {
    return append(m, seq_ids, n, slot_mapping, nullptr, nullptr, nullptr, "pkv_bm_append_slots");
  });
}

PKV_API int pkv_bm_append_slots_cow(pkv_block_manager *m, const int64_t *seq_ids, int32_t n,
                                    int64_t *slot_mapping, int32_t *block_pairs,
                                    int32_t *num_tokens, int32_t *num_pairs) {
  if (!m || !num_pairs || (n > 0 && (!seq_ids || !slot_mapping || !block_pairs || !num_tokens)))
    return set_error(PKV_ERR_NULL, "pkv_bm_append_slots_cow: NULL argument");
  if (n < 0) return set_error(PKV_ERR_SHAPE, "pkv_bm_append_slots_cow: n < 0");
  std::lock_guard<std::mutex> lk(m->mu);
  return guarded("pkv_bm_append_slots_cow", [&]() -> int {
    return append(m, seq_ids, n, slot_mapping, block_pairs, num_tokens, num_pairs,
                  "pkv_bm_append_slots_cow");
  });
}

PKV_API int pkv_bm_free_sequence(pkv_block_manager *m, int64_t seq_id) {
  if (!m) return set_error(PKV_ERR_NULL, "pkv_bm_free_sequence: NULL manager");
  std::lock_guard<std::mutex> lk(m->mu);
  auto it = m->seqs.find(seq_id);
  if (it == m->seqs.end())
    return set_error(PKV_ERR_SHAPE, "pkv_bm_free_sequence: unknown sequence %lld",
                     (long long)seq_id);
  m->release(it->second);
  m->seqs.erase(it);
  pkv::clear_error();
  return PKV_OK;
}

PKV_API int pkv_bm_truncate(pkv_block_manager *m, int64_t seq_id, int64_t num_tokens) {
  if (!m) return set_error(PKV_ERR_NULL, "pkv_bm_truncate: NULL manager");
  std::lock_guard<std::mutex> lk(m->mu);
  auto it = m->seqs.find(seq_id);
  if (it == m->seqs.end())
    return set_error(PKV_ERR_SHAPE, "pkv_bm_truncate: unknown sequence %lld", (long long)seq_id);
  if (num_tokens < 0 || num_tokens > it->second.len)
    return set_error(PKV_ERR_SHAPE, "pkv_bm_truncate: %lld tokens of a sequence of %lld",
                     (long long)num_tokens, (long long)it->second.len);
  m->release(it->second, (size_t)m->blocks_for(num_tokens));
  it->second.len = num_tokens;
  pkv::clear_error();
  return PKV_OK;
}

PKV_API int32_t pkv_bm_ref_count(pkv_block_manager *m, int32_t block) {
  if (!m) return set_error(PKV_ERR_NULL, "pkv_bm_ref_count: NULL manager");
  if (block < 0 || block >= m->num_blocks)
    return set_error(PKV_ERR_SHAPE, "pkv_bm_ref_count: block %d", block);
  std::lock_guard<std::mutex> lk(m->mu);
  return m->refs[(size_t)block];
}

PKV_API int pkv_bm_compact(pkv_block_manager *m, int32_t *block_moves, int64_t max_moves,
                           int64_t *num_moves, int32_t *block_map) {
  if (!m || !num_moves || !block_map || (max_moves > 0 && !block_moves))
    return set_error(PKV_ERR_NULL, "pkv_bm_compact: NULL argument");
  if (max_moves < 0) return set_error(PKV_ERR_SHAPE, "pkv_bm_compact: max_moves < 0");
  std::lock_guard<std::mutex> lk(m->mu);
  const int64_t used = m->num_blocks - (int64_t)m->free_stack.size();
  int64_t want = 0;  // blocks in use past the first `used` ids
  for (int64_t b = used; b < m->num_blocks; ++b) want += m->refs[(size_t)b] > 0;
  *num_moves = want;
  if (want > max_moves)
    return set_error(PKV_ERR_NOSPACE, "pkv_bm_compact: %lld moves, room for %lld", (long long)want,
                     (long long)max_moves);
  int64_t to = 0, n = 0;  // the next free id below `used`: there are exactly `want`
  for (int64_t b = 0; b < m->num_blocks; ++b) block_map[b] = (int32_t)b;
  for (int64_t b = used; b < m->num_blocks; ++b) {
    if (m->refs[(size_t)b] == 0) continue;
    while (m->refs[(size_t)to] > 0) ++to;
    block_moves[2 * n] = (int32_t)b;
    block_moves[2 * n + 1] = (int32_t)to;
    ++n;
    block_map[b] = (int32_t)to;
    std::swap(m->refs[(size_t)b], m->refs[(size_t)to]);
  }
  for (auto &kv : m->seqs)
    for (int32_t &b : kv.second.blocks) b = block_map[b];
  m->free_stack.clear();
  for (int64_t b = m->num_blocks - 1; b >= used; --b) m->free_stack.push_back((int32_t)b);
  pkv::clear_error();
  return PKV_OK;
}

PKV_API int pkv_bm_preempt_lifo(pkv_block_manager *m, int64_t *seq_id) {
  if (!m || !seq_id) return set_error(PKV_ERR_NULL, "pkv_bm_preempt_lifo: NULL argument");
  std::lock_guard<std::mutex> lk(m->mu);
  if (m->seqs.empty()) return set_error(PKV_ERR_NOSPACE, "pkv_bm_preempt_lifo: no sequence to preempt");
  auto victim = m->seqs.begin();
  for (auto it = m->seqs.begin(); it != m->seqs.end(); ++it)
    if (it->second.order > victim->second.order) victim = it;
  *seq_id = victim->first;
  m->release(victim->second);
  m->seqs.erase(victim);
  pkv::clear_error();
  return PKV_OK;
}

PKV_API int pkv_bm_block_tables(pkv_block_manager *m, const int64_t *seq_ids, int32_t n,
                                int32_t max_blocks_per_seq, int32_t *block_tables,
                                int32_t *context_lens) {
  if (!m || (n > 0 && (!seq_ids || !block_tables || !context_lens)))
    return set_error(PKV_ERR_NULL, "pkv_bm_block_tables: NULL argument");
  if (n < 0 || max_blocks_per_seq <= 0)
    return set_error(PKV_ERR_SHAPE, "pkv_bm_block_tables: bad sizes");
  std::lock_guard<std::mutex> lk(m->mu);
  for (int32_t i = 0; i < n; ++i) {
    auto it = m->seqs.find(seq_ids[i]);
    if (it == m->seqs.end())
      return set_error(PKV_ERR_SHAPE, "pkv_bm_block_tables: unknown sequence %lld",
                       (long long)seq_ids[i]);
    const std::vector<int32_t> &blk = it->second.blocks;
    if ((int64_t)blk.size() > max_blocks_per_seq)
      return set_error(PKV_ERR_SHAPE, "pkv_bm_block_tables: sequence %lld has %zu blocks > %d",
                       (long long)seq_ids[i], blk.size(), max_blocks_per_seq);
    if (it->second.len > 0x7fffffffLL)
      return set_error(PKV_ERR_UNSUPPORTED, "pkv_bm_block_tables: length over 2^31-1");
    int32_t *row = block_tables + (int64_t)i * max_blocks_per_seq;
    std::copy(blk.begin(), blk.end(), row);
    std::fill(row + blk.size(), row + max_blocks_per_seq, -1);
    context_lens[i] = (int32_t)it->second.len;
  }
  pkv::clear_error();
  return PKV_OK;
}
