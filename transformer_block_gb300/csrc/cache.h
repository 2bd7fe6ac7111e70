// cache.h — what the entry points on a paged cache share: the checks of a pb_cache, and the faults
// that its kernels record in its status word.
#pragma once

#include <cuda_bf16.h>

#include "heads.h"

namespace pb {

// Status word: PB_ERR_CACHE | fault << 8, the first one stays.
enum CacheFault : int {
  kFaultPages = 1,   // fewer free pages than needed
  kFaultRow = 2,     // a sequence longer than its row of the table
  kFaultSlot = 3,    // a slot outside [0, slots), or listed twice
  kFaultCounts = 4,  // starts that fall or leave [0, tokens], more tokens than the sequence has
  kFaultTable = 5,   // a page outside [0, pages), a length that is none
  kFaultPath = 6,    // a kept path that does not rise, or leaves the new tokens
  kFaultShared = 7,  // kept tokens would move into a page that another sequence uses too
};
constexpr int kMaxSlots = 1 << 16;  // a bit each in shared memory
constexpr int kMaxPages = 1 << 20;  // 1024 times as many are counted in 32 bits

inline int64_t page_values(const pb_cache& c) {  // of k or v in one page of one layer
  return int64_t(c.kv_heads) * c.page_size * c.head_dim;
}
inline size_t pool_bytes(const pb_cache& c) {
  return size_t(2 * c.layers * c.pages * page_values(c));
}
inline size_t table_bytes(const pb_cache& c) { return size_t(c.slots) * c.slot_pages * 4; }

inline pb_status check_cache_sizes(const pb_cache* c) {
  if (c == nullptr) return record_error(PB_ERR_INVALID_ARG, "cache is NULL");
  if (c->layers < 1 || c->pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->slots < 1 ||
      c->slot_pages < 1)
    return record_error(PB_ERR_INVALID_ARG, "cache: every size must be >= 1");
  if (c->head_dim != 64 && c->head_dim != 128)
    return record_error(PB_ERR_UNSUPPORTED, "cache: head_dim must be 64 or 128");
  if (c->slots > kMaxSlots) return record_error(PB_ERR_UNSUPPORTED, "cache: more than 2^16 slots");
  if (c->pages > kMaxPages || int64_t(c->slot_pages) * c->page_size > (1 << 30))
    return record_error(PB_ERR_UNSUPPORTED,
                        "cache: more than 2^20 pages, or 2^30 tokens in a row of the table");
  if (c->kv_heads > 65535 || c->layers > 65535)
    return record_error(PB_ERR_UNSUPPORTED, "cache: more than 65535 heads or layers");
  // values of a page, of a layer, of a pool: each product stays within 64 bits
  const int64_t most = int64_t(1) << 44;
  if (page_values(*c) > most / c->pages || page_values(*c) * c->pages > most / c->layers)
    return record_error(PB_ERR_UNSUPPORTED, "cache: more than 2^44 values in k or v");
  return PB_OK;
}

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

inline pb_status check_cache(const pb_cache* c) {
  const pb_status s = check_cache_sizes(c);
  if (s != PB_OK) return s;
  if (c->k == nullptr || c->v == nullptr || !aligned16(c->k) || !aligned16(c->v))
    return record_error(PB_ERR_INVALID_ARG, "cache: k and v must be 16-byte aligned device pointers");
  const Flat f[6] = {{c->k, pool_bytes(*c)},
                     {c->v, pool_bytes(*c)},
                     {c->table, table_bytes(*c)},
                     {c->lengths, size_t(c->slots) * 4},
                     {c->refs, size_t(c->pages) * 4},
                     {c->status, 4}};
  for (int i = 2; i < 6; ++i)
    if (f[i].p == nullptr || !aligned4(f[i].p))
      return record_error(PB_ERR_INVALID_ARG,
                          "cache: table, lengths, refs and status must be 4-byte aligned device "
                          "pointers");
  for (int i = 0; i < 6; ++i)
    for (int j = 0; j < i; ++j)
      if (!apart(f[i], f[j])) return record_error(PB_ERR_INVALID_ARG, "cache: its buffers overlap");
  return PB_OK;
}

// Whether f shares no byte with any buffer of the cache.
inline bool apart_from_cache(const Flat& f, const pb_cache& c) {
  return apart(f, Flat{c.k, pool_bytes(c)}) && apart(f, Flat{c.v, pool_bytes(c)}) &&
         apart(f, Flat{c.table, table_bytes(c)}) && apart(f, Flat{c.lengths, size_t(c.slots) * 4}) &&
         apart(f, Flat{c.refs, size_t(c.pages) * 4}) && apart(f, Flat{c.status, 4});
}

#ifdef __CUDACC__
__device__ __forceinline__ void cache_fault(int* status, int fault) {
  atomicCAS(status, 0, int(PB_ERR_CACHE) | (fault << 8));
}
#endif

}  // namespace pb
