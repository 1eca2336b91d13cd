// kv_cache.cuh -- the paged INT8 key/value cache as its kernels see it: the
// block of 16 tokens, where a code stands in it, and a sequence's new tokens.
#pragma once

#include <cstdint>

#include "qlin_device.cuh"
#include "qlin_internal.h"

namespace qlin {

constexpr int kHeadDim = 128;
constexpr int kVCodes = 2048;    // offsets in a block
constexpr int kKScales = 4096;
constexpr int kVScales = 4160;

// Offset, in a token's 128 codes, of component d (its 32-byte quarter moved).
__device__ __forceinline__ int code_place(int r, int d) { return ((((d >> 5) ^ (r >> 2)) & 3) << 5) + (d & 31); }

// A sequence's tokens in the cache, and how many of them are new.  (Read from L2:
// the kernel that joins the attention's parts reads them before its wait.)
struct SeqLen {
  int len, fresh;
};
__device__ __forceinline__ SeqLen seq_of(const CacheArgs& c, int64_t T, int total, int fresh) {
  SeqLen s;
  s.len = min(max(total, 0), static_cast<int>(c.max_pages * c.page_size));
  s.fresh = min(max(fresh, 0), static_cast<int>(T < s.len ? T : s.len));
  return s;
}
__device__ __forceinline__ int fresh_of(const CacheArgs& c, int64_t b) {
  return c.new_len == nullptr ? 0x7FFFFFFF : __ldcg(c.new_len + b);
}
__device__ __forceinline__ SeqLen seq_len(const CacheArgs& c, int64_t b, int64_t T) {
  return seq_of(c, T, __ldcg(c.total_len + b), fresh_of(c, b));
}

// Block of 16 that holds tokens 16 n .. 16 n + 15 of sequence b, head h;
// nullptr where its page is none.
__device__ __forceinline__ uint8_t* cache_block(const CacheArgs& c, int64_t b, int h, int n) {
  const int per_page = static_cast<int>(c.page_size) >> 4;
  const int in_table = per_page == 1 ? n : n / per_page;
  const int page = __ldg(c.block_table + b * c.max_pages + in_table);
  if (page < 0 || page >= c.pages) return nullptr;
  return c.cache + ((page * c.kv_heads + h) * per_page + (n - in_table * per_page)) * static_cast<int64_t>(kCacheBlock);
}

}  // namespace qlin
