// The 8-bit cache's pages: where a key of a sequence lies.
#pragma once
#include "ls_plan.cuh"

namespace ls {

struct KvQ8 {
  uint8_t* k_pages;  // [num_pages * page_size][Hkv][d]
  uint8_t* v_pages;
  float* k_scale;  // [num_pages * page_size / scale_block][Hkv]
  float* v_scale;
  const int32_t* page_table;  // [B][max_pages]
  int32_t page_size, scale_block, max_pages, num_pages;
  int32_t page_shift, scale_shift;  // their log2 (page_shift -1 where the page is no power of two)
};

// Tokens that a table may hold (max_pages * page_size): what lies ahead of a sequence's end, the
// rest of a page (2^20 at most) or of a kernel's steps, keeps its index in 31 bits.
constexpr int64_t kMaxCacheTokens = (int64_t(1) << 31) - (int64_t(1) << 21);

// First row of the page that holds key `key` of sequence b, plus the key's place in it. A
// table entry outside the cache reads page 0 instead, and a key past the table its last
// column (no fault, the result is unspecified): the row lies in the cache whatever the key is.
LS_HD int32_t q8_row(const KvQ8& kv, int32_t b, int32_t key) {
  const uint32_t k = (uint32_t)key;
  uint32_t lp = kv.page_shift >= 0 ? k >> kv.page_shift : k / (uint32_t)kv.page_size;
  const int32_t in = (int32_t)(k - lp * (uint32_t)kv.page_size);
  if (lp >= (uint32_t)kv.max_pages) lp = (uint32_t)kv.max_pages - 1;
  const int32_t page = kv.page_table[(size_t)b * kv.max_pages + lp];
  return ((uint32_t)page < (uint32_t)kv.num_pages ? page : 0) * kv.page_size + in;
}

}  // namespace ls
