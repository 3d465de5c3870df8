// Every key, also one that no sequence has, is looked up inside the table and the cache.
#include <cstdio>
#include <initializer_list>
#include <random>
#include <vector>

#include "q8_pages.cuh"

int main() {
  std::mt19937 r(1);
  for (int page_size : {16, 64, 128, 384, 1 << 20})
    for (int max_pages : {1, 3, 2046}) {
      ls::KvQ8 kv{};
      kv.page_size = page_size;
      kv.max_pages = max_pages;
      kv.num_pages = page_size == 1 << 20 ? 2047 : 5000;
      kv.page_shift = page_size == 384 ? -1 : __builtin_ctz(page_size);
      const int B = 3;
      std::vector<int32_t> table(B * max_pages);
      for (auto& x : table) x = r() % 4 ? (int32_t)(r() % kv.num_pages) : (int32_t)r();
      kv.page_table = table.data();
      const int64_t rows = (int64_t)kv.num_pages * page_size, held = (int64_t)max_pages * page_size;
      for (int i = 0; i < 400000; ++i) {
        int32_t key = (int32_t)r();
        if (i < 2000) key = INT32_MAX - i;
        else if (i < 4000) key = INT32_MIN + (i - 2000);
        else if (i < 200000) key = (int32_t)((uint32_t)r() % (uint32_t)(held < INT32_MAX ? held : INT32_MAX));
        const int b = i % B;
        const int64_t row = ls::q8_row(kv, b, key);
        if (row < 0 || row >= rows) {
          printf("page %d, key %d: row %lld\n", page_size, key, (long long)row);
          return 1;
        }
        if (key >= 0 && key < held) {
          const int32_t p = table[b * max_pages + key / page_size];
          const int64_t want = (int64_t)(p >= 0 && p < kv.num_pages ? p : 0) * page_size + key % page_size;
          if (row != want) {
            printf("page %d, key %d: row %lld, not %lld\n", page_size, key, (long long)row, (long long)want);
            return 1;
          }
        }
      }
    }
  // what the kernels look ahead of a sequence's end stays in 31 bits
  if (ls::kMaxCacheTokens + (1 << 20) + (1 << 16) > INT32_MAX) return 1;
  printf("ok\n");
  return 0;
}
