// How many CTAs sample one row (host only).
#pragma once
#include <stdint.h>

#include <algorithm>

namespace ls {

constexpr int kMaxCluster = 8;
// A sum of weights goes by three parts of 32 bits, each of fewer than 2^17 entries.
constexpr int kMaxSeg = 1 << 17;

// The fewest CTAs whose shared memory (`cap` entries each) holds the row; more while the rows
// leave places idle (two CTAs run on each of `sms` SMs) and a CTA's share is worth its part in
// the exchanges. Measured on 148 SMs, rows of 32,000 fp32 with top-p, 2 / 4 / 8 CTAs a row: 8
// rows 28.7 / 24.6 / 24.6 us, 16 rows 28.7 / 24.6 / 28.7, 32 rows 28.7 / 26.6 / 30.7, 36 rows
// 28.7 / 30.7 / 43.0, 48 rows 29.9 / 32.8 / 49.2: from 16 rows on the rule takes more CTAs than
// would be fastest (8 up to 37 rows, 4 up to 74), where clusters of 8 do not all fit at once.
inline int sample_cluster(int64_t rows, int32_t vocab, int cap, int sms) {
  int cluster = 1;
  while (cluster < kMaxCluster && (vocab + cluster - 1) / cluster > std::min(cap, kMaxSeg) - 8) cluster *= 2;
  while (cluster < kMaxCluster && rows * cluster * 2 <= 2ll * sms && vocab / cluster >= 4096) cluster *= 2;
  return cluster;
}

// Entries of a CTA's share: the last CTAs' may be shorter, or empty.
inline int32_t sample_share(int32_t vocab, int cluster) { return ((vocab + cluster - 1) / cluster + 7) / 8 * 8; }

}  // namespace ls
