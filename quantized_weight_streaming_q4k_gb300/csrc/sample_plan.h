// sample_plan.h -- how many CTAs share a row of sample_tokens (host, without CUDA).
#pragma once

#include <cstdint>

namespace qws {

constexpr int kSaThreads = 1024;
constexpr int kSaMaxCluster = 16;
constexpr int kSaMaxSlice = 43 * 1024;       // logits of a CTA, in shared memory

// As many CTAs a row as its logits need, and more, down to two logits a thread, while the rows
// do not take more turns for it: 64 rows of 262144, top_k 64, 61 us with 6 CTAs, 79 with 8; 9 rows
// 21.6 with 6, 17.5 with 10, 29 with 12; a row of 32000 17 with 1, 10.7 with 16.
// at_once(size): clusters of that size that the device runs at once; one that it does not run at
// all (0: too few neighbouring SMs in reach) is never chosen.  0: it runs none that is large enough.
template <class AtOnce>
int sample_cluster_size(int64_t vocab, int64_t n_rows, AtOnce at_once) {
  const int least = static_cast<int>((vocab + kSaMaxSlice - 1) / kSaMaxSlice);
  int size = 0;
  int64_t turns = 0;
  for (int i = least; i <= kSaMaxCluster; ++i) {
    if (size && vocab < int64_t(2) * kSaThreads * i) break;
    const int64_t n = at_once(i);
    if (n <= 0) continue;
    const int64_t t = (n_rows + n - 1) / n;
    if (size == 0 || t <= turns) {
      turns = t;
      size = i;
    }
  }
  return size;
}

}  // namespace qws
