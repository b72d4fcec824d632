// Which tiles of the products of one launch every CTA pair computes (linear_ce.cuh,
// gemm_fp8.cuh). Host code but for ce_round_tile.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define BL_HOST_DEVICE __host__ __device__
#else
#define BL_HOST_DEVICE
#endif

namespace bl {

constexpr int kMaxCePairs = 80;
constexpr int kMaxCeExtra = 48;
// Which tiles of a product a CTA pair computes: `count` of them, one a round; the pairs stand
// in the order of their counts (`pos`), so that a round's tiles are consecutive and its pairs
// the first ones. Every pair takes part in the first `common` rounds; round common + i
// begins at tile start[i].
struct CeShares {
  int16_t pos[kMaxCePairs];
  int count[kMaxCePairs];
  int common;
  int start[kMaxCeExtra];
};
// Tile of round r for the pair at position pos.
BL_HOST_DEVICE inline int ce_round_tile(const CeShares& S, int pairs, int pos, int r) {
  return (r < S.common ? r * pairs : S.start[r - S.common]) + pos;
}

// Shares of several products (`tiles` tiles of `costs` each) among `pairs` CTA pairs: every
// product raises the pairs' loads to a common level, its last tiles going to the least
// loaded. With the deepest products first all pairs end within about one tile of each other;
// tiles of different depth dealt out in turn left some with twice the work of others
// (2047 x 1536 x 32003, forward and backward: 738 -> 660 us).
inline void ce_shares(CeShares* share, const int64_t* tiles, const int64_t* costs, int products, int pairs) {
  int64_t load[kMaxCePairs] = {};
  for (int j = 0; j < products; ++j) {
    CeShares& S = share[j];
    const int64_t n = tiles[j], cost = costs[j];
    int64_t top = 0;
    for (int i = 0; i < pairs; ++i) top = top > load[i] ? top : load[i];
    // no pair may be more than the table's rounds ahead of another
    for (int i = 0; i < pairs; ++i)
      if (load[i] < top - (kMaxCeExtra - 2) * cost) load[i] = top - (kMaxCeExtra - 2) * cost;
    // the level that n tiles raise all loads to; where some load is already above it, the
    // highest one that takes at most n tiles
    int64_t sum = n * cost;
    for (int i = 0; i < pairs; ++i) sum += load[i];
    int64_t lo = sum / pairs;
    if (lo < top) {
      auto taken = [&](int64_t level) {
        int64_t fit = 0;
        for (int i = 0; i < pairs; ++i) fit += level > load[i] ? (level - load[i]) / cost : 0;
        return fit;
      };
      int64_t hi = top + 1;
      lo = 0;
      while (hi - lo > 1) {
        const int64_t mid = lo + (hi - lo) / 2;
        if (taken(mid) <= n) lo = mid;
        else hi = mid;
      }
    }
    int64_t left = n;
    for (int i = 0; i < pairs; ++i) {
      S.count[i] = lo > load[i] ? static_cast<int>((lo - load[i]) / cost) : 0;
      load[i] += S.count[i] * cost;
      left -= S.count[i];
    }
    for (; left > 0; --left) {   // fewer than there are pairs
      int least = 0;
      for (int i = 1; i < pairs; ++i)
        if (load[i] < load[least]) least = i;
      ++S.count[least];
      load[least] += cost;
    }
    int common = S.count[0], most = S.count[0];
    for (int i = 1; i < pairs; ++i) {
      common = common < S.count[i] ? common : S.count[i];
      most = most > S.count[i] ? most : S.count[i];
    }
    int at = 0;   // positions by falling count
    for (int c = most; c >= common; --c)
      for (int i = 0; i < pairs; ++i)
        if (S.count[i] == c) S.pos[i] = static_cast<int16_t>(at++);
    S.common = common;
    int start = common * pairs;
    for (int r = common; r < most; ++r) {
      S.start[r - common] = start;
      for (int i = 0; i < pairs; ++i) start += S.count[i] > r ? 1 : 0;
    }
  }
}

}  // namespace bl
