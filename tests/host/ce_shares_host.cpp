// Host check of ce_shares.cuh: over random launches every tile of every product is computed
// exactly once and the pairs' loads are level.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../sparsity_step_b200/csrc/ce_shares.cuh"

int main() {
  srand(1);
  for (int it = 0; it < 20000; ++it) {
    bl::CeShares share[3];
    int64_t tiles[3], costs[3], all = 0, most_cost = 1 << 30;
    const int products = 1 + rand() % 3;
    for (int j = 0; j < products; ++j) {
      int64_t c = 5 + rand() % (1 << (1 + rand() % 12));
      if (rand() % 4 && c > most_cost) c = most_cost;   // mostly the deepest first
      costs[j] = most_cost = c;
      tiles[j] = (1 + rand() % 40) * int64_t(1 + rand() % (1 << (1 + rand() % 8)));
      all += tiles[j];
    }
    const int limit = 1 + rand() % bl::kMaxCePairs, pairs = all < limit ? int(all) : limit;
    bl::ce_shares(share, tiles, costs, products, pairs);
    std::vector<int64_t> load(pairs, 0);
    int64_t total = 0, largest = 0;
    for (int j = 0; j < products; ++j) {
      std::vector<char> seen(tiles[j], 0);
      const bl::CeShares& S = share[j];
      for (int i = 0; i < pairs; ++i)
        for (int r = 0; r < S.count[i]; ++r) {
          if (r - S.common >= bl::kMaxCeExtra) return printf("launch %d: round %d is past the table\n", it, r), 1;
          const int t = bl::ce_round_tile(S, pairs, S.pos[i], r);
          if (t < 0 || t >= tiles[j] || seen[t]) return printf("launch %d: tile %d of product %d\n", it, t, j), 1;
          seen[t] = 1;
          load[i] += costs[j];
        }
      for (int64_t t = 0; t < tiles[j]; ++t)
        if (!seen[t]) return printf("launch %d: tile %ld of product %d is missing\n", it, long(t), j), 1;
      total += tiles[j] * costs[j];
      largest = costs[j] > largest ? costs[j] : largest;
    }
    int64_t high = 0;
    for (int64_t l : load) high = l > high ? l : high;
    if (high * pairs > total + 2 * largest * pairs) return printf("launch %d: load %ld\n", it, long(high)), 1;
  }
  puts("ok");
  return 0;
}
