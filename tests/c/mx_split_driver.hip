// The split of the grouped products' tile list over the XCDs, by the library's own functions, on
// random numbers of pairs an expert: every tile lies in one XCD's run, and the grid that the
// host launches covers the longest run. Host code alone: nothing is launched.
#include <cstdio>
#include <random>
#include <vector>

#include "qmoe_mx_internal.h"

using namespace qmoe;

static int failures = 0;
static long long longest = 0;

static void check(const std::vector<int>& pairs, const char* what) {
  std::vector<int> rows, expert;
  long long P = 0;
  for (size_t e = 0; e < pairs.size(); ++e) {
    for (int i = 0; i < pairs[e]; i += kMxBM) rows.push_back(std::min(kMxBM, pairs[e] - i)), expert.push_back((int)e);
    P += pairs[e];
  }
  if (P == 0) return;
  const int most = mx_max_mtiles((int)P, (int)pairs.size());
  if (most < (int)rows.size()) {
    std::printf("%s: %zu tiles, the host allows for %d\n", what, rows.size(), most);
    ++failures;
  }
  // the whole by experts, as the list's scan adds it up, is the whole by tiles
  int total = 0, by_tile = 0;
  for (int n : pairs) total += mx_tiles_cost((n + kMxBM - 1) / kMxBM, n);
  for (int r : rows) by_tile += mx_tiles_cost(1, r);
  int first[kMxXcds + 1];
  for (int& f : first) f = -1;
  first[kMxXcds] = (int)rows.size();
  int before = 0;
  for (size_t j = 0; j < rows.size(); ++j) {
    const int next = before + mx_tiles_cost(1, rows[j]);
    mx_xcd_starts((int)j, before, next, total, first);
    before = next;
  }
  bool good = total == by_tile && first[0] == 0;
  for (int x = 0; x < kMxXcds; ++x) good = good && first[x] >= 0 && first[x] <= first[x + 1];
  for (int ntn : {1, 3, 64})
    for (int x = 0; x < kMxXcds; ++x)
      good = good && (long long)(first[x + 1] - first[x]) * ntn <= mx_list_grid(most, ntn) / kMxXcds;
  if (!good) {
    std::printf("%s: %zu experts, %zu tiles, cost %d / %d\n", what, pairs.size(), rows.size(), total, by_tile);
    ++failures;
  }
  longest = std::max(longest, (long long)rows.size());
}

int main() {
  std::mt19937 rng(1);
  auto below = [&](int n) { return (int)(rng() % n); };
  for (int turn = 0; turn < 4000; ++turn) {
    const int sizes[] = {1, 2, 3, 64, 512, MOE_MAX_EXPERTS};
    std::vector<int> pairs(sizes[below(6)]);
    const int kind = below(5), one = 1 + below(400);
    for (int& n : pairs) switch (kind) {
        case 0: n = below(3) ? 0 : below(3000); break;
        case 1: n = below(40); break;
        case 2: n = one; break;
        case 3: n = below(50) ? 1 : 8192; break;
        default: n = kMxBM * below(3) + below(2); break;
      }
    check(pairs, "random");
  }
  // the ends: all pairs of the largest chunk to one expert, and one pair an expert
  std::vector<int> all(MOE_MAX_EXPERTS, 0);
  for (int e : {0, 500, MOE_MAX_EXPERTS - 1}) {
    all[e] = MOE_MAX_PREFILL_TOKENS * MOE_MAX_TOP_K;
    check(all, "one expert");
    all[e] = 0;
  }
  for (int n = 1; n <= MOE_MAX_EXPERTS; ++n) check(std::vector<int>(n, 1), "one pair each");
  std::printf("mx split: %d failures, at most %lld tiles\n", failures, longest);
  return failures != 0;
}
