// Randomised host checks of how the gated linear recurrence's one pass groups
// more sequences than it sorts (csrc/gdn_plan.cpp), built with g++ and the
// address / undefined-behaviour sanitizers by tests/test_lru_limits_sanitized.py.
// Exits non-zero on the first broken invariant; a sanitizer report aborts on its
// own.
#include <algorithm>
#include <cstdio>
#include <random>
#include <utility>
#include <vector>

#include "gdn_plan.h"

// Nullptr unless the one pass takes units that hold several sequences one after
// another for far longer than the longest would take alone, and longer than the
// three steps would (8 us and 3 us per million elements; a round takes 10.5 us at
// least).
static const char* check(const std::vector<int64_t>& lens, int32_t D, bool resume) {
  const int32_t N = static_cast<int32_t>(lens.size());
  std::vector<int32_t> cu(lens.size() + 1, 0);
  int64_t longest = 0, chunks = 0;
  for (int32_t n = 0; n < N; ++n) {
    cu[n + 1] = static_cast<int32_t>(cu[n] + lens[n]);
    longest = std::max(longest, lens[n]);
    chunks += (lens[n] + 31) / 32;
  }
  gdn::LruPlan p;
  if (gdn::lru_plan(cu.data(), N, chunks, D, longest, resume, &p))
    return cu[N] > GDN_LRU_SMALL ? nullptr : "three steps without a workspace";
  if (p.per < 1 || p.per > gdn::kLruPack || p.units != (N + p.per - 1) / p.per) return "neighbours";
  const int64_t slots = p.threads / p.lps, lead = resume ? 62 : 31;
  int64_t worst = 0;
  for (int32_t n0 = 0; n0 < N; n0 += p.per) {
    int64_t held = 0;
    for (int32_t n = n0; n < N && n < n0 + p.per; ++n) held += lens[n] > 0 ? (lens[n] + lead) / 32 : 0;
    worst = std::max(worst, (held + slots - 1) / slots);
  }
  const int64_t alone = std::max<int64_t>(1, ((longest + lead) / 32 + slots - 1) / slots);
  const double three = 8.0 + 3e-6 * static_cast<double>(chunks * 32) * ((D + 63) / 64 * 64);
  if (cu[N] > GDN_LRU_SMALL && worst > 2 * alone && 10.5 * static_cast<double>(worst) > three) return "a unit of long sequences";
  return nullptr;
}

int main() {
  auto batch = [](std::vector<std::pair<int, int64_t>> runs) {
    std::vector<int64_t> lens;
    for (auto [count, len] : runs) lens.insert(lens.end(), static_cast<size_t>(count), len);
    return lens;
  };
  // short prompts with the long ones next to one another
  const char* what = check(batch({{5000, 1}, {10, 8000}}), 512, false);
  if (!what) what = check(batch({{200, 20}, {8, 2000}}), 256, false);
  if (!what) what = check(batch({{1000, 1}, {10, 8000}}), 1024, false);
  if (!what) what = check(batch({{10, 8000}, {1000, 1}}), 1024, true);
  if (!what) what = check(batch({{300, 0}, {5, 4000}, {300, 2}, {5, 4000}}), 2000, false);
  if (what) {
    std::fprintf(stderr, "lru_units_fuzz: %s\n", what);
    return 1;
  }
  std::mt19937_64 rng(11);
  auto pick = [&](int64_t lo, int64_t hi) { return lo + static_cast<int64_t>(rng() % static_cast<uint64_t>(hi - lo + 1)); };
  for (int it = 0; it < 8000; ++it) {
    std::vector<int64_t> lens;
    const int64_t runs = pick(1, 6);
    for (int64_t r = 0; r < runs; ++r) {
      const int64_t most = int64_t{1} << pick(0, 14), count = pick(1, most > 1000 ? 30 : 800);
      const bool equal = pick(0, 1);
      for (int64_t i = 0; i < count; ++i) lens.push_back(equal ? most : pick(0, most));
    }
    while (lens.size() <= static_cast<size_t>(gdn::kLruPack)) lens.push_back(pick(0, 3));
    if (pick(0, 2) == 0) std::sort(lens.begin(), lens.end());
    const int32_t D = static_cast<int32_t>(pick(1, int64_t{1} << pick(0, 14)));
    if ((what = check(lens, D, pick(0, 1)))) {
      std::fprintf(stderr, "lru_units_fuzz: %s (iteration %d, %zu sequences, %d channels)\n", what, it, lens.size(), D);
      return 1;
    }
  }
  std::puts("lru_units_fuzz: ok");
  return 0;
}
