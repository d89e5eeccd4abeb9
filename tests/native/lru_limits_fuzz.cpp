// Randomised host checks of the sizes that the gated linear recurrence takes
// (csrc/gdn_plan.cpp), built with g++ and the address / undefined-behaviour
// sanitizers by tests/test_lru_limits_sanitized.py.  Exits non-zero on the first
// broken invariant; a sanitizer report aborts on its own.
#include <cstdio>
#include <random>
#include <vector>

#include "gdn_plan.h"

static int fail(const char* what, long long a, long long b, long long c) {
  std::fprintf(stderr, "lru_limits_fuzz: %s (%lld, %lld, %lld)\n", what, a, b, c);
  return 1;
}

int main() {
  // 32768 sequences x 4096 channels, one of them past a round: the trainer's chains run at 256 channels a block
  if (gdn::lru_chain_width(32768, 4096, 1100, 2) != 256) return fail("32768 x 4096", 32768, 4096, 1100);
  if (gdn::lru_chain_width(65536, 4096, 5000, 2) != 256) return fail("65536 x 4096", 65536, 4096, 5000);
  if (gdn::lru_chain_width(12, 200, 14162, 1) != 16) return fail("few long ones", 12, 200, 14162);
  if (gdn::lru_chain_width(15, 972, 4475, 1) != 32) return fail("some long ones", 15, 972, 4475);
  if (gdn::lru_chain_width(INT32_MAX, 1 << 20, 40, 2) != 0) return fail("past every launch", INT32_MAX, 1 << 20, 40);
  std::mt19937_64 rng(7);
  auto pick = [&](int64_t lo, int64_t hi) { return lo + static_cast<int64_t>(rng() % static_cast<uint64_t>(hi - lo + 1)); };
  for (int it = 0; it < 200000; ++it) {
    const int32_t N = static_cast<int32_t>((int64_t{1} << pick(0, 30)) + pick(0, 1000));
    const int32_t D = static_cast<int32_t>(pick(1, int64_t{1} << pick(0, 20)));
    const int64_t longest = pick(0, int64_t{1} << pick(0, 30));
    for (int dirs = 1; dirs <= 2; ++dirs) {
      const int w = gdn::lru_chain_width(N, D, longest, dirs);
      if (w != 0 && w != 16 && w != 32 && w != 256) return fail("width", N, D, longest);
      if (w && gdn::lru_chain_blocks(N, D, w) * dirs * 256 >= gdn::kLaunchThreads) return fail("launch", N, D, longest);
      // refused only where the widest blocks do not fit either
      if (!w && gdn::lru_chain_blocks(N, D, 256) * dirs * 256 < gdn::kLaunchThreads) return fail("refused", N, D, longest);
    }
  }
  // no batch of N max(D, 64) <= 2^24 and T max(D, 64) <= 2^35 is refused, whichever way it runs
  for (int it = 0; it < 400; ++it) {
    const int32_t D = static_cast<int32_t>(pick(1, int64_t{1} << pick(0, 20)));
    const int64_t wide = D > 64 ? D : 64, most = (int64_t{1} << 24) / wide;
    const int32_t N = static_cast<int32_t>(pick(0, 3) ? pick(1, most < 300 ? most : 300) : pick(most / 2 + 1, most));
    const int64_t tokens = (int64_t{1} << 35) / wide < INT32_MAX ? (int64_t{1} << 35) / wide : INT32_MAX;
    const int64_t mean = pick(0, 1) ? tokens / N : pick(0, 3);
    std::vector<int32_t> cu(static_cast<size_t>(N) + 1, 0);
    int64_t longest = 0, chunks = 0, left = tokens;
    for (int32_t n = 0; n < N; ++n) {
      int64_t len = pick(0, 3) ? pick(0, 2 * mean) : mean;
      len = len < left ? len : left;
      left -= len;
      cu[n + 1] = static_cast<int32_t>(cu[n] + len);
      longest = len > longest ? len : longest;
      chunks += (len + 31) / 32;
    }
    auto fits = [](int64_t blocks, int64_t threads) { return blocks * threads < gdn::kLaunchThreads; };
    gdn::LruPlan p;
    const bool three = gdn::lru_plan(cu.data(), N, chunks, D, longest, pick(0, 1), &p);
    if (!three && !fits(static_cast<int64_t>(p.units) * ((D + p.lps - 1) / p.lps) + 31, p.threads))
      return fail("one pass", N, D, cu[N]);
    if (gdn::lru_train_plan(cu.data(), N, chunks, D, longest, &p) &&
        !fits(static_cast<int64_t>(p.units) * ((D + p.lps - 1) / p.lps) + 31, p.threads))
      return fail("trainer's one pass", N, D, cu[N]);
    if (!gdn::lru_chain_width(N, D, longest, 2)) return fail("chain", N, D, longest);
    int64_t cw = 64;  // the other steps' blocks: cw channels of 256 / cw chunks
    while (cw < 256 && cw < D) cw *= 2;
    const int64_t per = 256 / cw, slots = gdn::lru_slots(cu[N], N);
    if (!fits((slots + per - 1) / per * ((D + cw - 1) / cw), 256)) return fail("steps", N, D, cu[N]);
  }
  std::puts("lru_limits_fuzz: ok");
  return 0;
}
