// Randomised host checks of the gated linear recurrence's plan and of the
// rotary frequencies (csrc/gdn_plan.cpp, csrc/gdn_rope.cpp), built with g++ and
// the address / undefined-behaviour sanitizers by
// tests/test_lru_plan_sanitized.py.  Exits non-zero on the first broken
// invariant; a sanitizer report aborts on its own.
#include <cmath>
#include <cstdio>
#include <random>
#include <vector>

#include "gdn_plan.h"

static int fail(const char* what, int iter) {
  std::fprintf(stderr, "lru_plan_fuzz: %s (iteration %d)\n", what, iter);
  return 1;
}

// Nullptr if a plan's units hold every sequence once, several together only
// where they fit a round.
static const char* units(const std::vector<int32_t>& cu, const gdn::LruPlan& p, bool resume) {
  const int N = static_cast<int>(cu.size()) - 1;
  if (p.per) {
    if (N <= gdn::kLruPack || p.per < 0 || p.per > gdn::kLruPack || p.units != (N + p.per - 1) / p.per)
      return "neighbours";
    return nullptr;
  }
  if (N > gdn::kLruPack || p.units > N || p.first[0] != 0 || p.first[p.units] != N) return "packing";
  std::vector<int> seen(static_cast<size_t>(N), 0);
  const int64_t round = p.threads / p.lps * GDN_LRU_CHUNK;
  for (int u = 0; u < p.units; ++u) {
    if (p.first[u + 1] <= p.first[u]) return "empty unit";
    int64_t chunks = 0;
    int held = 0;
    for (int i = p.first[u]; i < p.first[u + 1]; ++i) {
      const int n = p.seq[i];
      if (n >= N || seen[n]++) return "sequence";
      const int64_t len = static_cast<int64_t>(cu[n + 1]) - cu[n];
      if (len > 0) {
        ++held;
        chunks += (len + (resume ? 31 : 0) + 31) / 32;
      }
    }
    if (held > 1 && chunks * 32 > round) return "a unit of several sequences exceeds a round";
  }
  for (int s : seen)
    if (s != 1) return "a sequence is missing";
  return nullptr;
}

int main() {
  std::mt19937_64 rng(2024);
  auto pick = [&](int64_t lo, int64_t hi) { return lo + static_cast<int64_t>(rng() % static_cast<uint64_t>(hi - lo + 1)); };
  for (int it = 0; it < 20000; ++it) {
    const int N = static_cast<int>(pick(0, 3) ? pick(0, 64) : pick(65, 300));
    const int64_t most = pick(0, 2) == 0 ? 40 : pick(0, 1) ? pick(100, 2999) : 100000;
    std::vector<int32_t> cu(static_cast<size_t>(N) + 1, 0);
    int64_t longest = 0, chunks = 0;
    for (int n = 0; n < N; ++n) {
      const int64_t len = pick(0, 4) == 0 ? 0 : pick(0, most);
      cu[n + 1] = static_cast<int32_t>(cu[n] + len);
      longest = len > longest ? len : longest;
      chunks += (len + 31) / 32;
    }
    const int32_t D = static_cast<int32_t>(pick(0, 9) == 0 ? pick(1, 1 << 20) : pick(1, 9000));
    const bool resume = pick(0, 1);
    gdn::LruPlan p;
    const bool three = gdn::lru_plan(cu.data(), N, chunks, D, longest, resume, &p);
    if (three && cu[N] <= GDN_LRU_SMALL) return fail("three steps without a workspace", it);
    if (p.lps != 8 && p.lps != 16 && p.lps != 32 && p.lps != 64) return fail("tile", it);
    if (p.threads < 64 || p.threads > gdn::kLruThreads || p.threads % 64 != 0 || p.threads < p.lps)
      return fail("threads", it);
    if (!three) {
      if (const char* what = units(cu, p, resume)) return fail(what, it);
    }
    gdn::LruPlan q;
    if (!gdn::lru_train_plan(cu.data(), N, chunks, D, longest, &q)) continue;
    if (q.lps != 16 && q.lps != 32 && q.lps != 64) return fail("trainer's tile", it);
    if (q.threads < 64 || q.threads > gdn::kLruTrain || q.threads % 64 != 0) return fail("trainer's threads", it);
    if ((longest + 31) / 32 > q.threads / q.lps) return fail("a sequence exceeds the trainer's round", it);
    if (const char* what = units(cu, q, false)) return fail(what, it);
    for (int i0 = 0; q.per && i0 < N; i0 += q.per) {
      int64_t held = 0;
      for (int n = i0; n < N && n < i0 + q.per; ++n) held += (cu[n + 1] - cu[n] + 31) / 32;
      if (held > q.threads / q.lps) return fail("neighbours exceed the trainer's round", it);
    }
  }
  for (int it = 0; it < 20000; ++it) {
    const int32_t r = static_cast<int32_t>(pick(-4, 300));
    gdn_rope_scaling_t s{};
    s.kind = static_cast<int32_t>(pick(-1, 5));
    s.factor = static_cast<double>(pick(0, 400)) / 10.0;
    s.orig_len = static_cast<double>(pick(-1, 100000));
    s.low = static_cast<double>(pick(0, 40)) / 4.0;
    s.high = static_cast<double>(pick(0, 400)) / 4.0;
    s.attn = static_cast<double>(pick(-1, 20)) / 10.0;
    const double base = static_cast<double>(pick(0, 1) ? pick(0, 3) : pick(2, 10000000));
    std::vector<float> f(r > 0 ? static_cast<size_t>(r) / 2 : 0, -1.0f);
    float c = -1.0f;
    const int rc = gdn_rope_freqs(r, base, pick(0, 9) ? &s : nullptr, f.empty() ? nullptr : f.data(), &c);
    if (rc == GDN_OK) {
      if (!(c > 0.0f)) return fail("rope_scale", it);
      for (float v : f)
        if (!(v >= 0.0f && v <= 1.0f)) return fail("frequency", it);
    } else if (rc != GDN_ERR_INVALID_ARG || c != -1.0f) {
      return fail("status", it);
    }
  }
  std::puts("lru_plan_fuzz: ok");
  return 0;
}
