// What the library's device translation units share: element types, the search
// for a packed row's sequence, and the kernel timing.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "gdn.h"
#include "gdn_plan.h"

// ---------------------------------------------------------------------------
// Kernel timing: optional HIP events around every launch.
namespace gdn __attribute__((visibility("hidden"))) {

struct ProfRec {
  const char* name;
  hipEvent_t a, b;
};
struct Profiler {
  std::mutex mu;
  bool on = false;
  std::string filter;  // only launches whose name contains it (empty: all)
  std::vector<ProfRec> recs;
  std::vector<hipEvent_t> pool;
  hipEvent_t get() {
    if (!pool.empty()) {
      hipEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    // timing-only events: no system-scope fence (no cache writeback and
    // invalidation around the timed launches); they are read only after the
    // caller has synchronised the device
    hipEvent_t e = nullptr;
    if (hipEventCreateWithFlags(&e, hipEventDisableSystemFence) != hipSuccess) return nullptr;
    return e;
  }
};
inline Profiler& prof() {
  static Profiler p;
  return p;
}

// Brackets the launches made in its scope with events when timing is on.
class Timed {
 public:
  Timed(const char* name, hipStream_t st) : st_(st) {
    Profiler& p = prof();
    std::lock_guard<std::mutex> g(p.mu);
    if (!p.on) return;
    if (!p.filter.empty() && std::strstr(name, p.filter.c_str()) == nullptr) return;
    rec_.name = name;
    rec_.a = p.get();
    rec_.b = p.get();
    if (rec_.a && rec_.b) {
      (void)hipEventRecord(rec_.a, st_);
      active_ = true;
    }
  }
  ~Timed() {
    if (!active_) return;
    (void)hipEventRecord(rec_.b, st_);
    Profiler& p = prof();
    std::lock_guard<std::mutex> g(p.mu);
    p.recs.push_back(rec_);
  }

 private:
  hipStream_t st_;
  ProfRec rec_{};
  bool active_ = false;
};

}  // namespace gdn

namespace {

using gdn::prof;
using gdn::Profiler;
using gdn::ProfRec;
using gdn::Timed;

using bf16_t = uint16_t;
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Two fp32 values rounded to nearest even, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

// Largest n in [0, N) with arr[n] <= x (arr non-decreasing, arr[0] = 0): the
// sequence that owns slot x.  Uniform across the block.
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ arr, int N, int64_t x) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (arr[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace
