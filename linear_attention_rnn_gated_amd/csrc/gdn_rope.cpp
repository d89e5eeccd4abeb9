// Rotary frequencies (host only, pure C++).  See include/gdn.h.
#include <cmath>

#include "gdn.h"

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

// The index i (not whole) of the pair that turns `turns` times in orig_len
// tokens: orig_len base^(-2i/r) = 2 pi turns.
double index_of_turns(double turns, int32_t r, double base, double orig_len) {
  return r * std::log(orig_len / (kTwoPi * turns)) / (2.0 * std::log(base));
}

}  // namespace

extern "C" int gdn_rope_freqs(int32_t r, double base, const gdn_rope_scaling_t* scaling, float* inv_freq,
                              float* rope_scale) {
  const gdn_rope_scaling_t none{GDN_ROPE_NONE, 1.0, 0.0, 0.0, 0.0, 0.0};
  const gdn_rope_scaling_t s = scaling ? *scaling : none;
  if (r <= 0 || r % 2 != 0 || !(base > 1.0) || !std::isfinite(base) || !inv_freq || !rope_scale)
    return GDN_ERR_INVALID_ARG;
  if (s.kind < GDN_ROPE_NONE || s.kind > GDN_ROPE_BANDS) return GDN_ERR_INVALID_ARG;
  const bool blended = s.kind == GDN_ROPE_YARN || s.kind == GDN_ROPE_BANDS;
  if (s.kind != GDN_ROPE_NONE && (!(s.factor >= 1.0) || !std::isfinite(s.factor))) return GDN_ERR_INVALID_ARG;
  if (s.kind == GDN_ROPE_NTK && r == 2) return GDN_ERR_INVALID_ARG;  // r / (r - 2)
  if (blended && (!(s.orig_len > 0.0) || !std::isfinite(s.orig_len) || !(s.low > 0.0) || !(s.high > s.low) ||
                  !std::isfinite(s.high) || !(s.attn >= 0.0) || !std::isfinite(s.attn)))
    return GDN_ERR_INVALID_ARG;
  if (s.kind == GDN_ROPE_NTK) base *= std::pow(s.factor, static_cast<double>(r) / (r - 2));
  double first = 0.0, last = 0.0;  // YARN: the pair indices between which the two are blended
  if (s.kind == GDN_ROPE_YARN) {
    first = std::fmax(std::floor(index_of_turns(s.high, r, base, s.orig_len)), 0.0);
    last = std::fmin(std::ceil(index_of_turns(s.low, r, base, s.orig_len)), r - 1.0);
    if (last <= first) last = first + 0.001;  // a step, no division by zero
  }
  for (int32_t i = 0; i < r / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / r);
    double keep = 1.0;  // share of the unscaled frequency
    if (s.kind == GDN_ROPE_YARN) keep = 1.0 - std::fmin(std::fmax((i - first) / (last - first), 0.0), 1.0);
    if (s.kind == GDN_ROPE_BANDS)
      keep = std::fmin(std::fmax((s.orig_len * f / kTwoPi - s.low) / (s.high - s.low), 0.0), 1.0);
    if (s.kind == GDN_ROPE_LINEAR) keep = 0.0;
    const bool scaled = blended || s.kind == GDN_ROPE_LINEAR;
    inv_freq[i] = static_cast<float>(scaled ? keep * f + (1.0 - keep) * f / s.factor : f);
  }
  double c = 1.0;
  if (blended) c = s.attn > 0.0 ? s.attn : s.kind == GDN_ROPE_YARN ? 0.1 * std::log(s.factor) + 1.0 : 1.0;
  *rope_scale = static_cast<float>(c);
  return GDN_OK;
}
