// Rotary frequencies and positions (host side): the per-pair rotation speeds
// of a head, stretched for long contexts where asked, as 64-bit phases for the
// rotation kernels, and the position of every packed row of a lowered step.
// Plain C++; nothing here touches a GPU.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "pkv.h"

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

// Fraction of a turn per position as a 64-bit fixed-point number. The
// rotation of position p is then p * phase modulo 2^64, exactly, for any
// 32-bit p: whole turns fall off the top.
uint64_t phase_of(double f) {
  const double turns = std::fmod(std::fabs(f) / kTwoPi, 1.0);
  const uint64_t u = static_cast<uint64_t>(std::ldexp(turns, 64));  // turns < 1 - 2^-54: fits
  return f < 0 ? ~u + 1 : u;
}

}  // namespace

extern "C" {

pkv_status pkv_rope_phases(const double *frequencies, int32_t num_pairs, uint64_t *phases) {
  if (num_pairs < 0 || (num_pairs > 0 && (!frequencies || !phases))) return PKV_ERR_INVALID_ARG;
  for (int32_t i = 0; i < num_pairs; ++i)
    if (!std::isfinite(frequencies[i])) return PKV_ERR_INVALID_ARG;
  for (int32_t i = 0; i < num_pairs; ++i) phases[i] = phase_of(frequencies[i]);
  return PKV_OK;
}

pkv_status pkv_rope_plan(const pkv_rope_config *c, double *frequencies, uint64_t *phases, float *magnitude) {
  if (!c || c->rot_dim < 2 || c->rot_dim % 2 != 0 || c->rot_dim > 65536) return PKV_ERR_INVALID_ARG;
  if (!std::isfinite(c->base) || !(c->base > 1.0)) return PKV_ERR_INVALID_ARG;
  const bool scaled = c->scaling != PKV_ROPE_NONE;
  if (scaled && (!std::isfinite(c->factor) || !(c->factor > 0.0))) return PKV_ERR_INVALID_ARG;
  const bool by_turns = c->scaling == PKV_ROPE_BY_PARTS || c->scaling == PKV_ROPE_YARN;
  if (by_turns && (c->original_len <= 0 || !std::isfinite(c->high) || !(c->low > 0.0) || !(c->high > c->low)))
    return PKV_ERR_INVALID_ARG;
  const int32_t pairs = c->rot_dim / 2;
  const double n = c->rot_dim, s = scaled ? c->factor : 1.0;
  double base = c->base;
  float mag = 1.f;
  switch (c->scaling) {
    case PKV_ROPE_NONE:
    case PKV_ROPE_LINEAR:
    case PKV_ROPE_BY_PARTS: break;
    case PKV_ROPE_NTK:
      if (c->rot_dim < 4) return PKV_ERR_INVALID_ARG;  // the exponent rot_dim / (rot_dim - 2)
      base *= std::pow(s, n / (n - 2.0));
      if (!std::isfinite(base)) return PKV_ERR_INVALID_ARG;
      break;
    case PKV_ROPE_YARN:
      if (s > 1.0) mag = static_cast<float>(0.1 * std::log(s) + 1.0);
      break;
    default: return PKV_ERR_INVALID_ARG;
  }
  // Pair index at which a pair makes `turns` turns over the original context.
  auto index_of = [&](double turns) {
    return n * std::log(c->original_len / (kTwoPi * turns)) / (2.0 * std::log(c->base));
  };
  const double first = c->scaling == PKV_ROPE_YARN ? std::max(std::floor(index_of(c->high)), 0.0) : 0.0;
  const double last = c->scaling == PKV_ROPE_YARN ? std::min(std::ceil(index_of(c->low)), n - 1.0) : 0.0;
  auto frequency = [&](int32_t i) {
    const double f = std::pow(base, -2.0 * i / n);
    if (c->scaling == PKV_ROPE_LINEAR) return f / s;
    if (c->scaling == PKV_ROPE_BY_PARTS) {
      const double g =
          std::min(1.0, std::max(0.0, (c->original_len * f / kTwoPi - c->low) / (c->high - c->low)));
      return f * (g + (1.0 - g) / s);
    }
    if (c->scaling == PKV_ROPE_YARN) {
      const double g = std::min(1.0, std::max(0.0, (i - first) / std::max(last - first, 0.001)));
      return f * ((1.0 - g) + g / s);
    }
    return f;
  };
  // A factor near 0 can take a frequency past the largest double (and base past the smallest).
  for (int32_t i = 0; i < pairs; ++i)
    if (!std::isfinite(frequency(i))) return PKV_ERR_INVALID_ARG;
  for (int32_t i = 0; i < pairs; ++i) {
    const double f = frequency(i);
    if (frequencies) frequencies[i] = f;
    if (phases) phases[i] = phase_of(f);
  }
  if (magnitude) *magnitude = mag;
  return PKV_OK;
}

pkv_status pkv_plan_positions(const int32_t *cu, int32_t num_seqs, const int32_t *seq_slot,
                              const int32_t *context_lens, int32_t max_slots, int32_t *positions, int64_t capacity) {
  if (!cu || num_seqs < 0 || (num_seqs > 0 && (!seq_slot || !context_lens)) || max_slots <= 0 || cu[0] != 0)
    return PKV_ERR_INVALID_ARG;
  for (int32_t s = 0; s < num_seqs; ++s) {
    const int64_t n = static_cast<int64_t>(cu[s + 1]) - cu[s];
    if (n < 0) return PKV_ERR_INVALID_ARG;
    if (seq_slot[s] < 0 || seq_slot[s] >= max_slots) return PKV_ERR_OUT_OF_RANGE;
    if (n > context_lens[seq_slot[s]]) return PKV_ERR_INVALID_ARG;
  }
  if (cu[num_seqs] > 0 && (!positions || capacity < cu[num_seqs])) return PKV_ERR_WORKSPACE_TOO_SMALL;
  for (int32_t s = 0; s < num_seqs; ++s) {
    const int32_t n = cu[s + 1] - cu[s], first = context_lens[seq_slot[s]] - n;
    for (int32_t i = 0; i < n; ++i) positions[cu[s] + i] = first + i;
  }
  return PKV_OK;
}

}  // extern "C"
