// Frequencies of rotary positions (host and device; the host's use is its tests).
#pragma once
#include <math.h>
#include <stdint.h>

#include "ragged.cuh"

namespace fg {

// w_j = base^(-j / half), stretched for contexts longer than `original` positions: turns of w_j
// within them, r = original w_j / 2 pi, at least `high` leave w_j as it is, at most `low` divide it
// by `factor`, between them it goes over linearly in r; original 0 divides every w_j.
struct RopeScale {
  double base, factor, low, high, gain;
  int32_t original;
};
FG_HD double rope_frequency(const RopeScale& s, int j, int half) {
  const double w = pow(s.base, -(double)j / half);
  if (s.original == 0) return w / s.factor;
  const double r = s.original * w / 6.283185307179586476925;
  if (r >= s.high) return w;
  if (r <= s.low) return w / s.factor;
  const double g = (r - s.low) / (s.high - s.low);
  return w * g + w / s.factor * (1.0 - g);
}

}  // namespace fg
