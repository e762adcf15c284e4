// rope.h -- frequencies of a rotation (host only; the formulas are in
// include/w8a8.h).
//
// Worked out with 64 bits of mantissa (x87 long double) and rounded to binary64
// once: in binary64 the rounding of i / p alone, times ln(theta), costs several
// times as much as that rounding.  One power an axis, then a product a pair (64
// powers of long doubles take 31 us, as long as three whole calls; this 0.7).
//
// Relative errors but the last rounding, in units of 2^-53: the exponent's half
// step times ln(theta), below 710, 0.35; the same of factor's power 0.35; a power's
// last step and a product's half step, 255 times each, 0.25 + 0.125; a ramp next to
// 1, whose distance from it is 1/511 at least, 0.25 (not with factor's power).  In
// all 1.1, so a frequency is off by 1.25 * 2^-52 of itself at most; for theta and
// factor below 2^20 the logarithms give 0.04, in all 0.7, and it is off by 1.75 *
// 2^-53.
#pragma once

#include <math.h>

#include "w8a8.h"

namespace w8a8 {

inline long double ntk_theta(const w8a8_rope_t &r, int p) {
  if (p <= 1) return r.theta;
  return r.theta * powl(r.factor, (long double)p / (p - 1));
}

// Quarter turns a position of the pairs of an axis of p.
inline void rope_quarters(const w8a8_rope_t &r, int p, double *to) {
  const long double pi = 3.14159265358979323846264338327950288L;
  const long double theta =
      r.scaling == W8A8_ROPE_NTK ? ntk_theta(r, p) : (long double)r.theta;
  const long double step = powl(theta, -1.0L / p);
  long double low = 0, span = 1;
  if (r.scaling == W8A8_ROPE_YARN) {
    auto at = [&](long double turns) {
      return p * logl(r.original / (2 * pi * turns)) / logl(r.theta);
    };
    low = fmaxl(floorl(at(r.beta_fast)), 0.0L);
    const long double high = fminl(ceill(at(r.beta_slow)), 2.0L * p - 1);
    span = fmaxl(high - low, 0.001L);
  }
  long double power = 1;
  for (int i = 0; i < p; ++i, power *= step) {
    long double f = power;
    if (r.scaling == W8A8_ROPE_LINEAR) f /= r.factor;
    if (r.scaling == W8A8_ROPE_YARN) {
      const long double ramp = fminl(fmaxl((i - low) / span, 0.0L), 1.0L);
      f = f / r.factor * ramp + f * (1 - ramp);
    }
    to[i] = (double)(f * (2 / pi));
  }
}

}  // namespace w8a8
