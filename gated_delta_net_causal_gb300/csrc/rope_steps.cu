// The frequencies of rotary positions as steps of 2^-64 of a turn (host code).
//
// A position of 2^31 multiplies a step's error by 2^31, so steps have to be
// right to the unit: of frequencies of up to 2^62 units, more than the 53 bits
// of a double. So numbers here are sums of two doubles (hi + lo, lo at most half
// a step of hi; Dekker 1971, Knuth's exact sum), about 2^-100 of themselves
// exact. The powers base^(-i / m), m = rotary_dim / 2, need no logarithm: their
// ratio is a double's pow, corrected by what base ratio^m differs from 1 by.
// Built without contraction of products and sums, so that the errors of sums
// come out exactly, and the same on every machine.
#include <math.h>
#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

struct Two {
  double hi, lo;
};

// a + b exactly; ordered_sum: for |a| >= |b|
Two ordered_sum(double a, double b) {
  const double s = a + b;
  return Two{s, b - (s - a)};
}
Two sum(double a, double b) {
  const double s = a + b, t = s - a;
  return Two{s, (a - (s - t)) + (b - t)};
}
Two add(Two a, Two b) {
  Two s = sum(a.hi, b.hi);
  const Two t = sum(a.lo, b.lo);
  s = ordered_sum(s.hi, s.lo + t.hi);
  return ordered_sum(s.hi, s.lo + t.lo);
}
Two mul(Two a, Two b) {
  const double p = a.hi * b.hi;
  return ordered_sum(p, fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
Two negative(Two a) { return Two{-a.hi, -a.lo}; }
// a / b, whose quotient is finite
Two div(Two a, Two b) {
  const double q = a.hi / b.hi;
  Two r = add(a, negative(mul(Two{q, 0.0}, b)));
  const double q2 = r.hi / b.hi;
  r = add(r, negative(mul(Two{q2, 0.0}, b)));
  return add(ordered_sum(q, q2), Two{r.hi / b.hi, 0.0});
}

const Two kOne = {1.0, 0.0};
// 1 / (2 pi)
const Two kTurn = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};

// the part of x past a whole number, in units of 2^-64
uint64_t units(Two x) {
  const double hi = ldexp(x.hi - floor(x.hi), 64);  // exact, below 2^64
  double lo = x.lo - rint(x.lo);
  if (lo >= 0.5) lo -= 1.0;
  lo = ldexp(lo, 64);
  const double whole_hi = floor(hi), whole_lo = floor(lo);
  return (uint64_t)whole_hi + (uint64_t)(int64_t)whole_lo +
         (uint64_t)floor((hi - whole_hi) + (lo - whole_lo) + 0.5);
}

}  // namespace

bool rope_steps(int32_t rotary_dim, double base, int32_t scaling, double factor, double original_length, double low,
                double high, uint64_t* step) {
  const double R = rotary_dim, m = rotary_dim / 2;
  const double two_pi = 6.283185307179586476925286766559;
  Two ratio = {pow(base, -1.0 / m), 0.0};
  for (int round = 0; round < 2; ++round) {
    Two over = {base, 0.0};  // base ratio^m, close to 1
    for (int i = 0; i < rotary_dim / 2; ++i) over = mul(over, ratio);
    over = add(over, Two{-1.0, 0.0});
    ratio = add(ratio, negative(mul(ratio, div(over, Two{m, 0.0}))));
  }
  double first = 0.0, last = 0.0;
  if (scaling == GDN_ROPE_RAMP) {
    const auto at = [&](double turns) { return R * log(original_length / (two_pi * turns)) / (2.0 * log(base)); };
    first = fmax(floor(at(high)), 0.0);
    last = fmin(ceil(at(low)), R - 1.0);
  }
  Two b = kOne;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    Two keep = kOne;  // share of b that is not stretched
    if (scaling == GDN_ROPE_LINEAR) {
      keep = Two{0.0, 0.0};
    } else if (scaling == GDN_ROPE_BANDS || scaling == GDN_ROPE_RAMP) {
      Two part, span;
      if (scaling == GDN_ROPE_BANDS) {
        part = add(mul(mul(Two{original_length, 0.0}, b), kTurn), Two{-low, 0.0});
        span = sum(high, -low);
      } else {
        part = Two{i - first, 0.0};
        span = Two{fmax(last - first, 0.001), 0.0};
      }
      // (far from the span the quotient may overflow)
      const double about = part.hi / span.hi;
      if (about <= -1.0) keep = Two{0.0, 0.0};
      else if (about < 2.0) keep = div(part, span);
      if (keep.hi < 0.0) keep = Two{0.0, 0.0};
      if (keep.hi > 1.0 || (keep.hi == 1.0 && keep.lo > 0.0)) keep = kOne;
      if (scaling == GDN_ROPE_RAMP) keep = add(kOne, negative(keep));
    }
    const Two rest = add(kOne, negative(keep));
    if (!isfinite(rest.hi / factor) && scaling != GDN_ROPE_PLAIN) return false;
    if (rest.hi != 0.0) keep = add(keep, div(rest, Two{factor, 0.0}));
    const Two turns = mul(mul(b, keep), kTurn);
    if (!isfinite(turns.hi) || !isfinite(turns.lo)) return false;
    step[i] = units(turns);
    b = mul(b, ratio);
  }
  return true;
}

}  // namespace gdn
