// Host arithmetic with twice a double's precision: a number is the unevaluated
// sum of two doubles, the second at most half a unit in the last place of the
// first (Dekker, 1971; the error-free sum is Knuth's). Results are within a few
// 2^-104 of their value. Needs a compiler that does not contract a * b + c by itself.
#pragma once

#include <cmath>

namespace moe {

struct Twice {
  double hi, lo;
  constexpr Twice(double hi = 0.0, double lo = 0.0) : hi(hi), lo(lo) {}
};

// |a| >= |b|, or a is 0.
inline Twice quick_sum(double a, double b) {
  const double s = a + b;
  return {s, b - (s - a)};
}

inline Twice exact_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}

inline Twice operator+(Twice a, Twice b) {
  Twice s = exact_sum(a.hi, b.hi);
  const Twice t = exact_sum(a.lo, b.lo);
  s = quick_sum(s.hi, s.lo + t.hi);
  return quick_sum(s.hi, s.lo + t.lo);
}

inline Twice operator-(Twice a) { return {-a.hi, -a.lo}; }
inline Twice operator-(Twice a, Twice b) { return a + -b; }

inline Twice operator*(Twice a, Twice b) {
  const double p = a.hi * b.hi;
  return quick_sum(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}

// Digit by digit, a double each.
inline Twice operator/(Twice a, Twice b) {
  const double q0 = a.hi / b.hi;
  a = a - b * q0;
  const double q1 = a.hi / b.hi;
  a = a - b * q1;
  return quick_sum(q0, q1) + Twice(a.hi / b.hi);
}

inline Twice times_two_to(Twice a, int n) { return {std::ldexp(a.hi, n), std::ldexp(a.lo, n)}; }

constexpr Twice kLogOfTwo(0.693147180559945309417232, 2.31904681384629955842e-17);
constexpr Twice kTau(6.28318530717958647692529, 2.44929359829470635445e-16);

// e^x = 2^n (e^r)^64, r = (x - n log 2) / 64 up to 0.0055: eleven terms of its series leave 2^-119.
inline Twice exp_of(Twice x) {
  const double n = std::nearbyint(x.hi / kLogOfTwo.hi);
  const Twice r = times_two_to(x - kLogOfTwo * n, -6);
  Twice y = 1.0;
  for (int k = 11; k >= 1; --k) y = Twice(1.0) + y * r / Twice(k);
  for (int k = 0; k < 6; ++k) y = y * y;
  return times_two_to(y, static_cast<int>(n));
}

// log x = n log 2 + log m, m in [1/2, 1): one of Newton's steps from a double's logarithm of m, with its second term.
inline Twice log_of(double x) {
  int n = 0;
  const double m = std::frexp(x, &n), y = std::log(m);
  const Twice d = Twice(m) * exp_of(-y) - 1.0;
  return kLogOfTwo * static_cast<double>(n) + (Twice(y) + d - times_two_to(d * d, -1));
}

}  // namespace moe
