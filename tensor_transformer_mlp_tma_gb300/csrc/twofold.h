// Host arithmetic on numbers of two doubles, hi + lo with |lo| at most half a unit in the last place of hi: sums and products
// by Dekker's and Knuth's error terms, to about 2^-100.  For what a double is too short for: a position times a frequency,
// modulo a turn.
#pragma once

#include <cmath>

namespace tpmlp {

struct Twofold {
    double hi, lo;
};

inline Twofold two_sum(double a, double b) {
    const double s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
inline Twofold normal(double hi, double lo) {  // |hi| >= |lo|
    const double s = hi + lo;
    return {s, lo - (s - hi)};
}
inline Twofold operator+(Twofold a, Twofold b) {
    const Twofold s = two_sum(a.hi, b.hi), t = two_sum(a.lo, b.lo);
    const Twofold r = normal(s.hi, s.lo + t.hi);
    return normal(r.hi, r.lo + t.lo);
}
inline Twofold operator-(Twofold a) { return {-a.hi, -a.lo}; }
inline Twofold operator*(Twofold a, Twofold b) {
    const double p = a.hi * b.hi, e = std::fma(a.hi, b.hi, -p);
    return normal(p, e + (a.hi * b.lo + a.lo * b.hi));
}
inline Twofold operator/(Twofold a, Twofold b) {
    // two corrections of the quotient of the leading parts
    const double q0 = a.hi / b.hi;
    const Twofold r0 = a + -(b * Twofold{q0, 0.0});
    const double q1 = r0.hi / b.hi;
    const Twofold r1 = r0 + -(b * Twofold{q1, 0.0});
    return normal(q0, q1) + Twofold{r1.hi / b.hi, 0.0};
}
inline bool operator<(Twofold a, Twofold b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }

// e^x for |x| up to 745: the series at x / 2^20 (below 2^-10, so 12 terms are more than enough), squared 20 times, which
// costs 20 of the 100 bits.
inline Twofold exp_of(Twofold x) {
    const Twofold r = {std::ldexp(x.hi, -20), std::ldexp(x.lo, -20)};
    Twofold sum = {1.0, 0.0};
    for (int n = 12; n > 0; --n) sum = Twofold{1.0, 0.0} + r * sum / Twofold{static_cast<double>(n), 0.0};
    for (int i = 0; i < 20; ++i) sum = sum * sum;
    return sum;
}
// The double's logarithm and one step of Newton's method: x e^-y = 1 + d (in two halves, so that e^-y does not underflow).
inline Twofold log_of(double x) {
    const double y = std::log(x);
    const Twofold half = exp_of({-0.5 * y, 0.0}), d = Twofold{x, 0.0} * half * half + Twofold{-1.0, 0.0};
    return Twofold{y, 0.0} + d;
}
// pi: the sine of its leading part is what is missing, up to the cube of that.
inline Twofold pi_of() {
    const double p = std::acos(-1.0);
    return normal(p, std::sin(p));
}

}  // namespace tpmlp
