// The turns of a rotation's pairs from one position to the next, on the host
// (gpt2_rotary_turns): f_j = base^(-2 j / rot) / (2 pi), stretched, as whole
// numbers of 2^-64 turns.
//
// A position of 31 bits multiplies a table's error by up to 2^31, so the table
// is right to its last bit: numbers are sums of two doubles (Dekker 1971: about
// 106 bits), the exponential is a Taylor series of an argument reduced by ln 2
// and 2^9, squared back, and the logarithm a Newton step on the library's. A
// double's 53 bits leave 2^-56 of a turn, 2^-25 of one at the furthest position.
#include "common.cuh"
#include "launch.h"

#include <cmath>

namespace {

struct Two {
    double h, l;  // the value h + l, |l| at most half a unit of h's last place
};
constexpr Two LN2 = {0x1.62e42fefa39efp-1, 0x1.abc9e3b39803fp-56};
constexpr Two PER_RADIAN = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / (2 pi)

Two sum_of(double a, double b) {
    const double s = a + b, bb = s - a;
    return {s, (a - (s - bb)) + (b - bb)};
}
Two settled(double h, double l) {  // |l| <= |h|
    const double s = h + l;
    return {s, l - (s - h)};
}
Two operator+(Two x, Two y) {
    const Two s = sum_of(x.h, y.h), t = sum_of(x.l, y.l), u = settled(s.h, s.l + t.h);
    return settled(u.h, u.l + t.l);
}
Two operator*(Two x, Two y) {
    const double p = x.h * y.h;
    return settled(p, std::fma(x.h, y.h, -p) + (x.h * y.l + x.l * y.h));
}
Two operator-(Two x) { return {-x.h, -x.l}; }
Two operator/(Two x, Two y) {
    Two q = {0.0, 0.0};
    for (int i = 0; i < 3; i++) {
        const Two d = {x.h / y.h, 0.0};
        q = q + d;
        x = x + -(d * y);
    }
    return q;
}

Two exp_of(Two x) {
    const double k = std::nearbyint(x.h / LN2.h);
    Two r = x + -(Two{k, 0.0} * LN2);
    r = {std::ldexp(r.h, -9), std::ldexp(r.l, -9)};
    Two e = {1.0, 0.0};  // e^r - 1 = r (1 + r / 2 (1 + r / 3 (..))), |r| < 2^-10: 12 terms leave 2^-140
    for (int i = 12; i > 1; i--) e = Two{1.0, 0.0} + e * r / Two{(double)i, 0.0};
    e = e * r;
    for (int i = 0; i < 9; i++) e = Two{2 * e.h, 2 * e.l} + e * e;
    e = e + Two{1.0, 0.0};
    return {std::ldexp(e.h, (int)k), std::ldexp(e.l, (int)k)};
}
Two log_of(double b) {
    int e;
    const double m = std::frexp(b, &e), y = std::log(m);
    const Two t = exp_of({-y, 0.0}) * Two{m, 0.0} + Two{-1.0, 0.0};  // m = e^y (1 + t)
    return Two{y, 0.0} + t + -(t * t * Two{0.5, 0.0}) + Two{(double)e, 0.0} * LN2;
}

}  // namespace

void rotary_turns(uint64_t* turns, int rot, double base, int scaling, double factor, double context, double fast,
                  double slow) {
    Two log = log_of(base);
    if (scaling == GPT2_ROTARY_BASE && rot > 2)
        log = log + log_of(factor) * Two{(double)rot, 0.0} / Two{rot - 2.0, 0.0};
    for (int j = 0; j < rot / 2; j++) {
        Two f = exp_of(log * Two{-2.0 * j, 0.0} / Two{(double)rot, 0.0}) * PER_RADIAN;
        if (scaling == GPT2_ROTARY_LINEAR) f = f / Two{factor, 0.0};
        if (scaling == GPT2_ROTARY_PARTS) {
            const Two turned = (f * Two{context, 0.0} + Two{-slow, 0.0}) / sum_of(fast, -slow), one = {1.0, 0.0};
            // (a quotient past a double's range is no number here, and above 1)
            const Two keep = !(turned.h < 1.0) ? one : turned.h <= 0.0 ? Two{0.0, 0.0} : turned;
            if (keep.h < 1.0) f = f * (keep + (one + -keep) / Two{factor, 0.0});
        }
        const double h = std::ldexp(f.h, 64), whole = std::floor(h), rest = (h - whole) + std::ldexp(f.l, 64);
        turns[j] = (uint64_t)whole + (uint64_t)(int64_t)std::floor(rest + 0.5);
    }
}
