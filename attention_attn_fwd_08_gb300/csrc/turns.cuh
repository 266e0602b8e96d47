// turns.cuh -- angles of rotary positions as fractions of a turn in 64-bit fixed point: the
// frequency of a pair is held as the fraction of a turn that it adds from one position to the
// next, in units of 2^-64 turns, and its product with the position modulo 2^64 is the angle's
// fraction of a turn, right to p * 2^-64 at position p (a rounding to half a unit, and less than another
// quarter from the arithmetic before it).
#pragma once

#include <math.h>

#include <cuda_runtime.h>

namespace attn {
namespace {

struct TurnFreqs {
    unsigned long long f[128];  // of pair i, in units of 2^-64 turns
};

// A number to about 2^-104 of itself as an unevaluated sum of two doubles (T. J. Dekker, "A
// floating-point technique for extending the available precision", 1971).  Products that are
// added to are written as fma(a, b, 0), which no compiler joins with the addition.
struct Two {
    double hi, lo;
};
inline Two two_sum(double big, double small) {
    const double s = big + small;
    return {s, small - (s - big)};
}
inline Two two_mul(Two a, Two b) {
    const double p = fma(a.hi, b.hi, 0.0);
    return two_sum(p, fma(a.hi, b.lo, fma(a.lo, b.hi, fma(a.hi, b.hi, -p))));
}
inline Two two_sqrt(Two a) {  // a Newton step from the double's root
    const double x = sqrt(a.hi), p = fma(x, x, 0.0);
    return two_sum(x, ((a.hi - p) - fma(x, x, -p) + a.lo) / (2 * x));
}

constexpr Two kTurnsPerRadian = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / (2 pi)
// the fraction of a turn (at least 0) of `turns` >= 0, below 2^53: rounded once, what the upper part holds
// below 2^-64 together with the lower one
inline unsigned long long turn_fraction(Two turns) {
    const double upper = ldexp(turns.hi - floor(turns.hi), 64), whole = floor(upper);
    return (unsigned long long)whole + (unsigned long long)(long long)rint((upper - whole) + ldexp(turns.lo, 64));
}

// Sine and cosine of p turns of f: the upper 32 bits of the product become an angle in
// [-pi, pi) in fp32 (off by 3e-7 at most, near pi) for the hardware sine and cosine (off by
// 2^-21.4 and 2^-21.2 at most, by their documentation): 2^-20 in all.
__device__ __forceinline__ void turn_sincos(unsigned int p, unsigned long long f, float& s, float& c) {
    const unsigned int fl = (unsigned int)f, fh = (unsigned int)(f >> 32);
    const int frac = (int)(__umulhi(p, fl) + p * fh);      // upper half of p * f mod 2^64
    const float a = (float)frac * 1.46291807926715968e-9f;  // 2 pi / 2^32
    s = __sinf(a);
    c = __cosf(a);
}

}  // namespace
}  // namespace attn
