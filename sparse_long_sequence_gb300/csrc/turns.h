// The rotation's turns per position, theta^(-2i/rot) / (2 pi), as 128-bit fractions of a turn,
// on the host.
//
// The ratio x = theta^(-1/m) of neighbouring pairs (m = rot / 2) starts as a double and takes
// one step of Newton's kind on x^m theta = 1 + d with 128-bit mantissas:
//   x (1 + d)^(-1/m) = x (1 - d/m + (m + 1) d^2 / (2 m^2) - ...),  |d| < 2^-46,
// the next term below 2^-140.  The powers cost at most 2^-121 of d, so the ratio is good to
// 2^-125 and pair i's fraction, i products on, to 2^-120 of itself: a position p is off by
// at most |p| 2^-123 turns, 2^-60 for the farthest 64-bit one.  Integers all the way, so that
// machines whose long double differs agree.
#pragma once

#include <cmath>
#include <cstdint>

namespace dfs {
namespace turns {

typedef unsigned __int128 u128;

// mant 2^exp, mant in [2^127, 2^128)
struct Wide {
    u128 mant;
    int exp;
};

// rounded down by less than 2 units of the last place
inline Wide mul(const Wide& a, const Wide& b) {
    const uint64_t ah = (uint64_t)(a.mant >> 64), al = (uint64_t)a.mant, bh = (uint64_t)(b.mant >> 64), bl = (uint64_t)b.mant;
    const u128 lo = (u128)al * bl, m1 = (u128)ah * bl, m2 = (u128)al * bh;
    const u128 mid = (lo >> 64) + (uint64_t)m1 + (uint64_t)m2;
    const u128 top = (u128)ah * bh + (m1 >> 64) + (m2 >> 64) + (mid >> 64);
    if (top >> 127) return {top, a.exp + b.exp + 128};
    return {(top << 1) | ((uint64_t)mid >> 63), a.exp + b.exp + 127};
}
inline Wide wide(double x) {                 // x > 0
    int e;
    const uint64_t m = (uint64_t)std::ldexp(std::frexp(x, &e), 53);
    return {(u128)m << 75, e - 128};
}
inline Wide power(Wide x, int m) {           // m = 8, 16, 24, 32
    int n = m;
    if (m == 24) {
        x = mul(mul(x, x), x);
        n = 8;
    }
    for (; n > 1; n /= 2) x = mul(x, x);
    return x;
}
inline Wide ratio(double theta, int m) {
    const Wide x = wide(std::pow(theta, -1.0 / m)), q = mul(power(x, m), wide(theta));
    const u128 one = (u128)1 << 127;         // 1 in units of 2^-127
    // q lies within 2^-46 of 1: its last bit is 2^-127 or 2^-128
    const __int128 d = (__int128)((q.exp == -127 ? q.mant : q.mant >> 1) - one);
    const double small = std::ldexp((double)d, -127);
    const __int128 c = (__int128)std::ldexp((m + 1) / (2.0 * m * m) * small * small, 127) - d / m;
    const u128 f = one + (u128)c;
    return mul(x, c >= 0 ? Wide{f, -127} : Wide{f << 1, -128});
}

// theta >= 1 and finite, rot 16, 32, 48 or 64: rot / 2 fractions, their upper and lower 64 bits
inline void fill(uint64_t* hi, uint64_t* lo, double theta, int rot) {
    const int m = rot / 2;
    const Wide x = ratio(theta, m);
    Wide f = {((u128)0xa2f9836e4e441529ull << 64) | 0xfc2757d1f534ddc1ull, -130};      // 1 / (2 pi)
    for (int i = 0; i < m; ++i) {
        const int down = -128 - f.exp;       // 2 or more
        const u128 t = down < 128 ? f.mant >> down : 0;
        hi[i] = (uint64_t)(t >> 64);
        lo[i] = (uint64_t)t;
        if (i + 1 < m) f = mul(f, x);
    }
}

}  // namespace turns
}  // namespace dfs
