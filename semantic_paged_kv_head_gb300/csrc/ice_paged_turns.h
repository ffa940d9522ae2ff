// A frequency of the rotary positions as a fraction of a turn. Plain arithmetic, so that it also compiles and is tested on
// the host.
#pragma once

#include <cmath>

namespace ice {

// f 2^64 / 2 pi modulo 2^64, to the nearest for |f| up to 2^32 (|f| 2^-45 units more at most). A quotient in 53 bits would be off by up
// to 2^-23 turns at a position of 2^31, so what the division cuts off is added; whole turns are dropped from both, exactly.
inline unsigned long long turns(double f) {
    const double c = 6.283185307179586, c_lo = 2.4492935982947064e-16;  // 2 pi to 106 bits
    const double t = f / c, rest = (std::fma(-t, c, f) - t * c_lo) / c;
    const double units = std::ldexp(std::fmod(t, 1.0), 64), whole = std::trunc(units);
    const double part = std::nearbyint(std::ldexp(std::fmod(rest, 1.0), 64) + (units - whole));
    auto bits = [](double x) {  // of a whole number below 2^64
        const unsigned long long b = (unsigned long long)std::fabs(x);
        return x < 0.0 ? 0ull - b : b;
    };
    return bits(whole) + bits(part);
}

}  // namespace ice
