// A frequency as a fraction of a turn, for the rotation of rows by their positions. Plain C++, so that a CPU test can check it.
#pragma once

#include <cmath>
#include <cstdint>

namespace alibi {

// f / 2 pi modulo 1 in units of 2^-64, off by at most two units, for |f| < 2^31 (radians per token). n times it modulo 2^64 is the
// fraction of a turn that position n leaves, off by 2 n units: 2^-39 of a turn at position 2^24, whatever f is. In whole numbers:
// the quotient in double is off by 2^-53 of itself, and n times that is 2^-11 of a turn at f = 1e6.
inline uint64_t turns_of(double f)
{
    // floor(2^128 / 2 pi), in two words
    constexpr uint64_t kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;
    int e;
    const uint64_t m = static_cast<uint64_t>(std::ldexp(std::frexp(std::fabs(f), &e), 53));  // |f| = m 2^(e - 53)
    const int down = 53 - e;                                                                 // above 21
    using Wide = unsigned __int128;
    const Wide product = static_cast<Wide>(m) * kHigh + (static_cast<Wide>(m) * kLow >> 64);  // m 2^64 / 2 pi
    const uint64_t turns = down < 128 ? static_cast<uint64_t>(product >> down) : 0;
    return f < 0 ? 0 - turns : turns;
}

}  // namespace alibi
