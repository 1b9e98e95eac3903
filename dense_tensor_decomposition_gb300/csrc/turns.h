// Radians as turns in 64-bit fixed point (host).
#pragma once

#include <cstdint>
#include <cstring>

namespace mk {

constexpr double kMostRadians = 18446744073709551616.0;        // 2^64

// `radians`, of a magnitude below 2^64, in units of 2^-64 turn, modulo a turn, to the nearest: off by 2^-65
// turn at most, whatever their size.  (A quotient in double is off by 2^-53 of itself, which a position
// of 2^40 makes 1e-4 radians.)  The product of the 53 bits with 1 / 2 pi = kInverse 2^-192, and the 64 bits of
// it that lie behind the point.
inline uint64_t turns_of(double radians) {
    constexpr uint64_t kInverse[3] = {0x36d8a5664f10e410u, 0x7f09d5f47d4d3770u, 0x28be60db9391054au};
    // |radians| = bits 2^exponent (read from the number itself: a call makes up to 512 of these)
    uint64_t number;
    std::memcpy(&number, &radians, sizeof(number));
    const int field = (int)(number >> 52) & 0x7FF;
    const uint64_t bits = (number & 0xFFFFFFFFFFFFFu) | (field != 0 ? (uint64_t)1 << 52 : 0);
    const int exponent = (field != 0 ? field : 1) - 1075;
    const int shift = 128 - exponent;               // of the product, to units of 2^-64: 117 at least
    uint64_t product[4];
    unsigned __int128 carry = 0;
    for (int i = 0; i < 3; ++i) {
        carry += (unsigned __int128)bits * kInverse[i];
        product[i] = (uint64_t)carry;
        carry >>= 64;
    }
    product[3] = (uint64_t)carry;
    if (shift > 256) return 0;                      // below half a unit
    auto from = [&](int at) {                       // 64 bits of the product from bit `at` on
        const int word = at / 64, bit = at % 64;
        const uint64_t low = word < 4 ? product[word] >> bit : 0;
        return bit == 0 || word + 1 >= 4 ? low : low | product[word + 1] << (64 - bit);
    };
    const uint64_t turns = from(shift) + (from(shift - 1) & 1);
    return radians < 0.0 ? 0 - turns : turns;
}

}  // namespace mk
