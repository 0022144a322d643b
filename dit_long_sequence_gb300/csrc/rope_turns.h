// rope_turns.h -- host-only: a rotary frequency as a fraction of a turn.  Used
// by api_train.cu.
#pragma once

#include <cstdint>
#include <cstring>

namespace dit {

// 2^64 (w / 2 pi mod 1), rounded to the nearest: w's 53 bits times the first 128
// binary digits of 1 / 2 pi, in integers.  (The quotient in doubles is off by up
// to 2^-53 of itself, which a position of 2^40 multiplies to 10^-4 of a turn.)
// Good to the last bit for |w| < 2^60.
inline uint64_t turns_per_step(double w) {
    using u128 = unsigned __int128;
    constexpr uint64_t kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;
    uint64_t as_bits;
    std::memcpy(&as_bits, &w, sizeof w);
    const int biased = static_cast<int>(as_bits >> 52) & 0x7ff, e = (biased > 0 ? biased : 1) - 1075;
    const uint64_t m = (as_bits & 0xfffffffffffffull) | (biased > 0 ? uint64_t(1) << 52 : 0);    // |w| = m 2^e
    const u128 low = static_cast<u128>(m) * kLow, high = static_cast<u128>(m) * kHigh + (low >> 64);
    const uint64_t lowest = static_cast<uint64_t>(low);                          // |w| / 2 pi = (high 2^64 + lowest) 2^(e - 128)
    auto bits_from = [&](int at) -> uint64_t {                                   // 64 bits of that integer
        if (at >= 192 || at <= -64) return 0;
        if (at >= 64) return static_cast<uint64_t>(high >> (at - 64));
        if (at > 0) return static_cast<uint64_t>(high << (64 - at)) | (lowest >> at);
        return lowest << -at;
    };
    const int at = 64 - e;
    const uint64_t t = bits_from(at) + (bits_from(at - 1) & 1u);
    return w < 0.0 ? 0u - t : t;
}

}  // namespace dit
