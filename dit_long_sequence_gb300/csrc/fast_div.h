// fast_div.h -- division by a fixed number through one multiply.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define DIT_HD __host__ __device__ __forceinline__
#else
#define DIT_HD inline
#endif

namespace dit {

// n / d and n % d for 0 <= n < 2^31 and a fixed 1 <= d < 2^31 by one multiply:
// with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1,
// n / d = (umulhi(n, m) + n) >> s: the round-up reciprocal of Granlund and
// Montgomery, "Division by invariant integers using multiplication" (1994); the
// sum stays below 2^32 because umulhi(n, m) <= n < 2^31.
struct FastDiv {
    uint32_t d, m, s;
    FastDiv() : d(1), m(1), s(0) {}
    explicit FastDiv(uint32_t div) : d(div), s(0) {
        while ((uint64_t(1) << s) < d) ++s;
        m = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1);
    }
    DIT_HD uint32_t div(uint32_t n) const {
#ifdef __CUDA_ARCH__
        return (__umulhi(n, m) + n) >> s;
#else
        return (static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> 32) + n) >> s;
#endif
    }
    DIT_HD uint32_t divmod(uint32_t n, uint32_t& rem) const {
        const uint32_t q = div(n);
        rem = n - q * d;
        return q;
    }
};

}  // namespace dit
