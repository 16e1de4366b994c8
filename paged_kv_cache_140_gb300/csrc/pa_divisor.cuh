// Division by a number that the host knows, as a product.
#pragma once

#include <stdint.h>

namespace pa {

// x / by for x below 2^31: x mul 2^-(31 + shift) rounded down, mul = ceil(2^(31 + shift) / by).
struct Divisor {
    uint32_t mul, shift, by;
};
inline Divisor divisor(uint32_t by) {
    uint32_t k = 0;
    while ((uint64_t{1} << k) < by) ++k;
    // 2^k < 2 by, so that mul fits 32 bits; it is too large by less than 2^k 2^-(31 + k) of itself
    return {static_cast<uint32_t>(((uint64_t{1} << (31 + k)) + by - 1) / by), k, by};
}
__device__ __forceinline__ uint32_t divided(uint32_t x, const Divisor &d) {
    return static_cast<uint32_t>((static_cast<uint64_t>(x) * d.mul) >> (31 + d.shift));
}

}  // namespace pa
