// Division of numbers below 2^31 by one that the host knows, by one high product.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nrc {

struct Div {
    uint32_t mul, shift;  // mul 0: by 1
};
inline Div div_by(uint32_t d) {
    if (d <= 1) return Div{0, 0};
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return Div{(uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d), s - 1};
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, Div d) { return d.mul ? __umulhi(n, d.mul) >> d.shift : n; }

}  // namespace nrc
