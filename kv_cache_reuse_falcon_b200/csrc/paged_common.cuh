// What the paged pool's kernels share.
#pragma once

#include <cstdint>

namespace unipin {

// Division by a number that is the same for the whole launch (rows of a page, vectors of a token):
// j / d = umulhi(j, mul) >> shift for 0 <= j < 2^31 and d >= 2; mul = 0: d = 1.  With s = ceil(log2 d) and
// mul = floor(2^(31 + s) / d) + 1 <= 2^32 - 1 the product exceeds 2^(31 + s) j / d by at most
// j < 2^31 <= 2^(31 + s) / d, too little to reach the next quotient.
struct PgDiv {
    uint32_t mul;
    int shift;
    __device__ __forceinline__ int operator()(int j) const
    {
        return mul ? (int)(__umulhi((uint32_t)j, mul) >> shift) : j;
    }
};

inline PgDiv pg_divisor(int d)
{
    if (d < 2) return {0u, 0};
    int s = 0;
    while ((1ll << s) < d) ++s;
    return {(uint32_t)((1ull << (31 + s)) / (uint64_t)d + 1), s - 1};
}

}  // namespace unipin
