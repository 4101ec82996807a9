// Division by a number that the host knows, as a multiply-high, an add and a shift. Plain C++ (host and device), shared by
// the kernels and a CPU test.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define DIVIDE_HD __host__ __device__ __forceinline__
#else
#define DIVIDE_HD inline
#endif

namespace alibi {

// For d >= 1 and 0 <= n < 2^31 (Granlund and Montgomery, "Division by invariant integers using multiplication", PLDI 1994):
// with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d = (high word of n m + n) >> l. The kernels decode
// their work items with it, where a plain integer division is a long dependent sequence.
struct Divisor {
    uint32_t d, m, l;

    Divisor() = default;
    explicit Divisor(uint32_t d_) : d(d_), l(0)
    {
        while ((1ull << l) < d) ++l;
        m = static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - d)) / d + 1);
    }
    DIVIDE_HD int of(int n) const
    {
        const uint32_t u = static_cast<uint32_t>(n);
        return static_cast<int>((static_cast<uint32_t>(static_cast<uint64_t>(u) * m >> 32) + u) >> l);
    }
    DIVIDE_HD int rest(int n) const { return n - of(n) * static_cast<int>(d); }
};

}  // namespace alibi
