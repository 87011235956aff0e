// divisor.cuh -- division by a number that the host knows, without a division
// on the device: a kernel's start may have several in a row (without them a
// decode over 777 cached tokens fell from 7.2 to 6.8 us, rotary positions of 16
// tokens from 2.16 to 2.07).
#pragma once

namespace tq {

// Division of whole numbers below 2^31 by d: with 2^(l-1) < d <= 2^l and
// m = ceil(2^(31+l) / d), m d exceeds 2^(31+l) by less than 2^l, so that
// x m / 2^(31+l) is above x / d by less than 1 / d.
struct Divisor {
    unsigned m;
    int shift;

    Divisor() = default;
    explicit Divisor(int d) : m(0), shift(31)
    {
        while ((1ll << (shift - 31)) < d)
            ++shift;
        m = unsigned(((1ull << shift) + unsigned(d) - 1) / unsigned(d));
    }
    __device__ __forceinline__ int of(int x) const
    {
        return int((unsigned long long)unsigned(x) * m >> shift);
    }
};

}  // namespace tq
