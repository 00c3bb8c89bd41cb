// exp64.hpp -- 2^t in 64 bits on the device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

// t = n + f with n the nearest whole number, and 2^f = sum of (f ln 2)^k / k! up to
// k = 11, whose remainder at |f| = 1/2 is 6.3e-15 relative.  Below -1100 it is 0, above
// 1100 infinite; a NaN counts as -1100.
__device__ __forceinline__ double exp2_64(double t) {
    t = __builtin_fmin(__builtin_fmax(t, -1100.0), 1100.0);
    const double n = __builtin_rint(t), f = t - n;
    double p = 4.4455382718708116e-10;
    p = __builtin_fma(p, f, 7.054911620801123e-09);
    p = __builtin_fma(p, f, 1.01780860092397e-07);
    p = __builtin_fma(p, f, 1.321548679014431e-06);
    p = __builtin_fma(p, f, 1.5252733804059841e-05);
    p = __builtin_fma(p, f, 0.0001540353039338161);
    p = __builtin_fma(p, f, 0.0013333558146428443);
    p = __builtin_fma(p, f, 0.009618129107628477);
    p = __builtin_fma(p, f, 0.05550410866482158);
    p = __builtin_fma(p, f, 0.24022650695910072);
    p = __builtin_fma(p, f, 0.6931471805599453);
    p = __builtin_fma(p, f, 1.0);
    return __builtin_ldexp(p, (int)n);
}
// 2^(d rate) for |d rate| up to 1021 in fewer instructions, none of them a conversion.
__device__ __forceinline__ double exp2_64_within(double d, double rate) {
    // the nearest whole number in the last bits of the sum with 3 * 2^51
    const double shifted = __builtin_fma(d, rate, 0x1.8p52);
    const double f = __builtin_fma(d, rate, -(shifted - 0x1.8p52));
    double p = 4.4455382718708116e-10;
    p = __builtin_fma(p, f, 7.054911620801123e-09);
    p = __builtin_fma(p, f, 1.01780860092397e-07);
    p = __builtin_fma(p, f, 1.321548679014431e-06);
    p = __builtin_fma(p, f, 1.5252733804059841e-05);
    p = __builtin_fma(p, f, 0.0001540353039338161);
    p = __builtin_fma(p, f, 0.0013333558146428443);
    p = __builtin_fma(p, f, 0.009618129107628477);
    p = __builtin_fma(p, f, 0.05550410866482158);
    p = __builtin_fma(p, f, 0.24022650695910072);
    p = __builtin_fma(p, f, 0.6931471805599453);
    p = __builtin_fma(p, f, 1.0);
    // 2^n times p, which lies in 0.7 .. 1.5
    const uint64_t n = (uint64_t)(uint32_t)__double2loint(shifted) << 52;
    return __longlong_as_double((long long)((uint64_t)__double_as_longlong(p) + n));
}
// The same for d up to 0; `least` = -1000 / rate, and below it the result is 2^-1000.
__device__ __forceinline__ double exp2_64_low(double d, double rate, double least) {
    return exp2_64_within(__builtin_fmax(d, least), rate);
}
constexpr double kLog2E = 1.4426950408889634;
