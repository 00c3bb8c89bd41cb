// exp64.hpp -- 2^t in 64 bits on the device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

// 2^f for |f| up to 1/2: the polynomial of degree 9 that meets it at nine of the ten
// Chebyshev points of that interval and, instead of the least positive one, at 0 (computed
// to 50 digits), off by less than 2.8e-14 relative.  2^0 is exactly 1, so that a sigmoid of 0
// is 1/2 and ranks that are alike by it stay so (at all ten points it is off by less than
// 1.9e-14, but by 1.4e-14 at 0).
__device__ __forceinline__ double exp2_fraction(double f) {
    double p = 1.015059818177267e-07;
    p = __builtin_fma(p, f, 1.3259212647024628e-06);
    p = __builtin_fma(p, f, 1.5253015211389932e-05);
    p = __builtin_fma(p, f, 0.00015403436428521592);
    p = __builtin_fma(p, f, 0.0013333557465581899);
    p = __builtin_fma(p, f, 0.009618129188183683);
    p = __builtin_fma(p, f, 0.05550410867095325);
    p = __builtin_fma(p, f, 0.2402265069568963);
    p = __builtin_fma(p, f, 0.6931471805597738);
    return __builtin_fma(p, f, 1.0);
}

// 2^(d rate) for |d rate| up to 1021, without an instruction that converts.
__device__ __forceinline__ double exp2_64_within(double d, double rate) {
    // the nearest whole number in the last bits of the sum with 3 * 2^51
    const double shifted = __builtin_fma(d, rate, 0x1.8p52);
    const double p = exp2_fraction(__builtin_fma(d, rate, -(shifted - 0x1.8p52)));
    // 2^n times p, which lies in 0.7 .. 1.5
    const uint32_t n = (uint32_t)__double2loint(shifted);
    return __hiloint2double((int)((n << 20) + (uint32_t)__double2hiint(p)), __double2loint(p));
}
// The same for d up to 0; `least` = -1000 / rate, and below it the result is 2^-1000.
__device__ __forceinline__ double exp2_64_low(double d, double rate, double least) {
    return exp2_64_within(__builtin_fmax(d, least), rate);
}
constexpr double kLog2E = 1.4426950408889634;
