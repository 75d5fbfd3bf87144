// exp64.cuh -- a short exponential and inverse in 64 bits, for kernels that need few of them
// and then wait for the code of the library's.
#pragma once

namespace qmm {

// e^x to 2 ulp for |x| <= 700: x = k ln 2 + r with ln 2 in two parts (Cody and Waite),
// e^r by its Taylor sum to r^13 / 13! (|r| <= 0.35: the next term is 5e-18).
__device__ __forceinline__ double exp_mid(double x) {
    const double k = rint(x * 1.4426950408889634);
    double r = fma(k, -0.6931471805592082, x);                 // ln 2 cut off to 40 bits: k times it is exact
    r = fma(k, -7.371002565167799e-13, r);                     // the rest of it
    const double r2 = r * r, r4 = r2 * r2;
    const double p0 = fma(r, 1.0, 1.0), p1 = fma(r, 1.0 / 6, 0.5), p2 = fma(r, 1.0 / 120, 1.0 / 24), p3 = fma(r, 1.0 / 5040, 1.0 / 720);
    const double p4 = fma(r, 1.0 / 362880, 1.0 / 40320), p5 = fma(r, 1.0 / 39916800, 1.0 / 3628800);
    const double p6 = fma(r, 1.0 / 6227020800.0, 1.0 / 479001600);
    const double q0 = fma(p1, r2, p0), q1 = fma(p3, r2, p2), q2 = fma(p5, r2, p4);
    const double e = fma(fma(fma(p6, r4, q2), r4, q1), r4, q0);
    return __hiloint2double(__double2hiint(e) + (static_cast<int>(k) << 20), __double2loint(e));
}
// 1 / d to 1 ulp for 1 <= d <= 2^126: Newton's steps from an fp32 quotient.
__device__ __forceinline__ double inverse(double d) {
    double y = static_cast<double>(__fdividef(1.f, static_cast<float>(d)));
    y = fma(y, fma(-d, y, 1.0), y);
    return fma(y, fma(-d, y, 1.0), y);
}

}  // namespace qmm
