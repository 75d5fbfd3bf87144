// quant.cuh -- rounding of rows to block formats, eight consecutive elements a
// thread and four neighbouring lanes a block of 32.
#pragma once

#include "kv_common.cuh"

namespace qmm {

constexpr int kQuantN = 8;

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// a / 127 rounded once, for 0 <= a < 2^128 away from subnormal quotients (which
// f16 rounds to 0): the product with the rounded reciprocal, corrected once by
// its exact remainder (Markstein's scheme).
__device__ __forceinline__ float over_127(float a) {
    constexpr float r = 1.f / 127.f;
    const float q = a * r;
    return fmaf(fmaf(-q, 127.f, a), r, q);
}

// Q8_0: d = f16(max |x| / 127), code = rint(x / d) in [-127, 127], each division
// rounded once; a block of zeros (or whose d underflows) has d = 0 and codes
// 0. A block that holds an Inf or NaN, or whose d overflows f16, gets d = NaN
// and reads back as NaN, so that a bad activation stays visible.
//
// x / d is first taken as x * (1 / d), off by less than 2^-15 at |x / d| <= 128:
// only quotients that near to half an integer can round the other way, and
// only lanes that hold one divide (once in some thousand values). Adding 1.5 *
// 2^23 rounds to an integer and leaves its low byte in the low byte.
__device__ __forceinline__ void quant8(const float (&x)[kQuantN], uint2& codes, __half& d) {
    float amax = fabsf(x[0]);
#pragma unroll
    for (int j = 1; j < kQuantN; ++j) amax = max_nan(amax, fabsf(x[j]));
    amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    d = __float2half_rn(over_127(amax));
    const float df = __half2float(d);
    if (!(df < INFINITY)) d = __ushort_as_half(0x7fff);
    codes = make_uint2(0u, 0u);
    if (!(df > 0.f && df < INFINITY)) return;
    constexpr float kRound = 12582912.f;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(df));
    float q[kQuantN];
    float off = 0.f;                     // the largest distance of a quotient from its integer
#pragma unroll
    for (int j = 0; j < kQuantN; j += 2) {
        const float2 v = make_float2(x[j], x[j + 1]), rr = make_float2(r, r);
        const float2 n = fma2(v, rr, make_float2(kRound, kRound));
        const float2 m = fma2(n, make_float2(-1.f, -1.f), make_float2(kRound, kRound));   // minus the integer
        const float2 e = fma2(v, rr, m);
        off = fmaxf(fmaxf(off, fabsf(e.x)), fabsf(e.y));
        q[j] = n.x;
        q[j + 1] = n.y;
    }
    // a subnormal d is coarse: quotients reach 190 and are clamped
    if (off > 0.49996f || df < 6.103515625e-05f) {
#pragma unroll
        for (int j = 0; j < kQuantN; ++j) q[j] = fmaxf(-127.f, fminf(127.f, rintf(__fdiv_rn(x[j], df)))) + kRound;
    }
    unsigned w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const unsigned a = __byte_perm(__float_as_uint(q[4 * k]), __float_as_uint(q[4 * k + 1]), 0x0040);
        const unsigned b = __byte_perm(__float_as_uint(q[4 * k + 2]), __float_as_uint(q[4 * k + 3]), 0x0040);
        w[k] = __byte_perm(a, b, 0x5410);
    }
    codes = make_uint2(w[0], w[1]);
}

// Q4_0: d = f16(m / -8) for the value m of largest magnitude (the first of them),
// code = rint(x / d) in [-8, 7], each division rounded once; d = 0 gives codes 0,
// bad blocks d = NaN as above. Bits 4 j .. 4 j + 3 of `codes` are element j's
// code plus 8. Magnitudes are compared as integers, in which NaN is the largest.
// Quotients go the same way as above: |x / d| <= 12 is off by less than 2^-18.
__device__ __forceinline__ void quant4(const float (&x)[kQuantN], unsigned& codes, __half& d) {
    unsigned most = __float_as_uint(x[0]) & 0x7fffffffu;
    float m = x[0];
#pragma unroll
    for (int j = 1; j < kQuantN; ++j) {
        const unsigned b = __float_as_uint(x[j]) & 0x7fffffffu;
        m = b > most ? x[j] : m;
        most = max(most, b);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {                    // of equal ones the lower lane's
        const float other = __shfl_xor_sync(0xffffffffu, m, o);
        const unsigned b = __float_as_uint(other) & 0x7fffffffu;
        const bool take = b > most || (b == most && (threadIdx.x & o));
        m = take ? other : m;
        most = max(most, b);
    }
    d = __float2half_rn(m * -0.125f);
    const float df = __half2float(d);
    if (!(fabsf(df) < INFINITY)) d = __ushort_as_half(0x7fff);
    codes = 0x88888888u;
    if (!(fabsf(df) > 0.f && fabsf(df) < INFINITY)) return;
    constexpr float kRound = 12582912.f;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(df));
    float q[kQuantN];
    float off = 0.f;
#pragma unroll
    for (int j = 0; j < kQuantN; j += 2) {
        const float2 v = make_float2(x[j], x[j + 1]), rr = make_float2(r, r);
        const float2 n = fma2(v, rr, make_float2(kRound, kRound));
        const float2 k = fma2(n, make_float2(-1.f, -1.f), make_float2(kRound, kRound));   // minus the integer
        const float2 e = fma2(v, rr, k);
        off = fmaxf(fmaxf(off, fabsf(e.x)), fabsf(e.y));
        q[j] = n.x;
        q[j + 1] = n.y;
    }
    if (off > 0.49999f) {
#pragma unroll
        for (int j = 0; j < kQuantN; ++j) q[j] = rintf(__fdiv_rn(x[j], df)) + kRound;
    }
    codes = 0u;
#pragma unroll
    for (int j = 0; j < kQuantN; ++j) {
        const float c = fminf(fmaxf(q[j], kRound - 8.f), kRound + 7.f);
        codes |= ((__float_as_uint(c) + 8u) & 15u) << (4 * j);
    }
}

}  // namespace qmm
