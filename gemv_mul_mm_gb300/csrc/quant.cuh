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

__device__ __forceinline__ float min_nan(float a, float b) {   // NaN if either is
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Q4_0: d = f16(m / -8) for the value m of largest magnitude (the first of them),
// code = rint(x / d) in [-8, 7], each division rounded once; d = 0 gives codes 0,
// bad blocks d = NaN as above. Bits 4 j .. 4 j + 3 of `codes` are element j's
// code plus 8.
//
// m is the largest or the smallest value; which comes first matters only where they
// are opposite, and is looked up only then. Quotients go the same way as above:
// |x / d| <= 12 is off by less than 2^-18. Away from subnormal d they do not
// pass -8 by more than 2^-8, so that the upper end alone is clamped. Codes are put
// together in fp32, four in a sum below 2^16.
// K vectors at once, whose shuffles overlap. All 32 lanes call it.
template <int K> __device__ __forceinline__ void quant4(const float (&x)[K][kQuantN], unsigned (&codes)[K], __half (&d)[K]) {
    constexpr unsigned kAll = 0xffffffffu;
    float hi[K], lo[K], m[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        hi[k] = lo[k] = x[k][0];
#pragma unroll
        for (int j = 1; j < kQuantN; ++j) {
            hi[k] = max_nan(hi[k], x[k][j]);
            lo[k] = min_nan(lo[k], x[k][j]);
        }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            hi[k] = max_nan(hi[k], __shfl_xor_sync(kAll, hi[k], o));
            lo[k] = min_nan(lo[k], __shfl_xor_sync(kAll, lo[k], o));
        }
    bool tie = false;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        m[k] = hi[k] > -lo[k] ? hi[k] : lo[k];               // (NaN: lo is)
        tie |= hi[k] == -lo[k] && hi[k] > 0.f;
    }
    if (__any_sync(kAll, tie)) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float first = 0.f;                               // of this lane's that have the magnitude
#pragma unroll
            for (int j = kQuantN - 1; j >= 0; --j) first = fabsf(x[k][j]) == hi[k] ? x[k][j] : first;
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {                // the lower lane's before the upper one's
                const float other = __shfl_xor_sync(kAll, first, o);
                const bool upper = threadIdx.x & o;
                const float p = upper ? other : first, q = upper ? first : other;
                first = p != 0.f ? p : q;
            }
            if (hi[k] == -lo[k] && hi[k] > 0.f) m[k] = first;
        }
    }
    constexpr float kInt = 12582912.f;                       // 1.5 2^23: sums with it are integers
    constexpr float kRound = kInt + 8.f;                     // the sum less kInt is the code plus 8
#pragma unroll
    for (int k = 0; k < K; ++k) {
        d[k] = __float2half_rn(m[k] * -0.125f);
        const float df = __half2float(d[k]);
        const bool bad = !(fabsf(df) < INFINITY), zero = df == 0.f;
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(df));
        float2 u[4];                                         // codes plus 8 of elements j and j + 4
        float off = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = make_float2(x[k][j], x[k][j + 4]), rr = make_float2(r, r);
            const float2 n = fma2(v, rr, make_float2(kRound, kRound));
            const float2 i = fma2(n, make_float2(-1.f, -1.f), make_float2(kRound, kRound));   // minus the integer
            const float2 e = fma2(v, rr, i);
            off = fmaxf(fmaxf(off, fabsf(e.x)), fabsf(e.y));
            u[j] = add2(make_float2(fminf(n.x, kRound + 7.f), fminf(n.y, kRound + 7.f)), make_float2(-kInt, -kInt));
        }
        if (off > 0.49999f || fabsf(df) < 6.103515625e-05f) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u[j].x = 8.f + fmaxf(-8.f, fminf(7.f, rintf(__fdiv_rn(x[k][j], df))));
                u[j].y = 8.f + fmaxf(-8.f, fminf(7.f, rintf(__fdiv_rn(x[k][j + 4], df))));
            }
        }
        const float2 by16 = make_float2(16.f, 16.f);
        const float2 w = add2(fma2(fma2(fma2(u[3], by16, u[2]), by16, u[1]), by16, u[0]), make_float2(8388608.f, 8388608.f));
        codes[k] = bad || zero ? 0x88888888u : __byte_perm(__float_as_uint(w.x), __float_as_uint(w.y), 0x5410);
        if (bad) d[k] = __ushort_as_half(0x7fff);
    }
}

}  // namespace qmm
