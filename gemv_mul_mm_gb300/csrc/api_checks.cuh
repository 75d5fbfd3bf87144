// api_checks.cuh -- argument checks that the entry points share: types, alignment,
// sizes and overlaps of strided rows.
#pragma once

#include <algorithm>
#include <cstdint>
#include <cstdlib>

#include "qmm.h"

namespace qmm {

inline bool dtype_ok(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }
inline int64_t esize(int t) { return t == QMM_F32 ? 4 : 2; }
inline bool aligned(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Whether rows x cols x last elements with these strides stay inside `elems`
// elements. Strides and sizes are at most 2^40, so nothing overflows.
constexpr int64_t kBig = int64_t(1) << 40;
inline bool fits(size_t elems, int64_t rows, int64_t rs, int64_t cols, int64_t cs, int64_t last) {
    const __int128 need = static_cast<__int128>(rows - 1) * rs + static_cast<__int128>(cols - 1) * cs + last;
    return need <= static_cast<__int128>(elems);
}

// Whether some |o + t * ts| < D with |t| < T (t = 0 not counted with `apart`).
inline bool comes_near(int64_t o, int64_t T, int64_t ts, int64_t D, bool apart) {
    const int64_t at = ts ? std::min(std::max(-o / ts, 1 - T), T - 1) : T > 1;
    for (int64_t t = std::max(at - 1, 1 - T); t <= std::min(at + 1, T - 1); ++t)
        if (!(apart && t == 0) && std::llabs(o + t * ts) < D) return true;
    return false;
}

// Whether two rows of Y (t, h), D elements at t * ts + h * hs, share an element.
inline bool rows_meet(int64_t T, int64_t ts, int64_t H, int64_t hs, int64_t D) {
    if ((H == 1 || hs >= D) && (T == 1 || ts >= (H - 1) * hs + D)) return false;   // the usual order
    if ((T == 1 || ts >= D) && (H == 1 || hs >= (T - 1) * ts + D)) return false;
    for (int64_t h = 0; h < H; ++h)
        if (comes_near(h * hs, T, ts, D, h == 0)) return true;
    return false;
}

// Whether rows of Y may be written while those of X are read, T x H rows of D
// elements each: Y is X, or they share no element. Where their ranges meet and
// their token strides differ that is not looked into.
inline bool apart_or_same(const void* X, int64_t x_ts, int64_t x_hs, const void* Y, int64_t y_ts, int64_t y_hs, int64_t T, int64_t H,
                   int64_t D, int64_t size) {
    const int64_t x0 = reinterpret_cast<intptr_t>(X) / size, y0 = reinterpret_cast<intptr_t>(Y) / size;
    const int64_t xn = (T - 1) * x_ts + (H - 1) * x_hs + D, yn = (T - 1) * y_ts + (H - 1) * y_hs + D;
    if (x0 + xn <= y0 || y0 + yn <= x0) return true;
    const bool same_ts = T == 1 || x_ts == y_ts, same_hs = H == 1 || x_hs == y_hs;
    if (X == Y && same_ts && same_hs) return true;
    if (!same_ts || (!same_hs && H > 1024)) return false;
    const int64_t lo = same_hs ? 1 - H : 0;          // same_hs: h is a difference of heads
    for (int64_t h = lo; h < H; ++h)
        for (int64_t g = 0; g < (same_hs ? 1 : H); ++g)
            if (comes_near(y0 - x0 + h * y_hs - g * x_hs, T, x_ts, D, false)) return false;
    return true;
}

}  // namespace qmm
