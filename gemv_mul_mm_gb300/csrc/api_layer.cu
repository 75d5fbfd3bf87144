// api_layer.cu -- the C ABI of the norm and the router (include/qmm.h): argument
// validation and dispatch.
#include <cmath>

#include "api_checks.cuh"
#include "layer_common.cuh"

using namespace qmm;

namespace {

int done(cudaError_t e, int path) {
    if (e != cudaSuccess) return QMM_ERR_CUDA;
    set_last_path(path);
    return QMM_OK;
}

// A T x H array of rows of D elements in memory.
struct Rows {
    const void* p;
    int64_t ts, hs, D, size;       // strides and D in elements of `size` bytes
};

bool strides_ok(int64_t ts, int64_t hs) { return ts >= 0 && hs >= 0 && ts <= kBig && hs <= kBig; }

// Whether the ranges of bytes that two arrays lie in are apart.
bool apart(const Rows& a, const Rows& b, int64_t T, int64_t H) {
    auto bytes = [&](const Rows& r) { return ((T - 1) * static_cast<__int128>(r.ts) + (H - 1) * static_cast<__int128>(r.hs) + r.D) * r.size; };
    const __int128 pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    return pa + bytes(a) <= pb || pb + bytes(b) <= pa;
}

// Whether rows of `out` may be written while those of `in` are read by the thread
// that writes the same elements.
bool may_write(const Rows& out, const Rows& in, bool same_type, int64_t T, int64_t H) {
    if (apart(out, in, T, H)) return true;
    return same_type && apart_or_same(in.p, in.ts, in.hs, out.p, out.ts, out.hs, T, H, out.D, out.size);
}

}  // namespace

extern "C" {

int qrmsnorm(const void* X, int x_dtype, size_t x_elems, int64_t x_ts, int64_t x_hs, const void* residual, int r_dtype,
             size_t r_elems, int64_t r_ts, int64_t r_hs, void* residual_out, size_t ro_elems, int64_t ro_ts, int64_t ro_hs,
             const float* weight, size_t weight_elems, float weight_offset, float eps, void* Y, int y_fmt, size_t y_elems,
             int64_t y_ts, int64_t y_hs, int64_t T, int64_t H, int64_t D, void* stream) {
    const bool q8 = y_fmt == QMM_NORM_Q8_0;
    if (!dtype_ok(x_dtype) || (residual && !dtype_ok(r_dtype)) || (!q8 && !dtype_ok(y_fmt))) return QMM_ERR_BAD_DTYPE;
    if (T < 0 || H < 0 || D < 0 || !strides_ok(x_ts, x_hs) || !strides_ok(y_ts, y_hs)) return QMM_ERR_BAD_ARGUMENT;
    if (residual && !strides_ok(r_ts, r_hs)) return QMM_ERR_BAD_ARGUMENT;
    if (residual_out && (!residual || !strides_ok(ro_ts, ro_hs))) return QMM_ERR_BAD_ARGUMENT;
    if (T == 0 || H == 0 || D == 0) return QMM_ERR_EMPTY_SHAPE;
    if (H > 65536 || D > (1 << 20) || T > 0x7fffffff / H) return QMM_ERR_BAD_ARGUMENT;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(weight_offset)) return QMM_ERR_BAD_ARGUMENT;
    if (q8 && D % 32) return QMM_ERR_COLS_NOT_BLOCK_ALIGNED;
    if (!X || !Y) return QMM_ERR_NULL_POINTER;
    const int64_t y_size = q8 ? 1 : esize(y_fmt), y_row = q8 ? D / 32 * 34 : D;
    if (!aligned(X, esize(x_dtype)) || !aligned(weight, 4) || !aligned(Y, q8 ? 2 : y_size)) return QMM_ERR_MISALIGNED;
    if (q8 && ((T > 1 && y_ts % 2) || (H > 1 && y_hs % 2))) return QMM_ERR_MISALIGNED;
    if (residual && (!aligned(residual, esize(r_dtype)) || !aligned(residual_out, esize(r_dtype)))) return QMM_ERR_MISALIGNED;
    if (!fits(x_elems, T, x_ts, H, x_hs, D) || (residual && !fits(r_elems, T, r_ts, H, r_hs, D)) ||
        (weight && weight_elems < static_cast<size_t>(D)))
        return QMM_ERR_ACTIVATIONS_TOO_SMALL;
    if (!fits(y_elems, T, y_ts, H, y_hs, y_row) || (residual_out && !fits(ro_elems, T, ro_ts, H, ro_hs, D)))
        return QMM_ERR_OUTPUT_TOO_SMALL;

    const Rows x{X, x_ts, x_hs, D, esize(x_dtype)}, y{Y, y_ts, y_hs, y_row, y_size};
    const Rows w{weight, 0, 0, D, 4};
    if (rows_meet(T, y_ts, H, y_hs, y_row) || !may_write(y, x, !q8 && y_fmt == x_dtype, T, H) ||
        (weight && !apart(y, w, T, H)))
        return QMM_ERR_BAD_ARGUMENT;
    if (residual) {
        const Rows r{residual, r_ts, r_hs, D, esize(r_dtype)};
        if (!apart(y, r, T, H)) return QMM_ERR_BAD_ARGUMENT;
        if (residual_out) {
            const Rows o{residual_out, ro_ts, ro_hs, D, esize(r_dtype)};
            if (rows_meet(T, ro_ts, H, ro_hs, D) || !may_write(o, r, true, T, H) || !may_write(o, x, r_dtype == x_dtype, T, H) ||
                !apart(o, y, T, H) || (weight && !apart(o, w, T, H)))
                return QMM_ERR_BAD_ARGUMENT;
        }
    }
    NormArgs a;
    a.X = X;
    a.R = residual;
    a.RO = residual_out;
    a.W = weight;
    a.Y = Y;
    a.x_dt = x_dtype;
    a.r_dt = r_dtype;
    a.y_fmt = y_fmt;
    a.x_ts = x_ts;
    a.x_hs = x_hs;
    a.r_ts = r_ts;
    a.r_hs = r_hs;
    a.ro_ts = ro_ts;
    a.ro_hs = ro_hs;
    a.y_ts = y_ts;
    a.y_hs = y_hs;
    a.w_off = weight_offset;
    a.eps = eps;
    a.T = T;
    a.H = H;
    a.D = D;
    return done(launch_norm(a, static_cast<cudaStream_t>(stream)), 12);
}

int qmoe_route(const void* logits, int dtype, size_t elems, int64_t stride, const float* bias, int score, int n_groups,
               int top_groups, int group_top, int top_k, int renorm, float scale, int32_t* ids, float* weights,
               size_t out_elems, int64_t T, int n_experts, void* stream) {
    if (!dtype_ok(dtype)) return QMM_ERR_BAD_DTYPE;
    if (T < 0 || n_experts < 0 || top_k < 0 || stride < 0 || stride > kBig) return QMM_ERR_BAD_ARGUMENT;
    if (T == 0 || n_experts == 0 || top_k == 0) return QMM_ERR_EMPTY_SHAPE;
    if (score != QMM_SCORE_SOFTMAX && score != QMM_SCORE_SIGMOID) return QMM_ERR_BAD_ARGUMENT;
    if (n_groups < 1 || n_experts % n_groups || top_groups < 1 || top_groups > n_groups || group_top < 1 || group_top > 2 ||
        !std::isfinite(scale))
        return QMM_ERR_BAD_ARGUMENT;
    const int group = n_experts / n_groups;
    if ((n_groups > 1 && group_top > group) || top_k > static_cast<int64_t>(top_groups) * group) return QMM_ERR_BAD_ARGUMENT;
    if (n_experts > kMaxExperts || top_k > kMaxTopK || n_groups > kMaxGroups) return QMM_ERR_UNIMPLEMENTED;
    if (T > (int64_t(1) << 33)) return QMM_ERR_BAD_ARGUMENT;
    if (!logits || !ids || !weights) return QMM_ERR_NULL_POINTER;
    if (!aligned(logits, esize(dtype)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return QMM_ERR_MISALIGNED;
    if (!fits(elems, T, stride, 1, 0, n_experts)) return QMM_ERR_ACTIVATIONS_TOO_SMALL;
    if (!fits(out_elems, T, top_k, 1, 0, top_k)) return QMM_ERR_OUTPUT_TOO_SMALL;
    const Rows x{logits, stride, 0, n_experts, esize(dtype)}, b{bias, 0, 0, n_experts, 4};
    const Rows i{ids, top_k, 0, top_k, 4}, w{weights, top_k, 0, top_k, 4};
    if (!apart(i, x, T, 1) || !apart(w, x, T, 1) || !apart(i, w, T, 1) || (bias && (!apart(i, b, T, 1) || !apart(w, b, T, 1))))
        return QMM_ERR_BAD_ARGUMENT;
    RouteArgs a;
    a.logits = logits;
    a.dtype = dtype;
    a.stride = stride;
    a.bias = bias;
    a.score = score;
    a.E = n_experts;
    a.groups = n_groups;
    a.top_groups = top_groups;
    a.group_top = group_top;
    a.top_k = top_k;
    a.renorm = renorm != 0;
    a.scale = scale;
    a.ids = ids;
    a.weights = weights;
    a.T = T;
    return done(launch_route(a, static_cast<cudaStream_t>(stream)), 13);
}

}  // extern "C"
