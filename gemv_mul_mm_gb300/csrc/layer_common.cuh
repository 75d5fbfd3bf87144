// layer_common.cuh -- the norm and the router: arguments and launchers.
#pragma once

#include "kv_common.cuh"

namespace qmm {

// k_norm.cu
struct NormArgs {
    const void* X;
    const void* R;                 // residual or nullptr
    void* RO;                      // where x + residual goes, or nullptr
    const float* W;                // nullptr: ones
    void* Y;
    int x_dt, r_dt;                // QMM_F32 / QMM_F16 / QMM_BF16
    int y_fmt;                     // one of them, or QMM_NORM_Q8_0 (y strides in bytes)
    int64_t x_ts, x_hs, r_ts, r_hs, ro_ts, ro_hs, y_ts, y_hs;
    float w_off, eps;
    unsigned h_mul = 0;            // row / H (set by the launcher, as is x_shift)
    int h_shift = 0;
    bool w_at16 = false;           // W on a 16-byte boundary
    int x_shift = 0;               // elements by which X begins past an 8-element grid
    int64_t T, H, D;
};
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s);

// k_route.cu
constexpr int kMaxExperts = 1024, kMaxTopK = 32, kMaxGroups = 32;
struct RouteArgs {
    const void* logits;
    int dtype;
    int64_t stride;
    const float* bias;             // or nullptr
    int score;                     // QMM_SCORE_*
    int E, groups, top_groups, group_top, top_k;
    bool renorm;
    float scale;
    int32_t* ids;
    float* weights;
    int64_t T;
};
cudaError_t launch_route(const RouteArgs& a, cudaStream_t s);

}  // namespace qmm
