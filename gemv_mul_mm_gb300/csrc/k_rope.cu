// k_rope.cu -- rotary positions (qrope).
//
// For token t, head h and pair i < rot / 2, with a = 2 pi frac(pos_t * turns_i):
//   y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a)
// (x1, x2) = elements (i, i + rot/2) (half layout) or (2i, 2i + 1)
// (interleaved). Elements from rot on are copied.
#include <algorithm>

#include "kv_common.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;

// A thread holds two vectors of N elements of each of its heads: in the half
// layout N elements of the first half and their partners, interleaved 2 N
// consecutive elements; past `rot` it copies 2 N (the last thread N)
// elements. cos and sin are computed once per thread and serve all its heads.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads) k_rope(RopeArgs a, int64_t threads, int units, int rot_units, int head_groups,
                                                   int heads_per) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t id = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    if (id >= threads) return;
    const int u = static_cast<int>(id % units);
    const int64_t th = id / units;
    const int hg = static_cast<int>(th % head_groups);
    const int64_t t = th / head_groups;
    const int64_t h0 = static_cast<int64_t>(hg) * heads_per;
    const int64_t h1 = imin64(h0 + heads_per, a.H);
    const bool turn = u < rot_units;
    const bool half = a.layout == QMM_ROPE_HALF;
    const int64_t e0 = turn ? (half ? static_cast<int64_t>(u) * N : static_cast<int64_t>(u) * 2 * N)
                            : a.rot + static_cast<int64_t>(u - rot_units) * 2 * N;
    const int64_t e1 = turn && half ? e0 + a.rot / 2 : e0 + N;
    const bool second = e1 < a.D;

    float c[N], s[N];
    if (turn) {
        const int32_t pos = a.pos[t];
#pragma unroll
        for (int j = 0; j < N; ++j) rope_cs(pos, a.turns[u * N + j], a.mscale, c[j], s[j]);
    }
    const T* x = static_cast<const T*>(a.X) + t * a.x_ts;
    T* y = static_cast<T*>(a.Y) + t * a.y_ts;
#pragma unroll 4
    for (int64_t h = h0; h < h1; ++h) {
        float v0[N], v1[N];
        load_vec<T, N>(x + h * a.x_hs + e0, v0);
        if (second) load_vec<T, N>(x + h * a.x_hs + e1, v1);
        if (turn) {
            if (half) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float x1 = v0[j], x2 = v1[j];
                    v0[j] = x1 * c[j] - x2 * s[j];
                    v1[j] = x2 * c[j] + x1 * s[j];
                }
            } else if constexpr (N == 1) {
                const float x1 = v0[0], x2 = v1[0];
                v0[0] = x1 * c[0] - x2 * s[0];
                v1[0] = x2 * c[0] + x1 * s[0];
            } else {
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    float x1 = v0[2 * j], x2 = v0[2 * j + 1];
                    v0[2 * j] = x1 * c[j] - x2 * s[j];
                    v0[2 * j + 1] = x2 * c[j] + x1 * s[j];
                    x1 = v1[2 * j], x2 = v1[2 * j + 1];
                    v1[2 * j] = x1 * c[N / 2 + j] - x2 * s[N / 2 + j];
                    v1[2 * j + 1] = x2 * c[N / 2 + j] + x1 * s[N / 2 + j];
                }
            }
        }
        store_vec<T, N>(y + h * a.y_hs + e0, v0);
        if (second) store_vec<T, N>(y + h * a.y_hs + e1, v1);
    }
}

// Whether N-element vectors of `size`-byte elements fit every address of the
// call.
bool vec_ok(const RopeArgs& a, int n, int size) {
    const int64_t b = static_cast<int64_t>(n) * size < 16 ? n * size : 16;
    const int64_t strides[4] = {a.x_ts, a.x_hs, a.y_ts, a.y_hs};
    for (int64_t st : strides)
        if ((st * size) % b) return false;
    if (reinterpret_cast<uintptr_t>(a.X) % b || reinterpret_cast<uintptr_t>(a.Y) % b) return false;
    return a.rot % (2 * n) == 0 && (a.D - a.rot) % n == 0;
}

template <typename T, int N> cudaError_t run(const RopeArgs& a, cudaStream_t s) {
    const bool in_place = a.X == a.Y && a.x_ts == a.y_ts && a.x_hs == a.y_hs;
    const int rot_units = a.rot / (2 * N);
    const int rest = static_cast<int>((a.D - a.rot + 2 * N - 1) / (2 * N));
    const int units = rot_units + (in_place ? 0 : rest);
    // heads per thread: as many as leave about two blocks of 256 threads per SM
    // in flight, so that cos and sin are shared; one where the call is small
    int dev = 0;
    cudaGetDevice(&dev);
    const int64_t want = static_cast<int64_t>(sm_count(dev)) * 2 * kThreads;
    const int64_t all = a.T * units * a.H;
    const int64_t per = std::max<int64_t>(1, std::min<int64_t>({a.H, 16, all / want}));
    const int groups = static_cast<int>((a.H + per - 1) / per);
    const int64_t threads = a.T * units * groups;
    const int64_t blocks = (threads + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_chained(k_rope<T, N>, dim3(static_cast<unsigned>(blocks)), kThreads, 0, s, a, threads, units, rot_units, groups,
                          static_cast<int>(per));
}

template <typename T> cudaError_t pick(const RopeArgs& a, cudaStream_t s) {
    constexpr int S = static_cast<int>(sizeof(T));
    if (vec_ok(a, 16 / S, S)) return run<T, 16 / S>(a, s);
    if (vec_ok(a, 2, S)) return run<T, 2>(a, s);
    return run<T, 1>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
    if (a.dtype == QMM_F32) return pick<float>(a, s);
    if (a.dtype == QMM_F16) return pick<__half>(a, s);
    return pick<__nv_bfloat16>(a, s);
}

}  // namespace qmm
