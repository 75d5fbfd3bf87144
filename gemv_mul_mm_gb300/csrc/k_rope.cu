// k_rope.cu -- rotary positions (qrope).
//
// For token t, head h and pair i < rot / 2, with a = 2 pi frac(pos_t * turns_i):
//   y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a)
// (x1, x2) = elements (i, i + rot/2) (half layout) or (2i, 2i + 1)
// (interleaved). Elements from rot on are copied.
//
// Bound by reading X and writing Y. An item is two vectors of N elements of one
// head (half layout: N elements of the first half and their partners;
// interleaved: 2 N consecutive ones; past rot: up to 2 N copied). A block takes
// a few tokens and one to four items a thread; it loads them all, computes each
// (token, pair)'s cos and sin once into shared memory meanwhile (a thread that
// computed its own spent as many instructions on them as on four heads), and
// then rotates and stores.
#include <algorithm>

#include "kv_common.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kAngles = 1024;    // (token, pair)s per block

struct RopeShape {
    int units, rot_units;        // items of a head, those of them that rotate
    int heads;                   // heads per block
    int tokens;                  // tokens per block
    int head_groups;
};

template <typename T, int N, int ITEMS>
__global__ void __launch_bounds__(kThreads) k_rope(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeShape g) {
    grid_dep_launch();
    grid_dep_wait();
    __shared__ float2 cs[kAngles];   // [token][j][unit]: pair unit * N + j, units side by side for the reads
    const int hg = static_cast<int>(blockIdx.x % static_cast<unsigned>(g.head_groups));
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / static_cast<unsigned>(g.head_groups)) * g.tokens;
    const int tokens = static_cast<int>(imin64(g.tokens, a.T - t0));
    const int h0 = hg * g.heads, heads = static_cast<int>(imin64(g.heads, a.H - h0));
    const int pairs = a.rot / 2;
    const bool half = a.layout == QMM_ROPE_HALF;

    Vec<T, N> v0[ITEMS], v1[ITEMS];
    int unit[ITEMS], tok[ITEMS];
    int64_t off_x[ITEMS], off_y[ITEMS];
    // item = (token, head, unit), units innermost; a thread's items are 256 apart
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const unsigned i = threadIdx.x + k * kThreads, th = i / static_cast<unsigned>(g.units);
        unit[k] = static_cast<int>(i - th * g.units);
        tok[k] = static_cast<int>(th / static_cast<unsigned>(heads));
        const int h = h0 + static_cast<int>(th) - tok[k] * heads;
        const bool turn = unit[k] < g.rot_units;
        const int e0 = turn ? (half ? unit[k] * N : unit[k] * 2 * N) : a.rot + (unit[k] - g.rot_units) * 2 * N;
        off_x[k] = (t0 + tok[k]) * a.x_ts + h * a.x_hs + e0;
        off_y[k] = (t0 + tok[k]) * a.y_ts + h * a.y_hs + e0;
        if (tok[k] < tokens) {
            const T* x = static_cast<const T*>(a.X) + off_x[k];
            v0[k].load(x);
            if (turn) v1[k].load(x + (half ? pairs : N));
            else if (e0 + N < a.D) v1[k].load(x + N);
        }
    }
    for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
        const int tt = i / pairs, p = i - tt * pairs;
        float2 v;
        rope_cs(a.pos[t0 + tt], a.turns[p], a.mscale, v.x, v.y);
        cs[tt * pairs + p % N * g.rot_units + p / N] = v;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        if (tok[k] >= tokens) break;
        const bool turn = unit[k] < g.rot_units;
        if (turn) {
            float f0[N], f1[N];
            v0[k].get(f0);
            v1[k].get(f1);
            const float2* c = cs + tok[k] * pairs + unit[k];
            auto turn_pair = [&](float& x1, float& x2, int j) {
                const float2 w = c[j * g.rot_units];
                const float y1 = x1 * w.x - x2 * w.y;
                x2 = x2 * w.x + x1 * w.y;
                x1 = y1;
            };
            if (half || N == 1) {
#pragma unroll
                for (int j = 0; j < N; ++j) turn_pair(f0[j], f1[j], j);
            } else {
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    turn_pair(f0[2 * j], f0[(2 * j + 1) % N], j);
                    turn_pair(f1[2 * j], f1[(2 * j + 1) % N], N / 2 + j);
                }
            }
            v0[k].set(f0);
            v1[k].set(f1);
        }
        T* y = static_cast<T*>(a.Y) + off_y[k];
        v0[k].store(y);
        if (turn) v1[k].store(y + (half ? pairs : N));
        else if (a.rot + (unit[k] - g.rot_units) * 2 * N + N < a.D) v1[k].store(y + N);
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
    RopeShape g;
    g.rot_units = a.rot / (2 * N);
    g.units = g.rot_units + (in_place ? 0 : static_cast<int>((a.D - a.rot + 2 * N - 1) / (2 * N)));
    // Items per thread, whose loads are in flight together: four where that still
    // leaves twelve blocks per SM (four waves), two down to two blocks per SM, one
    // below
    int dev = 0;
    cudaGetDevice(&dev);
    const int64_t per_sm = a.T * a.H * g.units / (static_cast<int64_t>(sm_count(dev)) * kThreads);
    const int per_thread = per_sm >= 48 ? 4 : per_sm >= 4 ? 2 : 1;
    const int items = per_thread * kThreads;
    g.heads = static_cast<int>(std::min<int64_t>(a.H, std::max(1, items / g.units)));
    g.head_groups = static_cast<int>((a.H + g.heads - 1) / g.heads);
    // (a head of more units than that, up to 1024, has a block of its own below)
    g.tokens = std::max(1, std::min(items / (g.heads * g.units), kAngles / (a.rot / 2)));
    const int64_t blocks = (a.T + g.tokens - 1) / g.tokens * g.head_groups;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    auto go = [&](auto kernel) { return launch_chained(kernel, dim3(static_cast<unsigned>(blocks)), kThreads, 0, s, a, g); };
    const int need = g.tokens * g.heads * g.units;
    return need <= kThreads ? go(k_rope<T, N, 1>) : need <= 2 * kThreads ? go(k_rope<T, N, 2>) : go(k_rope<T, N, 4>);
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
