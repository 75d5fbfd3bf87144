// k_route.cu -- qmoe_route: the experts of each token and their weights.
//
//   s = softmax(x) or 1 / (1 + e^-x),  c = s + bias
//   groups: the top_groups largest sums of a group's group_top largest c stay
//   ids: the top_k largest c of those, ties to the lower index
//   w = s (/ their sum) * scale
//
// A warp takes a token, a lane V consecutive experts of it. Reading the logits
// bounds the operator only in the largest calls; before that it is the number of
// instructions a token takes, so that the selection does not go round the warp
// for each of the top_k:
//   1. a lower bound of the top_k-th value: the top_k-th largest of the lanes'
//      own largest values (a warp reduction each, three instructions);
//   2. the few values that reach it go to shared memory, by a scan of the lanes'
//      counts; of values equal to it the first top_k;
//   3. a lane for each of them counts those before it: its place.
//
// Order. Without a bias the scores are in the order of the logits, which are
// compared as they are. With one (and for sums over groups) fp32 values of c are off by
// up to half of `tau`: where two that matter lie closer than that and do not come from
// equal inputs, the warp computes the candidates (or, for groups, all c) in 64
// bits and counts again. With scores of 256 experts that is one token in some hundred.
#include <algorithm>

#include "layer_common.cuh"

namespace qmm {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// Unsigned keys in the order of the floats: NaN above all, 0 below all.
__device__ __forceinline__ unsigned key_of(float v) {
    const unsigned u = __float_as_uint(v + 0.f);     // -0 counts as 0
    return isnan(v) ? kAll : u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) { return value_of(__reduce_max_sync(kAll, key_of(v))); }

// A candidate: value, expert, and what its value in 64 bits is made from (or that value).
struct __align__(16) Cand {
    float c;
    int e;
    union {
        struct {
            float x, bias;
        };
        double c64;
    };
};

struct Soft {                        // softmax of a row: its largest logit, the sum relative to that
    float top, sum;
    double sum64;
};

__device__ __forceinline__ float score32(const RouteArgs& a, float x, const Soft& s) {
    if (a.score == QMM_SCORE_SIGMOID) return __fdividef(1.f, 1.f + __expf(-x));
    return s.top == -INFINITY ? 0.f : __expf(x - s.top) / s.sum;
}
__device__ __noinline__ double score64(int score, float x, float top, double sum64) {
    if (score == QMM_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-static_cast<double>(x)));
    return top == -INFINITY ? 0.0 : exp(static_cast<double>(x) - top) / sum64;
}

// Loads of V consecutive values of a row from e0 on, -Inf past n.
template <int V, typename T> __device__ __forceinline__ void load_row(const T* p, int e0, int n, bool wide, float (&x)[V]) {
    constexpr int PER = 16 / static_cast<int>(sizeof(T)), N = V < PER ? V : PER;
    if (wide) {                      // V divides n and the addresses are aligned
        Vec<T, N> v[V / N];
#pragma unroll
        for (int i = 0; i < V / N; ++i)
            if (e0 < n) v[i].load(p + e0 + i * N);
#pragma unroll
        for (int i = 0; i < V / N; ++i) {
            float f[N];
            v[i].get(f);
#pragma unroll
            for (int j = 0; j < N; ++j) x[i * N + j] = e0 < n ? f[j] : -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = e0 + i < n ? to_f32<T>(p[e0 + i]) : -INFINITY;
    }
}

template <int V, typename T>
__global__ void k_route(const __grid_constant__ RouteArgs a, bool wide) {
    grid_dep_launch();
    grid_dep_wait();
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t t = blockIdx.x * static_cast<int64_t>(blockDim.x / 32) + warp;
    if (t >= a.T) return;
    Cand* cand = reinterpret_cast<Cand*>(smem) + static_cast<size_t>(warp) * a.E;
    const int e0 = lane * V;
    float x[V];
    load_row<V, T>(static_cast<const T*>(a.logits) + t * a.stride, e0, a.E, wide, x);
    const bool softmax = a.score == QMM_SCORE_SOFTMAX, biased = a.bias != nullptr;
    const bool sums = a.groups > 1 && a.group_top == 2;

    // ---- c in fp32 (the logits themselves where their order is the scores')
    Soft soft{0.f, 1.f, 0.0};
    if (softmax && (biased || sums || !a.renorm)) {
        float m = x[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = x[i] > m || isnan(x[i]) ? x[i] : m;
        soft.top = warp_max(m);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s += soft.top == -INFINITY ? 0.f : __expf(x[i] - soft.top);
        soft.sum = warp_sum(s);
    }
    float c[V], bias[V];
    if (biased) load_row<V, float>(a.bias, e0, a.E, wide, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (!biased) bias[i] = 0.f;
        c[i] = biased || sums ? score32(a, x[i], soft) + bias[i] : x[i];
    }
    // twice the error of a c of magnitude |c|: the sigmoid's exponential and quotient
    // 2^-21.5; the softmax's, relative to its largest score 1 / sum, 2^-22, and a common factor
    // of the sum that is off by up to (V + 5) 2^-23
    const float base = softmax ? 1.52587890625e-05f / soft.sum : 1.9073486328125e-06f;   // 2^-16, 2^-19
    auto tau = [&](float v) { return base + 4.76837158203125e-07f * fabsf(v); };         // 2^-21

    auto sum64 = [&]() {                                  // of the softmax, when asked for
        if (!softmax) return 0.0;
        double s = 0.0;
#pragma unroll 1
        for (int i = 0; i < V; ++i) {
            float xi = x[0];
#pragma unroll
            for (int j = 1; j < V; ++j) xi = i == j ? x[j] : xi;
            s += e0 + i < a.E ? score64(QMM_SCORE_SOFTMAX, xi, soft.top, 1.0) : 0.0;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        return s;
    };

    // ---- groups
    unsigned kept = kAll;
    const int gs = a.E / a.groups;
    if (a.groups > 1) {
        // a lane for each group: its one or two largest c, summed
        float v = 0.f;
        const int lanes = gs / V;
        if (gs % V == 0 && (lanes & (lanes - 1)) == 0) {  // whole lanes, a power of two of them
            float m1 = c[0], m2 = -INFINITY;
            auto take = [&](float b1, float b2) {         // of (m1, m2) and (b1, b2) the two largest; NaN the largest
                const bool over = b1 > m1 || isnan(b1);
                const float lo = over ? m1 : b1;
                const float other = over ? b2 : m2;
                m1 = over ? b1 : m1;
                m2 = lo > other || isnan(lo) ? lo : other;
            };
#pragma unroll
            for (int i = 1; i < V; ++i) take(c[i], -INFINITY);
            for (int o = 1; o < lanes; o <<= 1) {
                const float b1 = __shfl_xor_sync(kAll, m1, o), b2 = __shfl_xor_sync(kAll, m2, o);
                take(b1, b2);
            }
            v = __shfl_sync(kAll, a.group_top == 2 ? m1 + m2 : m1, (lane * lanes) & 31);
        } else {
            float* all = reinterpret_cast<float*>(cand);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e0 + i < a.E) all[e0 + i] = c[i];
            __syncwarp();
            if (lane < a.groups) {
                float m1 = all[lane * gs], m2 = -INFINITY;
                for (int i = 1; i < gs; ++i) {
                    const float b = all[lane * gs + i];
                    const bool over = b > m1 || isnan(b);
                    const float lo = over ? m1 : b;
                    m1 = over ? b : m1;
                    m2 = lo > m2 || isnan(lo) ? lo : m2;
                }
                v = a.group_top == 2 ? m1 + m2 : m1;
            }
            __syncwarp();
        }
        const bool mine = lane < a.groups;
        const unsigned k = mine ? key_of(v) : 0u;
        int place = 0;
        for (int g = 0; g < a.groups; ++g) {
            const unsigned other = __shfl_sync(kAll, k, g);
            place += other > k || (other == k && g < lane);
        }
        kept = __ballot_sync(kAll, mine && place < a.top_groups);
        if ((biased || sums) && a.top_groups < a.groups) {
            const unsigned last = __reduce_min_sync(kAll, kept >> lane & 1 ? k : kAll);
            const unsigned next = __reduce_max_sync(kAll, kept >> lane & 1 ? 0u : k);
            const float lo = value_of(last);
            if (last != kAll && lo - value_of(next) <= 2.f * (tau(lo) + tau(value_of(next)))) {   // decided in 64 bits
                const double s64 = sum64();
                double* all = reinterpret_cast<double*>(cand);
#pragma unroll 1
                for (int i = 0; i < V; ++i) {
                    float xi = x[0], bi = bias[0];
#pragma unroll
                    for (int j = 1; j < V; ++j) {
                        xi = i == j ? x[j] : xi;
                        bi = i == j ? bias[j] : bi;
                    }
                    if (e0 + i < a.E) all[e0 + i] = score64(a.score, xi, soft.top, s64) + bi;
                }
                __syncwarp();
                double w = -INFINITY;
                if (mine) {
                    double m1 = all[lane * gs], m2 = -INFINITY;
                    for (int i = 1; i < gs; ++i) {
                        const double b = all[lane * gs + i];
                        const bool over = b > m1;
                        const double lo64 = over ? m1 : b;
                        m1 = over ? b : m1;
                        m2 = fmax(m2, lo64);
                    }
                    w = a.group_top == 2 ? m1 + m2 : m1;
                }
                place = 0;
                for (int g = 0; g < a.groups; ++g) {
                    const double other = __shfl_sync(kAll, w, g);
                    place += other > w || (other == w && g < lane);
                }
                kept = __ballot_sync(kAll, mine && place < a.top_groups);
                __syncwarp();
            }
        }
    }

    // ---- keys; 0 where an expert does not stay
    unsigned key[V], most = 0u;
    {
        int g = 0, left = gs;                             // group of the lane's first expert, experts of it still to come
        if (a.groups > 1) {
            g = e0 / gs;
            left = gs - (e0 - g * gs);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool in = e0 + i < a.E && (a.groups == 1 || (kept >> g & 1));
            key[i] = in ? key_of(biased ? c[i] : x[i]) : 0u;
            most = max(most, key[i]);
            if (--left == 0) {
                ++g;
                left = gs;
            }
        }
    }
    // ---- 1. the bound
    unsigned bound = 0u;
    for (int r = 0; r < a.top_k; ++r) {
        bound = __reduce_max_sync(kAll, most);
        most = most == bound ? 0u : most;
    }
    bound = max(bound, 1u);
    const unsigned exact_bound = bound;
    if (biased && bound != 1u) {                          // all that may be the top_k-th by more exact values
        const float v = value_of(bound);
        if (!isnan(v)) bound = min(bound, max(1u, key_of(v - 2.f * tau(v))));
    }
    // ---- 2. the candidates; equal keys at the bound: the first top_k of them, where keys are exact
    const bool limit = bound == exact_bound && !biased;
    unsigned count = 0u;                                  // above the bound; equal to it in the upper half
#pragma unroll
    for (int i = 0; i < V; ++i) count += key[i] > bound ? 1u : key[i] == bound ? (limit ? 0x10000u : 1u) : 0u;
    unsigned scan = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned up = __shfl_up_sync(kAll, scan, o);
        scan += lane >= o ? up : 0u;
    }
    const unsigned total = __shfl_sync(kAll, scan, 31);
    const int above = static_cast<int>(total & 0xffffu), n = above + min(static_cast<int>(total >> 16), a.top_k);
    {
        unsigned at = scan - count;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool over = key[i] > bound || (!limit && key[i] == bound), same = limit && key[i] == bound;
            const int where = over ? static_cast<int>(at & 0xffffu) : above + static_cast<int>(at >> 16);
            if (over || (same && static_cast<int>(at >> 16) < a.top_k)) {
                Cand q;
                q.c = biased ? c[i] : x[i];
                q.e = e0 + i;
                q.x = x[i];
                q.bias = bias[i];
                cand[where] = q;
            }
            at += over ? 1u : same ? 0x10000u : 0u;
        }
    }
    __syncwarp();
    // ---- 3. their places; the chosen lie in lane `place` at the end
    int* order = reinterpret_cast<int*>(smem + static_cast<size_t>(blockDim.x / 32) * a.E * sizeof(Cand)) + warp * kMaxTopK;
    bool close = false;
    for (int i = lane; i < n; i += 32) {
        const Cand me = cand[i];
        const unsigned k = key_of(me.c);
        int place = 0;
        bool near = false;
        for (int j = 0; j < n; ++j) {
            const Cand q = cand[j];
            const unsigned o = key_of(q.c);
            place += o > k || (o == k && q.e < me.e);
            near |= fabsf(q.c - me.c) <= tau(me.c) && j != i && (q.x != me.x || q.bias != me.bias);
        }
        close |= biased && near && place < a.top_k;
        if (place < a.top_k) order[place] = i;
    }
    float lx = 0.f;                                       // the chosen expert's logit, a lane each
    int le = 0;
    if (__any_sync(kAll, close)) {
        const double s64 = sum64();
        for (int i = lane; i < n; i += 32) {
            const Cand q = cand[i];
            cand[i].c = q.x;
            cand[i].c64 = score64(a.score, q.x, soft.top, s64) + q.bias;
        }
        __syncwarp();
        for (int i = lane; i < n; i += 32) {
            const double w = cand[i].c64;
            const int e = cand[i].e;
            int place = 0;
            for (int j = 0; j < n; ++j) {
                const double o = cand[j].c64;
                place += o > w || (o == w && cand[j].e < e) || (isnan(o) && (!isnan(w) || cand[j].e < e) && j != i);
            }
            if (place < a.top_k) order[place] = i;
        }
        __syncwarp();
        if (lane < a.top_k) {
            lx = cand[order[lane]].c;
            le = cand[order[lane]].e;
        }
    } else {
        __syncwarp();
        if (lane < a.top_k) {
            lx = cand[order[lane]].x;
            le = cand[order[lane]].e;
        }
    }

    // ---- weights
    const bool chosen = lane < a.top_k;
    float w = 0.f;
    if (softmax) {
        // renormalised, the row's sum falls out; relative to the largest chosen logit
        const float top = a.renorm ? warp_max(chosen ? lx : -INFINITY) : soft.top;
        w = chosen && top != -INFINITY ? expf(lx - top) : 0.f;
        if (!a.renorm) w /= soft.sum;
    } else if (chosen) {
        w = 1.f / (1.f + expf(-lx));
    }
    if (a.renorm) {
        const float sum = warp_sum(w);
        w = sum == 0.f ? 0.f : w / sum;
    }
    if (chosen) {
        a.ids[t * a.top_k + lane] = le;
        a.weights[t * a.top_k + lane] = w * a.scale;
    }
}

template <int V, typename T> cudaError_t go(const RouteArgs& a, cudaStream_t s) {
    // warps of a block: what fits 48 KB, at most eight, fewer where that fills more SMs
    int dev = 0;
    cudaGetDevice(&dev);
    const int64_t per_sm = (a.T + sm_count(dev) - 1) / sm_count(dev);
    const size_t warp_bytes = static_cast<size_t>(a.E) * sizeof(Cand) + kMaxTopK * 4;
    int warps = static_cast<int>(std::min<int64_t>({8, static_cast<int64_t>(49152 / warp_bytes), per_sm}));
    warps = std::max(1, warps);
    const int64_t blocks = (a.T + warps - 1) / warps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const bool wide = a.E % V == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0 &&
                      (a.T == 1 || a.stride * static_cast<int64_t>(sizeof(T)) % 16 == 0);
    return launch_chained(k_route<V, T>, dim3(static_cast<unsigned>(blocks)), warps * 32, static_cast<int>(warps * warp_bytes), s, a, wide);
}

template <typename T> cudaError_t pick(const RouteArgs& a, cudaStream_t s) {
    if (a.E <= 32) return go<1, T>(a, s);
    if (a.E <= 64) return go<2, T>(a, s);
    if (a.E <= 128) return go<4, T>(a, s);
    if (a.E <= 256) return go<8, T>(a, s);
    if (a.E <= 512) return go<16, T>(a, s);
    return go<32, T>(a, s);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
    if (a.dtype == QMM_F32) return pick<float>(a, s);
    if (a.dtype == QMM_F16) return pick<__half>(a, s);
    return pick<__nv_bfloat16>(a, s);
}

}  // namespace qmm
