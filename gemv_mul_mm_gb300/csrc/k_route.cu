// k_route.cu -- qmoe_route: the experts of each token and their weights.
//
//   s = softmax(x) or 1 / (1 + e^-x),  c = s + bias
//   groups: the top_groups largest sums of a group's group_top largest c stay
//   ids: the top_k largest c of those, ties to the lower index
//   w = s (/ their sum) * scale
//
// A warp takes a token, a lane V consecutive experts of it (or, of many tokens with few
// experts to choose, eight lanes take one: k_route_four). The instructions that a
// token takes bound the operator, not the reading of its logits, so that the
// selection does not search the whole warp again for each of the top_k:
//   1. a lower bound of the top_k-th value: the top_k-th largest of the lanes'
//      own largest values (a warp reduction and two instructions each);
//   2. the few values that reach it go to shared memory, by a scan of the lanes'
//      counts; of values equal to it the first top_k;
//   3. a lane for each of them counts those before it: its place.
//
// Order. Values are compared as unsigned keys. Without a bias the scores are in
// the order of the logits, which are compared as they are. With one (and for sums
// over groups; BY_SCORE) fp32 values of c are off by up to half of `tau`: where two neighbours of
// the order that matter lie closer than that and do not come from equal inputs,
// the warp computes the candidates (for groups: the few that may be among a group's largest)
// in 64 bits and counts again. With the scores of 256 experts that is one token in some hundred.
//
// Measured: 65536 tokens x 128 experts, bf16, top 8: 13.6 us (1.5 TB/s; 25.6 with a warp a
// token, 183 instructions a token against 496); 8192 x 256 in 8 groups, sigmoid with a
// bias: 11.5 us and, where a token's groups lie close enough to be decided in 64 bits, up to 21;
// 65536 x 256 in groups 70 us (450 instructions a token at 31 % of the issue slots: 16 warps an
// SM, by registers), with a bias and no groups 53 (a warp a token, 710, 62 %); one token 2 to 4 us.
#include <algorithm>
#include <type_traits>

#include "exp64.cuh"
#include "layer_common.cuh"

namespace qmm {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// Unsigned keys in the order of the floats: NaN above all, 0 below all. The sum with
// zero makes -0 equal to 0 and every NaN the positive one of all ones.
__device__ __forceinline__ unsigned key_of(float v) {
    const unsigned u = __float_as_uint(__fadd_rn(v, 0.f));
    return u ^ (static_cast<unsigned>(static_cast<int>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned k) {
    return __uint_as_float(k ^ (static_cast<unsigned>(static_cast<int>(~k) >> 31) | 0x80000000u));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// A candidate: its expert in the low half (complemented: of equal keys the lower
// index is the larger number), its key above.
using Cand = unsigned long long;
__device__ __forceinline__ Cand cand_of(unsigned key, int e) { return static_cast<Cand>(key) << 32 | static_cast<unsigned>(~e); }
__device__ __forceinline__ unsigned key_in(Cand q) { return static_cast<unsigned>(q >> 32); }
__device__ __forceinline__ int expert_in(Cand q) { return static_cast<int>(~static_cast<unsigned>(q)); }

__device__ __forceinline__ float logit(const RouteArgs& a, int64_t t, int e) {
    const int64_t i = t * a.stride + e;
    return a.dtype == QMM_F32   ? static_cast<const float*>(a.logits)[i]
           : a.dtype == QMM_F16 ? __half2float(static_cast<const __half*>(a.logits)[i])
                                : __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[i]);
}

// ---- in 64 bits, for the few tokens that need it. What they take is felt at the end of
// every call of some thousand tokens, all of which run at once, and is mostly the
// fetching of code that ran nowhere before: hence a short exponential and quotient (exp64.cuh).

// The sum of a row's exponentials relative to its largest logit `top`, inverted.
__device__ __noinline__ double sum64(const RouteArgs& a, int64_t t, float top) {
    if (a.score == QMM_SCORE_SIGMOID || top == -INFINITY) return 1.0;
    double s = 0.0;
    for (int e = threadIdx.x % 32; e < a.E; e += 32) {
        const double x = static_cast<double>(logit(a, t, e)) - top;
        s += x >= -700.0 ? exp_mid(x) : isnan(x) ? x : 0.0;
    }
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    return inverse(s);
}
__device__ __noinline__ double value64(const RouteArgs& a, int64_t t, int e, float top, double by_sum) {
    const double x = logit(a, t, e), b = a.bias ? a.bias[e] : 0.0;
    if (a.score == QMM_SCORE_SIGMOID) {
        if (fabs(x) <= 80.0) return inverse(1.0 + exp_mid(-x)) + b;
        return 1.0 / (1.0 + exp(-x)) + b;
    }
    const double y = x - top;
    return (top == -INFINITY ? 0.0 : (y >= -700.0 ? exp_mid(y) : exp(y)) * by_sum) + b;
}
// Keys of doubles as key_of's of floats.
__device__ __forceinline__ unsigned long long key64(double v) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v + 0.0));
    return isnan(v) ? ~0ull : u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
// c in fp32.
__device__ __forceinline__ float score32(bool softmax, float x, float top, float sum) {
    if (!softmax) return __fdividef(1.f, 1.f + __expf(-x));
    return top == -INFINITY ? 0.f : __fdividef(__expf(x - top), sum);
}
// A chosen expert's sigmoid, times e^-at, at <= 0.
__device__ __forceinline__ float sigmoid_from(float x, float at) {
    const float e = expf(-fabsf(x));
    return (x < 0.f ? (at < 0.f ? expf(x - at) : e) : 1.f) / (1.f + e);
}
// Renormalised sigmoids below 2^-11 are taken relative to the largest chosen one's logit: what its
// exponential would take out of fp32's range drops out of the quotient.
__device__ __forceinline__ float sigmoid_at(float top) { return top < -8.f && top > -INFINITY ? top : 0.f; }
// Twice its error at magnitude |c| (see route_token), from its part at c = 0.
__device__ __forceinline__ float tau_of(float base, float v) { return base + 2.384185791015625e-07f * fabsf(v); }   // 2^-22

// Whether q may come before p, which has the larger or an equal fp32 value: where that is near,
// unless the inputs are the same.
enum Near { kFar, kNear, kSame };
__device__ __forceinline__ Near near_of(const RouteArgs& a, int64_t t, float base, Cand p, Cand q) {
    const float v = value_of(key_in(p));
    if (!(v - value_of(key_in(q)) <= tau_of(base, v))) return kFar;
    const int e = expert_in(p), f = expert_in(q);
    return logit(a, t, e) != logit(a, t, f) || a.bias[e] != a.bias[f] ? kNear : kSame;
}

// Whether any of this lane's candidates may.
__device__ __noinline__ bool near_behind(const RouteArgs& a, int64_t t, float base, Cand p, const Cand* cand, int i, int step, int n) {
    bool any = false;
    for (; i < n; i += step) any |= cand[i] < p && near_of(a, t, base, p, cand[i]) == kNear;
    return any;
}

// What a group's value is off by at most, with some room: a sum of two by as much as
// both, whatever is left of them, and by its rounding. Infinite values are not off, and those of
// equal ones (and NaN) that stay are the first, as in 64 bits.
__device__ __forceinline__ float group_off(float base, int group_top, unsigned m1, unsigned m2) {
    const float v1 = value_of(m1), v2 = group_top == 2 ? value_of(m2) : 0.f;
    return isinf(v1) || isinf(v2) ? 0.f : tau_of(base, fabsf(v1) + fabsf(v2));
}

// The groups that stay, as bits; 16 bytes of `mem` an expert. Of all c in fp32 only the
// few that may be among a group's group_top largest are computed, a lane for each.
__device__ __noinline__ unsigned groups64(const RouteArgs& a, int64_t t, float top, float sum, float base, uint8_t* mem) {
    const int lane = threadIdx.x % 32, gs = a.E / a.groups;
    float* c = reinterpret_cast<float*>(mem);
    int* list = reinterpret_cast<int*>(c + a.E);
    double* value = reinterpret_cast<double*>(mem) + a.E;
    const double by_sum = sum64(a, t, top);
    for (int first = 0; first < a.E; first += 256) {      // eight loads in flight
        float x[8], b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = min(first + 32 * i + lane, a.E - 1);
            x[i] = logit(a, t, e);
            b[i] = a.bias ? a.bias[e] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = first + 32 * i + lane;
            const float s = score32(a.score == QMM_SCORE_SOFTMAX, x[i], top, sum);
            if (e < a.E) c[e] = a.bias ? s + b[i] : s;
            if (e < a.E) value[e] = -INFINITY;
        }
    }
    __syncwarp();
    float least = INFINITY;                               // what one of the group's largest has at least in fp32
    if (lane < a.groups) {
        float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll 8
        for (int i = 0; i < gs; ++i) {
            const float b = c[lane * gs + i];
            m2 = fmaxf(m2, fminf(m1, b));
            m1 = fmaxf(m1, b);
        }
        least = a.group_top == 2 ? m2 : m1;
        least -= tau_of(base, least);
    }
    int n = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane;
        const float from = __shfl_sync(kAll, least, min(e, a.E - 1) / gs);
        const bool in = e < a.E && !(c[min(e, a.E - 1)] < from);
        const unsigned b = __ballot_sync(kAll, in);
        if (in) list[n + __popc(b & ((1u << lane) - 1u))] = e;
        n += __popc(b);
    }
    __syncwarp();
    for (int i = lane; i < n; i += 32) value[list[i]] = value64(a, t, list[i], top, by_sum);
    __syncwarp();
    double w = -INFINITY;
    if (lane < a.groups) {
        double m1 = -INFINITY, m2 = -INFINITY;
        bool bad = false;                                 // a NaN: the largest
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const int e = list[i];
            const double b = e / gs == lane ? value[e] : -INFINITY;
            bad |= isnan(b);
            m2 = b > m1 ? m1 : b > m2 ? b : m2;
            m1 = b > m1 ? b : m1;
        }
        w = bad ? NAN : a.group_top == 2 ? m1 + m2 : m1;
    }
    const unsigned long long k = lane < a.groups ? key64(w) : 0ull;
    int place = 0;
    for (int g = 0; g < a.groups; ++g) {
        const unsigned long long other = __shfl_sync(kAll, k, g);
        place += other > k || (other == k && g < lane);
    }
    __syncwarp();
    return __ballot_sync(kAll, lane < a.groups && place < a.top_groups);
}
// The top_k of n candidates, into `sorted`.
__device__ __noinline__ void places64(const RouteArgs& a, int64_t t, float top, const Cand* cand, unsigned long long* value, int n, Cand* sorted) {
    const int lane = threadIdx.x % 32;
    const double by_sum = sum64(a, t, top);
    for (int i = lane; i < n; i += 32) value[i] = key64(value64(a, t, expert_in(cand[i]), top, by_sum));
    __syncwarp();
    for (int i = lane; i < n; i += 32) {
        const Cand me = cand[i];
        const unsigned long long w = value[i];
        int place = 0;
        for (int j = 0; j < n; ++j)                       // of equal ones the lower index
            place += value[j] > w || (value[j] == w && static_cast<unsigned>(cand[j]) > static_cast<unsigned>(me));
        if (place < a.top_k) sorted[place] = me;
    }
    __syncwarp();
}

// V consecutive values of a row from e0 on, -Inf past n.
template <int V, typename T> __device__ __forceinline__ void load_row(const T* p, int e0, int n, bool wide, float (&x)[V]) {
    constexpr int PER = 16 / static_cast<int>(sizeof(T)), N = V < PER ? V : PER;
    if (wide) {                      // V divides n and the addresses are aligned
        Vec<T, N> v[V / N];
        if (e0 < n) {
#pragma unroll
            for (int i = 0; i < V / N; ++i) v[i].load(p + e0 + i * N);
#pragma unroll
            for (int i = 0; i < V / N; ++i) {
                float f[N];
                v[i].get(f);
#pragma unroll
                for (int j = 0; j < N; ++j) x[i * N + j] = f[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = e0 + i < n ? to_f32<T>(p[e0 + i]) : -INFINITY;
    }
}

// Shared memory of a warp: the candidates (padded to fours), and for BY_SCORE as many doubles; then the chosen.
__host__ __device__ constexpr int cands_of(int E) { return (E + 3) / 4 * 4; }
__host__ __device__ constexpr size_t warp_bytes(int E, bool by_score) {
    return static_cast<size_t>(cands_of(E)) * (by_score ? 16 : 8) + (kMaxTopK + 2) * 8;
}

// One token by a whole warp.
template <int V, typename T, bool BY_SCORE>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, bool wide, uint8_t* smem) {
    const int lane = threadIdx.x % 32;
    Cand* cand = reinterpret_cast<Cand*>(smem);
    double* value = reinterpret_cast<double*>(cand + cands_of(a.E));
    Cand* sorted = cand + cands_of(a.E) * (BY_SCORE ? 2 : 1);
    const int e0 = lane * V;
    float x[V];
    load_row<V, T>(static_cast<const T*>(a.logits) + t * a.stride, e0, a.E, wide, x);
    const bool softmax = a.score == QMM_SCORE_SOFTMAX, biased = BY_SCORE && a.bias != nullptr;

    // ---- the softmax's largest logit and sum, where scores are asked for
    float top = 0.f, sum = 1.f;
    if (softmax && (BY_SCORE || !a.renorm)) {
        unsigned m = key_of(x[0]);
#pragma unroll
        for (int i = 1; i < V; ++i) m = max(m, key_of(x[i]));
        top = value_of(__reduce_max_sync(kAll, m));
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s += top == -INFINITY ? 0.f : __expf(x[i] - top);
        s = warp_sum(s);
        sum = top == -INFINITY ? 1.f : s;
    }
    // ---- c in fp32, as keys (the logits themselves where their order is the scores')
    unsigned key[V];
    [[maybe_unused]] float base = 0.f;
    // Twice the error of a c of magnitude |c|. A sigmoid's exponential (2 + 1.2 |x| ulp), its 1 + e
    // (1/2) and its quotient (2) put it off by 1.8 2^-23 at most, their largest parts not
    // falling together: twice that is below 2^-21. Two softmax scores, relative to the
    // largest, 1 / sum, are off from one another by 2 2^-23 from their exponentials, up to 4 from their
    // quotients, and where one is far below the other by a common factor: the sum's V + 5
    // roundings, half each, and up to 7 from its small exponentials; 8.4 in all for 32
    // experts, 27 for 1024. The sum with the bias: 2^-24 |c|.
    auto tau = [&](float v) { return tau_of(base, v); };
    if constexpr (BY_SCORE) {
        base = softmax ? static_cast<float>(V + 12) * 1.1920928955078125e-07f / sum : 4.76837158203125e-07f;   // 2^-23, 2^-21
        float bias[V];
        if (biased) load_row<V, float>(a.bias, e0, a.E, wide, bias);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float s = score32(softmax, x[i], top, sum);
            key[i] = key_of(biased ? s + bias[i] : s);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key_of(x[i]);
    }

    // ---- groups
    unsigned kept = kAll;
    if (a.groups > 1) {
        const int gs = a.E / a.groups;
        // a lane for each group: its one or two largest c, summed
        unsigned m1, m2 = 0u;
        auto take = [&](unsigned b) {
            m2 = max(m2, min(m1, b));
            m1 = max(m1, b);
        };
        const int lanes = gs / V;
        if (gs == lanes * V && (lanes & (lanes - 1)) == 0) {   // whole lanes, a power of two of them
            m1 = key[0];
#pragma unroll
            for (int i = 1; i < V; ++i) take(key[i]);
            for (int o = 1; o < lanes; o <<= 1) {
                const unsigned b1 = __shfl_xor_sync(kAll, m1, o), b2 = __shfl_xor_sync(kAll, m2, o);
                take(b1);
                m2 = max(m2, b2);
            }
            m1 = __shfl_sync(kAll, m1, (lane * lanes) & 31);
            m2 = __shfl_sync(kAll, m2, (lane * lanes) & 31);
        } else {
            unsigned* all = reinterpret_cast<unsigned*>(cand);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e0 + i < a.E) all[e0 + i] = key[i];
            __syncwarp();
            const int at = lane < a.groups ? lane * gs : 0;
            m1 = all[at];
            for (int i = 1; i < gs; ++i) take(all[at + i]);
            __syncwarp();
        }
        const bool mine = lane < a.groups;
        const unsigned k = !mine ? 0u : a.group_top == 2 ? key_of(value_of(m1) + value_of(m2)) : m1;
        int place = 0;
        for (int g = 0; g < a.groups; ++g) {
            const unsigned other = __shfl_sync(kAll, k, g);
            place += other > k || (other == k && g < lane);
        }
        kept = __ballot_sync(kAll, mine && place < a.top_groups);
        if (BY_SCORE && a.top_groups < a.groups) {
            const float v = value_of(k), off = group_off(base, a.group_top, m1, m2);
            const float lo = value_of(__reduce_min_sync(kAll, kept >> lane & 1 ? key_of(v - off) : kAll));
            const float hi = value_of(__reduce_max_sync(kAll, mine && !(kept >> lane & 1) ? key_of(v + off) : 0u));
            if (lo <= hi && fabsf(hi) < INFINITY) kept = groups64(a, t, top, sum, base, smem);
        }
        // those that do not stay: key 0
        int g = e0 / gs, left = gs - (e0 - g * gs);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (e0 + i >= a.E || !(kept >> (g & 31) & 1)) key[i] = 0u;
            else if (BY_SCORE && !biased) key[i] = key_of(x[i]);
            if (--left == 0) {
                ++g;
                left = gs;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e0 + i >= a.E) key[i] = 0u;
    }

    // ---- 1. the bound
    unsigned most = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) most = max(most, key[i]);
    unsigned bound = 0u;
#pragma unroll 4
    for (int r = 0; r < a.top_k; ++r) {
        bound = __reduce_max_sync(kAll, most);
        most = most == bound ? 0u : most;
    }
    bound = max(bound, 1u);
    if (biased) {                                         // all that may be the top_k-th by more exact values
        const float v = value_of(bound);
        if (bound != 1u && !isnan(v)) bound = min(bound, max(1u, key_of(v - tau(v))));
    }
    // ---- 2. the candidates
    int count = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) count += key[i] >= bound;
    int scan = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kAll, scan, o);
        if (lane >= o) scan += up;
    }
    int n = __shfl_sync(kAll, scan, 31);
    if (n <= 64 || biased) {
        int at = scan - count;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] >= bound) cand[at++] = cand_of(key[i], e0 + i);
    } else {
        // many equal keys at the bound (a row of padding), and keys are exact: the first top_k of those
        unsigned both = 0u;                               // above the bound; equal to it in the upper half
#pragma unroll
        for (int i = 0; i < V; ++i) both += key[i] > bound ? 1u : key[i] == bound ? 0x10000u : 0u;
        unsigned sum2 = both;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned up = __shfl_up_sync(kAll, sum2, o);
            if (lane >= o) sum2 += up;
        }
        const unsigned total = __shfl_sync(kAll, sum2, 31);
        const int above = static_cast<int>(total & 0xffffu), equal = min(static_cast<int>(total >> 16), a.top_k);
        unsigned at = sum2 - both;
#pragma unroll 1
        for (int i = 0; i < V; ++i) {
            unsigned k = key[0];
#pragma unroll
            for (int j = 1; j < V; ++j) k = i == j ? key[j] : k;
            const int nth = static_cast<int>(at >> 16);
            if (k > bound) cand[at & 0xffffu] = cand_of(k, e0 + i);
            else if (k == bound && nth < equal) cand[above + nth] = cand_of(k, e0 + i);
            at += k > bound ? 1u : k == bound ? 0x10000u : 0u;
        }
        n = above + equal;
    }
    if (lane < 3 && n + lane < cands_of(a.E)) cand[n + lane] = 0u;
    __syncwarp();
    // ---- 3. their places; the first top_k (and the next) in `sorted`
    for (int i = lane; i < n; i += 32) {
        const Cand me = cand[i];
        int place = 0;
        for (int j = 0; j < n; j += 4) {
            const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(cand + j), q = *reinterpret_cast<const ulonglong2*>(cand + j + 2);
            place += (p.x > me) + (p.y > me) + (q.x > me) + (q.y > me);
        }
        if (place <= a.top_k) sorted[place] = me;
    }
    __syncwarp();
    const bool chosen = lane < a.top_k;
    if (biased) {
        Near near = kFar;
        if (chosen && lane + 1 < n) near = near_of(a, t, base, sorted[lane], sorted[lane + 1]);
        const bool run = near == kSame && lane + 1 == a.top_k;
        if (__any_sync(kAll, run || near == kNear)) {
            // behind a run of equal inputs at the end others may come
            bool close = near == kNear;
            if (__any_sync(kAll, run)) close |= near_behind(a, t, base, sorted[a.top_k - 1], cand, lane, 32, n);
            if (__any_sync(kAll, close)) places64(a, t, top, cand, reinterpret_cast<unsigned long long*>(value), n, sorted);
        }
    }

    // ---- weights
    const Cand mine = sorted[chosen ? lane : 0];
    const int e = expert_in(mine);
    const float lx = biased ? logit(a, t, e) : value_of(key_in(mine));
    float w;
    auto most_chosen = [&] { return biased ? value_of(__reduce_max_sync(kAll, key_of(lx))) : value_of(key_in(sorted[0])); };
    if (softmax) {
        // renormalised, the row's sum falls out; relative to the largest chosen logit
        if (a.renorm) top = most_chosen();
        w = top == -INFINITY ? 0.f : expf(lx - top);
        if (!a.renorm) w /= sum;
        if (BY_SCORE && isnan(sum)) w = sum;              // by a logit that need not be among the chosen
    } else {
        w = sigmoid_from(lx, a.renorm && __any_sync(kAll, lx < -8.f) ? sigmoid_at(most_chosen()) : 0.f);
    }
    if (a.renorm) {
        float s = chosen ? w : 0.f;
        for (int o = 1; o < a.top_k; o <<= 1) s += __shfl_xor_sync(kAll, s, o);
        w = s == 0.f ? 0.f : softmax ? __fdividef(w, s) : w / s;   // (a softmax's s is 1 .. top_k)
    }
    if (chosen) {
        a.ids[t * a.top_k + lane] = e;
        a.weights[t * a.top_k + lane] = w * a.scale;
    }
}

template <int V, typename T, bool BY_SCORE>
__global__ void __launch_bounds__(256) k_route(const __grid_constant__ RouteArgs a, bool wide) {
    grid_dep_launch();
    grid_dep_wait();
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x / 32;
    const int64_t t = blockIdx.x * static_cast<int64_t>(blockDim.x / 32) + warp;
    if (t < a.T) route_token<V, T, BY_SCORE>(a, t, wide, smem + warp * warp_bytes(a.E, BY_SCORE));
}

// For the tokens that k_route_four leaves.
template <int V, typename T, bool BY_SCORE>
__device__ __noinline__ void route_again(const RouteArgs& a, int64_t t, uint8_t* smem) {
    route_token<V, T, BY_SCORE>(a, t, true, smem);
    __syncwarp();
}

// Four tokens a warp, eight lanes each, for top_k up to 8 and experts in 8 V that
// V divides: what a warp does together (the bound, the scan, the few lanes that count
// places and weigh) serves four tokens. Tokens whose candidates are many (equal
// keys) are left to the whole warp at the end.
constexpr int kFew = 32;                                  // candidates of a token
constexpr int kFourBytes = (4 * (kFew + 10) + kFew) * 8;  // of a warp: candidates, the chosen and the next, values in 64 bits
constexpr int kFourTopK = 8;

__device__ __forceinline__ unsigned max8(unsigned v) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

template <int V, typename T, bool BY_SCORE>
__global__ void __launch_bounds__(256, V > 16 ? 2 : 4) k_route_four(const __grid_constant__ RouteArgs a) {
    grid_dep_launch();
    grid_dep_wait();
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, seg = lane / 8, sl = lane % 8;
    const size_t bytes = max(warp_bytes(a.E, BY_SCORE), static_cast<size_t>(kFourBytes));
    uint8_t* mem = smem + warp * bytes;
    Cand* cand = reinterpret_cast<Cand*>(mem) + seg * kFew;
    Cand* sorted = reinterpret_cast<Cand*>(mem) + 4 * kFew + seg * 10;
    const int64_t t0 = (blockIdx.x * static_cast<int64_t>(blockDim.x / 32) + warp) * 4;
    if (t0 >= a.T) return;
    const int64_t t = imin64(t0 + seg, a.T - 1);
    const int e0 = sl * V;
    float x[V];
    load_row<V, T>(static_cast<const T*>(a.logits) + t * a.stride, e0, a.E, true, x);
    const bool softmax = a.score == QMM_SCORE_SOFTMAX, biased = BY_SCORE && a.bias != nullptr;
    bool leave = false;

    float top = 0.f, sum = 1.f;
    if (softmax && (BY_SCORE || !a.renorm)) {
        unsigned m = key_of(x[0]);
#pragma unroll
        for (int i = 1; i < V; ++i) m = max(m, key_of(x[i]));
        top = value_of(max8(m));
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s += top == -INFINITY ? 0.f : __expf(x[i] - top);
        s = sum8(s);
        sum = top == -INFINITY ? 1.f : s;
    }
    unsigned key[V];
    [[maybe_unused]] float base = 0.f;
    auto tau = [&](float v) { return tau_of(base, v); };
    if constexpr (BY_SCORE) {
        base = softmax ? static_cast<float>(V + 12) * 1.1920928955078125e-07f / sum : 4.76837158203125e-07f;
        float bias[V];
        if (biased) load_row<V, float>(a.bias, e0, a.E, true, bias);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float s = score32(softmax, x[i], top, sum);
            key[i] = key_of(biased ? s + bias[i] : s);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key_of(x[i]);
    }
    bool mine = e0 < a.E;
    if (a.groups > 1) {
        // groups of whole lanes, a power of two of them
        const int lanes = a.E / a.groups / V;
        unsigned m1 = key[0], m2 = 0u;
#pragma unroll
        for (int i = 1; i < V; ++i) {
            m2 = max(m2, min(m1, key[i]));
            m1 = max(m1, key[i]);
        }
        for (int o = 1; o < lanes; o <<= 1) {
            const unsigned b1 = __shfl_xor_sync(kAll, m1, o), b2 = __shfl_xor_sync(kAll, m2, o);
            m2 = max(max(m2, b2), min(m1, b1));
            m1 = max(m1, b1);
        }
        const unsigned k = !mine ? 0u : a.group_top == 2 ? key_of(value_of(m1) + value_of(m2)) : m1;
        int place = 0;
        for (int from = 0; from < 8; from += lanes) {     // (lanes past the experts have 0)
            const unsigned other = __shfl_sync(kAll, k, from, 8);
            place += other > k || (other == k && from + lanes <= sl);
        }
        bool stays = mine && place < a.top_groups;
        if (BY_SCORE && a.top_groups < a.groups) {
            const float v = value_of(k), off = group_off(base, a.group_top, m1, m2);
            const float lo = value_of(~max8(stays ? ~key_of(v - off) : 0u));
            const float hi = value_of(max8(mine && !stays ? key_of(v + off) : 0u));
            const bool near = lo <= hi && fabsf(hi) < INFINITY;
            for (unsigned redo = __ballot_sync(kAll, near && sl == 0); redo; redo &= redo - 1u) {
                // by the whole warp, whose shared memory holds nothing yet
                const int from = __ffs(static_cast<int>(redo)) - 1;
                const unsigned kept = groups64(a, imin64(t0 + from / 8, a.T - 1), __shfl_sync(kAll, top, from), __shfl_sync(kAll, sum, from),
                                               __shfl_sync(kAll, base, from), mem);
                if (lane / 8 == from / 8) stays = mine && (kept >> (sl / lanes) & 1);
            }
        }
        mine = stays;
        if (BY_SCORE && !biased) {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = key_of(x[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = mine ? key[i] : 0u;

    // ---- 1. the bound: of the largest values of the lanes' quarters, in order in each lane
    unsigned m[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        m[q] = key[q * (V / 4)];
#pragma unroll
        for (int i = 1; i < V / 4; ++i) m[q] = max(m[q], key[q * (V / 4) + i]);
    }
    auto order = [&](int i, int j) {
        const unsigned hi = max(m[i], m[j]);
        m[j] = min(m[i], m[j]);
        m[i] = hi;
    };
    order(0, 1);
    order(2, 3);
    order(0, 2);
    order(1, 3);
    order(1, 2);
    unsigned bound = 0u;
    for (int r = 0; r < a.top_k; ++r) {
        bound = max8(m[0]);
        if (m[0] == bound) {
            m[0] = m[1];
            m[1] = m[2];
            m[2] = m[3];
            m[3] = 0u;
        }
    }
    bound = max(bound, 1u);
    if (biased) {
        const float v = value_of(bound);
        if (bound != 1u && !isnan(v)) bound = min(bound, max(1u, key_of(v - tau(v))));
    }
    // ---- 2. the candidates
    int count = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) count += key[i] >= bound;
    int scan = count;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const int up = __shfl_up_sync(kAll, scan, o, 8);
        if (sl >= o) scan += up;
    }
    int n = __shfl_sync(kAll, scan, 7, 8);
    leave |= n > kFew;
    if (!leave) {
        int at = scan - count;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] >= bound) cand[at++] = cand_of(key[i], e0 + i);
        if (sl == 0 && (n & 1)) cand[n] = 0u;
    } else {
        n = 0;
    }
    __syncwarp();
    // ---- 3. their places
    auto places = [&](auto rounds) {
        constexpr int R = decltype(rounds)::value;
        Cand me[R];
        int place[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            me[r] = cand[min(sl + 8 * r, kFew - 1)];
            place[r] = 0;
        }
        for (int j = 0; j < n; j += 2) {
            const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(cand + j);
#pragma unroll
            for (int r = 0; r < R; ++r) place[r] += (q.x > me[r]) + (q.y > me[r]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (sl + 8 * r < n && place[r] <= a.top_k) sorted[place[r]] = me[r];
    };
    if (__any_sync(kAll, n > 16)) places(std::integral_constant<int, 4>{});
    else places(std::integral_constant<int, 2>{});
    __syncwarp();
    const bool chosen = sl < a.top_k;
    if (biased) {
        bool close = false, run = false;
        if (chosen && sl + 1 < n) {
            const Near near = near_of(a, t, base, sorted[sl], sorted[sl + 1]);
            close = near == kNear;
            run = near == kSame && sl + 1 == a.top_k;
        }
        if (__ballot_sync(kAll, run) >> (seg * 8) & 0xffu) {   // what is behind a run of equal inputs at the end
            close |= near_behind(a, t, base, sorted[a.top_k - 1], cand, sl, 8, n);
        }
        unsigned redo = __ballot_sync(kAll, close && !leave);
        redo = (redo | redo >> 4) & 0x0f0f0f0fu;
        redo = (redo | redo >> 2) & 0x03030303u;
        redo = (redo | redo >> 1) & 0x01010101u;          // a bit for each token
        for (; redo; redo &= redo - 1u) {
            const int from = __ffs(static_cast<int>(redo)) - 1;
            const int64_t tq = imin64(t0 + from / 8, a.T - 1);
            places64(a, tq, __shfl_sync(kAll, top, from), reinterpret_cast<Cand*>(mem) + from / 8 * kFew,
                     reinterpret_cast<unsigned long long*>(mem) + 4 * (kFew + 10), __shfl_sync(kAll, n, from),
                     reinterpret_cast<Cand*>(mem) + 4 * kFew + from / 8 * 10);
        }
    }

    // ---- weights
    const Cand own = sorted[chosen && !leave ? sl : 0];
    const int e = leave ? 0 : expert_in(own);
    const float lx = leave ? 0.f : biased ? logit(a, t, e) : value_of(key_in(own));
    float w;
    auto most_chosen = [&] { return biased ? value_of(max8(chosen ? key_of(lx) : 0u)) : value_of(key_in(sorted[0])); };
    if (softmax) {
        if (a.renorm) top = most_chosen();
        w = top == -INFINITY ? 0.f : expf(lx - top);
        if (!a.renorm) w /= sum;
        if (BY_SCORE && isnan(sum)) w = sum;              // by a logit that need not be among the chosen
    } else {
        w = sigmoid_from(lx, a.renorm && __any_sync(kAll, lx < -8.f) ? sigmoid_at(most_chosen()) : 0.f);
    }
    if (a.renorm) {
        const float s = sum8(chosen ? w : 0.f);
        w = s == 0.f ? 0.f : softmax ? __fdividef(w, s) : w / s;   // (a softmax's s is 1 .. top_k)
    }
    if (chosen && !leave && t0 + seg < a.T) {
        a.ids[t * a.top_k + sl] = e;
        a.weights[t * a.top_k + sl] = w * a.scale;
    }
    unsigned again = __ballot_sync(kAll, leave && sl == 0 && t0 + seg < a.T);
    for (; again; again &= again - 1u) {
        __syncwarp();
        route_again<V / 4, T, BY_SCORE>(a, t0 + (__ffs(static_cast<int>(again)) - 1) / 8, mem);
    }
}

// Warps of a block: what fits 48 KB, at most eight, fewer where that fills more SMs.
int block_warps(int64_t warps, size_t bytes, int sms) {
    const int64_t per_sm = (warps + sms - 1) / sms;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({8, static_cast<int64_t>(49152 / bytes), per_sm})));
}

// V: experts a lane where a warp takes a token.
template <int V, typename T, bool BY_SCORE> cudaError_t go(const RouteArgs& a, cudaStream_t s) {
    int dev = 0;
    cudaGetDevice(&dev);
    const int sms = sm_count(dev);
    const bool at16 = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0 &&
                      (a.T == 1 || a.stride * static_cast<int64_t>(sizeof(T)) % 16 == 0);
    if constexpr (V == 2 || V == 4 || V == 8) {
        // Four tokens a warp from 24 tokens an SM on (128 experts: 4800 tokens 3.1 us, a warp each 3.8;
        // 2400 2.7 and 2.8), by score from 40 on (256 experts in groups: 8192 tokens 11.9 and
        // 14.4 us, 4800 10.0 and 8.3); but not by score with 32 experts a lane and no groups,
        // where registers decide (sigmoids: 8192 tokens 11.0 and 9.3 us, 65536 58.4 and 52.7;
        // softmax: 20.1 and 18.3, 75.8 and 74.5).
        const int gs = a.E / a.groups, lanes = gs / (4 * V);
        const bool whole = a.groups == 1 || (gs == lanes * 4 * V && (lanes & (lanes - 1)) == 0);
        if (a.top_k <= kFourTopK && a.E % (4 * V) == 0 && at16 && whole && !(BY_SCORE && V == 8 && a.groups == 1) &&
            a.T >= (BY_SCORE ? 40 : 24) * static_cast<int64_t>(sms)) {
            const size_t bytes = std::max(warp_bytes(a.E, BY_SCORE), static_cast<size_t>(kFourBytes));
            const int warps = block_warps((a.T + 3) / 4, bytes, sms);
            const int64_t blocks = (a.T + 4 * warps - 1) / (4 * warps);
            if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
            return launch_chained(k_route_four<4 * V, T, BY_SCORE>, dim3(static_cast<unsigned>(blocks)), warps * 32,
                                  static_cast<int>(warps * bytes), s, a);
        }
    }
    const size_t bytes = warp_bytes(a.E, BY_SCORE);
    const int warps = block_warps(a.T, bytes, sms);
    const int64_t blocks = (a.T + warps - 1) / warps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_chained(k_route<V, T, BY_SCORE>, dim3(static_cast<unsigned>(blocks)), warps * 32, static_cast<int>(warps * bytes), s, a,
                          at16 && a.E % V == 0);
}

template <int V, typename T> cudaError_t by(const RouteArgs& a, cudaStream_t s) {
    return a.bias || (a.groups > 1 && a.group_top == 2) ? go<V, T, true>(a, s) : go<V, T, false>(a, s);
}

template <typename T> cudaError_t pick(const RouteArgs& a, cudaStream_t s) {
    if (a.E <= 32) return by<1, T>(a, s);
    if (a.E <= 64) return by<2, T>(a, s);
    if (a.E <= 128) return by<4, T>(a, s);
    if (a.E <= 256) return by<8, T>(a, s);
    if (a.E <= 512) return by<16, T>(a, s);
    return by<32, T>(a, s);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
    if (a.dtype == QMM_F32) return pick<float>(a, s);
    if (a.dtype == QMM_F16) return pick<__half>(a, s);
    return pick<__nv_bfloat16>(a, s);
}

}  // namespace qmm
