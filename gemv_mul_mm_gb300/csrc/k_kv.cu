// k_kv.cu -- the paged key-value cache: rows written (qkv_store) and read back
// (qkv_load).
//
// A thread owns eight consecutive elements of a row; four neighbouring lanes
// own one 32-element block. Head dims are multiples of 32, so a block never
// straddles a row or a warp.
#include <algorithm>

#include "kv_common.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int N = 8;

// Elements [e, e + 8) of a row in fp32.
template <typename T, bool ALIGNED> __device__ __forceinline__ void load8(const T* p, float (&x)[N]) {
    if constexpr (ALIGNED) {
        load_vec<T, N>(p, x);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = to_f32<T>(p[j]);
    }
}

// Q8_0: d = f16(max |x| / 127), code = rint(x / d) in [-127, 127], each division
// rounded once; a block of zeros (or whose d underflows) has d = 0 and codes
// 0. A block that holds an Inf or NaN, or whose d overflows f16, gets d = NaN
// and reads back as NaN, so that a bad activation stays visible.
__device__ __forceinline__ void quant8(const float (&x)[N], uint2& codes, __half& d) {
    float amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        amax = fmaxf(amax, fabsf(x[j]));
        bad |= !isfinite(x[j]);
    }
    if (bad) amax = INFINITY;
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    d = __float2half_rn(__fdiv_rn(amax, 127.f));
    const float df = __half2float(d);
    const bool finite = isfinite(df);
    if (!finite) d = __ushort_as_half(0x7fff);
    unsigned w[2] = {0u, 0u};
    if (finite && df > 0.f) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int q = max(-127, min(127, __float2int_rn(__fdiv_rn(x[j], df))));
            w[j / 4] |= (static_cast<unsigned>(q) & 0xffu) << (8 * (j % 4));
        }
    }
    codes = make_uint2(w[0], w[1]);
}

// All 32 lanes of a warp call this together (quant8 shuffles); `active` lanes
// write.
template <int FMT>
__device__ __forceinline__ void put8(const KvCache& c, uint8_t* unit, int64_t row, int e, const float (&x)[N], bool active) {
    if constexpr (FMT == QMM_KV_Q8_0) {
        uint2 codes;
        __half d;
        quant8(x, codes, d);
        if (!active) return;
        *reinterpret_cast<uint2*>(unit + row * c.D + e) = codes;
        if (e % 32 == 0)
            reinterpret_cast<__half*>(unit + (static_cast<int64_t>(c.D) << c.page_shift))[row * (c.D / 32) + e / 32] = d;
    } else {
        if (!active) return;
        using T = typename std::conditional<FMT == QMM_KV_F16, __half, __nv_bfloat16>::type;
        store_vec<T, N>(reinterpret_cast<T*>(unit) + row * c.D + e, x);
    }
}

// Index e of the pair that element e belongs to, its partner element and the
// sign of the sine, in either layout (e < rot).
__device__ __forceinline__ void pair_of(int e, int rot, bool half, int& pair, int& partner, float& sign) {
    if (half) {
        const bool first = e < rot / 2;
        pair = first ? e : e - rot / 2;
        partner = first ? e + rot / 2 : e - rot / 2;
        sign = first ? -1.f : 1.f;
    } else {
        pair = e / 2;
        partner = e ^ 1;
        sign = e & 1 ? 1.f : -1.f;
    }
}

// One thread: eight elements of `heads_per` heads of one token, of K or of V.
// Key elements are rotated as y_e = x_e cos a + sign x_partner sin a; the
// partner vector (half layout) is read through L1, which the lane that owns
// it reads too, so no row is staged and no lane waits for another.
template <typename T, int FMT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_kv_store(KvStoreArgs a, int64_t threads, int head_groups, int heads_per) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t id0 = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    const bool active = id0 < threads;
    const int64_t id = active ? id0 : threads - 1;
    const int vecs = a.c.D / N;
    const int e = static_cast<int>(id % vecs) * N;
    int64_t r = id / vecs;
    const bool is_v = r & 1;
    r >>= 1;
    const int hg = static_cast<int>(r % head_groups);
    const int64_t t = r / head_groups;
    const int h0 = hg * heads_per, h1 = min(h0 + heads_per, a.c.heads);
    const int64_t slot = a.slots[t];
    const bool bad = slot < -1 || slot >= (a.c.n_pages << a.c.page_shift);
    if (bad && active && e == 0) atomicOr(a.err, DEV_ERR_BAD_SLOT);
    const bool writes = active && !bad && slot >= 0;
    const int64_t page = writes ? slot >> a.c.page_shift : 0;
    const int64_t row = writes ? slot & ((1ll << a.c.page_shift) - 1) : 0;
    uint8_t* base = (is_v ? a.c.v : a.c.k) + page * a.c.page_stride;
    const int64_t unit = a.c.unit();
    const bool turn = !is_v && a.pos && e < a.rot;
    const bool half = a.layout == QMM_ROPE_HALF;
    // all eight partners are one aligned vector
    const bool vec_pair = ALIGNED && half && a.rot % (2 * N) == 0;

    float c[N], s[N];
    if (turn) {
        const int32_t pos = a.pos[t];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            c[j] = 1.f;
            s[j] = 0.f;
            if (e + j < a.rot) {
                int pair, partner;
                float sign;
                pair_of(e + j, a.rot, half, pair, partner, sign);
                rope_cs(pos, a.turns[pair], a.mscale, c[j], s[j]);
                s[j] *= sign;
            }
        }
    }
    const T* x = static_cast<const T*>(is_v ? a.V : a.K) + t * (is_v ? a.v_ts : a.k_ts);
    const int64_t hs = is_v ? a.v_hs : a.k_hs;
#pragma unroll 4
    for (int i = 0; i < heads_per; ++i) {
        const int h = min(h0 + i, h1 - 1);   // the last group repeats its last head: lanes stay together
        const T* xh = x + h * hs;
        float v[N];
        load8<T, ALIGNED>(xh + e, v);
        if (turn) {
            float w[N];
            if (vec_pair) {
                load8<T, ALIGNED>(xh + (e < a.rot / 2 ? e + a.rot / 2 : e - a.rot / 2), w);
            } else if (!half) {
#pragma unroll
                for (int j = 0; j < N; ++j) w[j] = v[j ^ 1];
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    int pair, partner = e + j;
                    float sign;
                    if (e + j < a.rot) pair_of(e + j, a.rot, half, pair, partner, sign);
                    w[j] = to_f32<T>(xh[partner]);
                }
            }
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = e + j < a.rot ? v[j] * c[j] + w[j] * s[j] : v[j];
        }
        put8<FMT>(a.c, base + h * unit, row, e, v, writes);
    }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) k_kv_load(KvLoadArgs a, int64_t threads, int head_groups, int heads_per) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t id = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    if (id >= threads) return;
    const int vecs = a.c.D / N;
    const int e = static_cast<int>(id % vecs) * N;
    int64_t r = id / vecs;
    const bool is_v = r & 1;
    r >>= 1;
    const int hg = static_cast<int>(r % head_groups);
    const int64_t t = r / head_groups;
    const int h0 = hg * heads_per, h1 = min(h0 + heads_per, a.c.heads);
    const int64_t slot = a.slots[t];
    const bool bad = slot < -1 || slot >= (a.c.n_pages << a.c.page_shift);
    if (bad && e == 0) atomicOr(a.err, DEV_ERR_BAD_SLOT);
    T* y = static_cast<T*>(is_v ? a.V : a.K) + t * a.c.heads * a.c.D + e;
    if (bad || slot < 0) {
        float v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = bad ? NAN : 0.f;
        for (int h = h0; h < h1; ++h) store_vec<T, N>(y + static_cast<int64_t>(h) * a.c.D, v);
        return;
    }
    const int64_t row = slot & ((1ll << a.c.page_shift) - 1);
    const int64_t unit = a.c.unit();
    const uint8_t* base = (is_v ? a.c.v : a.c.k) + (slot >> a.c.page_shift) * a.c.page_stride;
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
        const uint8_t* p = base + h * unit;
        float v[N];
        if constexpr (FMT == QMM_KV_Q8_0) {
            const uint2 w = *reinterpret_cast<const uint2*>(p + row * a.c.D + e);
            const float d = __half2float(
                reinterpret_cast<const __half*>(p + (static_cast<int64_t>(a.c.D) << a.c.page_shift))[row * (a.c.D / 32) + e / 32]);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const unsigned word = j < 4 ? w.x : w.y;
                v[j] = d * static_cast<float>(static_cast<int8_t>(word >> (8 * (j % 4))));
            }
        } else {
            using S = typename std::conditional<FMT == QMM_KV_F16, __half, __nv_bfloat16>::type;
            load_vec<S, N>(reinterpret_cast<const S*>(p) + row * a.c.D + e, v);
        }
        store_vec<T, N>(y + static_cast<int64_t>(h) * a.c.D, v);
    }
}

struct Shape {
    int64_t threads;
    int64_t blocks;
    int groups, per;
};

// Heads per thread: as many as leave about four blocks of 256 threads per SM, at
// most eight; one where the call is small.
Shape shape(int64_t T, int heads, int D) {
    int dev = 0;
    cudaGetDevice(&dev);
    const int64_t want = static_cast<int64_t>(sm_count(dev)) * 4 * kThreads;
    const int64_t all = T * 2 * (D / N) * heads;
    Shape s;
    s.per = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({heads, 8, all / want})));
    s.groups = (heads + s.per - 1) / s.per;
    s.threads = T * 2 * (D / N) * s.groups;
    s.blocks = (s.threads + kThreads - 1) / kThreads;
    return s;
}

template <typename T> cudaError_t store(const KvStoreArgs& a, cudaStream_t s) {
    const Shape g = shape(a.T, a.c.heads, a.c.D);
    if (g.blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const int64_t S = sizeof(T);
    const bool al = reinterpret_cast<uintptr_t>(a.K) % 16 == 0 && reinterpret_cast<uintptr_t>(a.V) % 16 == 0 &&
                    a.k_ts * S % 16 == 0 && a.k_hs * S % 16 == 0 && a.v_ts * S % 16 == 0 && a.v_hs * S % 16 == 0;
    auto go = [&](auto kernel) {
        return launch_chained(kernel, dim3(static_cast<unsigned>(g.blocks)), kThreads, 0, s, a, g.threads, g.groups, g.per);
    };
    switch (a.c.fmt) {
    case QMM_KV_F16: return al ? go(k_kv_store<T, QMM_KV_F16, true>) : go(k_kv_store<T, QMM_KV_F16, false>);
    case QMM_KV_BF16: return al ? go(k_kv_store<T, QMM_KV_BF16, true>) : go(k_kv_store<T, QMM_KV_BF16, false>);
    default: return al ? go(k_kv_store<T, QMM_KV_Q8_0, true>) : go(k_kv_store<T, QMM_KV_Q8_0, false>);
    }
}

template <typename T> cudaError_t load(const KvLoadArgs& a, cudaStream_t s) {
    const Shape g = shape(a.T, a.c.heads, a.c.D);
    if (g.blocks > 0x7fffffff) return cudaErrorInvalidValue;
    auto go = [&](auto kernel) {
        return launch_chained(kernel, dim3(static_cast<unsigned>(g.blocks)), kThreads, 0, s, a, g.threads, g.groups, g.per);
    };
    switch (a.c.fmt) {
    case QMM_KV_F16: return go(k_kv_load<T, QMM_KV_F16>);
    case QMM_KV_BF16: return go(k_kv_load<T, QMM_KV_BF16>);
    default: return go(k_kv_load<T, QMM_KV_Q8_0>);
    }
}

}  // namespace

cudaError_t launch_kv_store(const KvStoreArgs& a, cudaStream_t s) {
    if (a.dtype == QMM_F32) return store<float>(a, s);
    if (a.dtype == QMM_F16) return store<__half>(a, s);
    return store<__nv_bfloat16>(a, s);
}

cudaError_t launch_kv_load(const KvLoadArgs& a, cudaStream_t s) {
    if (a.dtype == QMM_F32) return load<float>(a, s);
    if (a.dtype == QMM_F16) return load<__half>(a, s);
    return load<__nv_bfloat16>(a, s);
}

}  // namespace qmm
