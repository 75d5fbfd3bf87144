// k_kv.cu -- the paged key-value cache: rows written (qkv_store) and read back
// (qkv_load).
//
// A thread owns eight consecutive elements of a row; four neighbouring lanes
// own one 32-element block. Head dims are multiples of 32, so a block never
// straddles a row or a warp.
#include <algorithm>
#include <type_traits>

#include "quant.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int N = kQuantN;

// Eight q4_0 codes, and their block's scale from the lane that has its first.
__device__ __forceinline__ void put4(const KvCache& c, uint8_t* unit, int64_t row, int e, unsigned codes, __half d) {
    *reinterpret_cast<unsigned*>(unit + row * (c.D / 2) + e / 2) = codes;
    if (e % 32 == 0)
        reinterpret_cast<__half*>(unit + (static_cast<int64_t>(c.D / 2) << c.page_shift))[row * (c.D / 32) + e / 32] = d;
}

// Where a thread's eight elements of a row go: the same place in every head's
// unit (q4_0: put4). All 32 lanes of a warp call put8 together (quant8 shuffles); lanes with
// `writes` false write nothing.
template <int FMT>
__device__ __forceinline__ void put8(const KvCache& c, uint8_t* unit, int64_t row, int e, const float (&x)[N], bool writes) {
    if constexpr (FMT == QMM_KV_Q8_0) {
        uint2 codes;
        __half d;
        quant8(x, codes, d);
        if (!writes) return;
        *reinterpret_cast<uint2*>(unit + row * c.D + e) = codes;
        if (e % 32 == 0)
            reinterpret_cast<__half*>(unit + (static_cast<int64_t>(c.D) << c.page_shift))[row * (c.D / 32) + e / 32] = d;
    } else {
        if (!writes) return;
        using T = typename std::conditional<FMT == QMM_KV_F16, __half, __nv_bfloat16>::type;
        Vec<T, N> v;
        v.set(x);
        v.store(reinterpret_cast<T*>(unit) + row * c.D + e);
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

// An element's rotation. q4_0 keys are rotated operation by operation as a plain
// fp32 computation does it (rope_cs_plain, products rounded before their sum): their
// codes are an eighth of a block's largest value apart, and a difference in the
// last bit turns a few of ten million over, which are then the ones that such a
// computation stores.
template <int FMT> __device__ __forceinline__ void angle_of(int32_t pos, uint64_t turns, float mscale, float& c, float& s) {
    if constexpr (FMT == QMM_KV_Q4_0) rope_cs_plain(pos, turns, mscale, c, s);
    else rope_cs(pos, turns, mscale, c, s);
}
// x c + y s
template <int FMT> __device__ __forceinline__ float turned(float x, float c, float y, float s) {
    if constexpr (FMT == QMM_KV_Q4_0) return __fadd_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    else return x * c + y * s;
}

// Where a token's rows go.
struct Place {
    uint8_t* base;               // its page
    int64_t row;
    bool writes;                 // a slot of the cache (-1 skips, others are errors)
};
__device__ __forceinline__ Place place_of(const KvStoreArgs& a, int64_t t, bool is_v, bool active, bool reports) {
    const int64_t slot = a.slots[t];
    const bool bad = slot < -1 || slot >= (a.c.n_pages << a.c.page_shift);
    if (bad && active && reports) atomicOr(a.err, DEV_ERR_BAD_SLOT);
    Place p;
    p.writes = active && !bad && slot >= 0;
    p.row = p.writes ? slot & ((1ll << a.c.page_shift) - 1) : 0;
    p.base = (is_v ? a.c.v : a.c.k) + (p.writes ? slot >> a.c.page_shift : 0) * a.c.page_stride;
    return p;
}

// Whether a thread issues the next heads' loads before it quantises and writes these.
// (q4_0, 16384 x 8 x 128 rotated: fp32 32.7 us, 34.3 without; f16 27.2 and 27.9. The issue slots
// are busy half of the time, fp32 waits for its loads, f16 for its own instructions.)
template <int FMT> constexpr bool kPrefetch = FMT == QMM_KV_Q4_0;

// The usual rotation: half layout, whole heads, dims a multiple of 64, aligned.
// One thread owns eight elements of a head's first half and their partners, of
// `heads_per` heads of one token of K (blockIdx.y 0) or of V: every element
// is read once and a cos and sin serve two of them in every head. 16384 x 8 x
// 128 fp32 to q8_0: 38 us, against 45 with the partner reads of k_kv_store.
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads, 3) k_kv_store_pairs(KvStoreArgs a, int64_t threads, int head_groups, int heads_per) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t id0 = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    const bool active = id0 < threads;
    int vec, hg;
    int64_t r, t;
    div_mod(active ? id0 : threads - 1, a.c.D / (2 * N), r, vec);
    const int e = vec * N, half = a.c.D / 2;
    const bool is_v = blockIdx.y;
    div_mod(r, head_groups, t, hg);
    const int h0 = hg * heads_per, h1 = min(h0 + heads_per, a.c.heads);
    const Place at = place_of(a, t, is_v, active, e == 0);
    constexpr bool AHEAD = kPrefetch<FMT>;
    constexpr int kB = AHEAD ? 1 : 2;    // heads whose loads are in flight together
    const int64_t unit = a.c.unit();
    const T* x = static_cast<const T*>(is_v ? a.V : a.K) + t * (is_v ? a.v_ts : a.k_ts);
    const int64_t hs = is_v ? a.v_hs : a.k_hs;
    float c[N], s[N];
    // the last group repeats its last head: lanes stay together
    auto head = [&](int k) { return min(h0 + k, h1 - 1); };
    auto load = [&](int i, Vec<T, N> (&v0)[kB], Vec<T, N> (&v1)[kB]) {
#pragma unroll
        for (int k = 0; k < kB; ++k) {
            v0[k].load(x + head(i + k) * hs + e);
            v1[k].load(x + head(i + k) * hs + e + half);
        }
    };
    Vec<T, N> n0[kB], n1[kB];
    if constexpr (AHEAD) load(0, n0, n1);
#pragma unroll 1
    for (int i = 0; i < heads_per; i += kB) {
        Vec<T, N> v0[kB], v1[kB];
        if constexpr (AHEAD) {
#pragma unroll
            for (int k = 0; k < kB; ++k) {
                v0[k] = n0[k];
                v1[k] = n1[k];
            }
            if (i + kB < heads_per) load(i + kB, n0, n1);
        } else {
            load(i, v0, v1);
        }
        if (!is_v && i == 0) {           // behind the first loads
            const int32_t pos = a.pos[t];
#pragma unroll
            for (int j = 0; j < N; ++j) angle_of<FMT>(pos, a.turns[e + j], a.mscale, c[j], s[j]);
        }
#pragma unroll
        for (int k = 0; k < kB; ++k) {
            if (i + k >= heads_per) break;
            float f[2][N];
            float (&f0)[N] = f[0], (&f1)[N] = f[1];
            v0[k].get(f0);
            v1[k].get(f1);
            if (!is_v) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float y = FMT == QMM_KV_Q4_0 ? turned<FMT>(f0[j], c[j], f1[j], -s[j]) : f0[j] * c[j] - f1[j] * s[j];
                    f1[j] = turned<FMT>(f1[j], c[j], f0[j], s[j]);
                    f0[j] = y;
                }
            }
            uint8_t* to = at.base + head(i + k) * unit;
            if constexpr (FMT == QMM_KV_Q4_0) {
                unsigned codes[2];
                __half d[2];
                quant4<2>(f, codes, d);
                if (at.writes) {
                    put4(a.c, to, at.row, e, codes[0], d[0]);
                    put4(a.c, to, at.row, e + half, codes[1], d[1]);
                }
            } else {
                put8<FMT>(a.c, to, at.row, e, f0, at.writes);
                put8<FMT>(a.c, to, at.row, e + half, f1, at.writes);
            }
        }
    }
}

// One thread: eight elements of `heads_per` heads of one token, of K (blockIdx.y
// 0) or of V.
// Key elements are rotated as y_e = x_e cos a + sign x_partner sin a; the
// partner vector (half layout) is read through L1, which the lane that owns
// it reads too, so no row is staged and no lane waits for another.
template <typename T, int FMT, bool ALIGNED, bool ROPE>
__global__ void __launch_bounds__(kThreads, ROPE ? 3 : 5) k_kv_store(KvStoreArgs a, int64_t threads, int head_groups, int heads_per) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t id0 = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    const bool active = id0 < threads;
    int vec, hg;
    int64_t r, t;
    div_mod(active ? id0 : threads - 1, a.c.D / N, r, vec);
    const int e = vec * N;
    const bool is_v = blockIdx.y;        // keys and values in blocks of their own: one path a warp
    div_mod(r, head_groups, t, hg);
    const int h0 = hg * heads_per, h1 = min(h0 + heads_per, a.c.heads);
    const Place at = place_of(a, t, is_v, active, e == 0);
    constexpr int kB = ROPE || sizeof(T) == 4 ? 2 : 4;   // heads whose loads are in flight together
    const int64_t unit = a.c.unit();
    const bool turn = ROPE && !is_v && e < a.rot;
    const bool half = a.layout == QMM_ROPE_HALF;
    // all eight partners are one aligned vector
    const bool vec_pair = ALIGNED && half && a.rot % (2 * N) == 0;

    float c[N], s[N];
    const T* x = static_cast<const T*>(is_v ? a.V : a.K) + t * (is_v ? a.v_ts : a.k_ts);
    const int64_t hs = is_v ? a.v_hs : a.k_hs;
    const int partner = e < a.rot / 2 ? e + a.rot / 2 : e - a.rot / 2;
#pragma unroll 1
    for (int i = 0; i < heads_per; i += kB) {
        Vec<T, N> v[kB], w[kB];
        // the last group repeats its last head: lanes stay together
        auto head = [&](int k) { return min(h0 + i + k, h1 - 1); };
#pragma unroll
        for (int k = 0; k < kB; ++k) {
            const T* xh = x + head(k) * hs;
            if constexpr (ALIGNED) v[k].load(xh + e);
            else v[k].load_unaligned(xh + e);
            if (turn && vec_pair) w[k].load(xh + partner);
        }
        if (turn && i == 0) {               // behind the first loads
            const int32_t pos = a.pos[t];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                c[j] = 1.f;
                s[j] = 0.f;
                if (e + j < a.rot) {
                    int pair, other;
                    float sign;
                    pair_of(e + j, a.rot, half, pair, other, sign);
                    if (!half && (j & 1)) {          // the pair of the element before
                        c[j] = c[j - 1];
                        s[j] = -s[j - 1];
                    } else {
                        angle_of<FMT>(pos, a.turns[pair], a.mscale, c[j], s[j]);
                        s[j] *= sign;
                    }
                }
            }
        }
        auto rotated = [&](int k, float (&f)[N]) {
            v[k].get(f);
            if (turn) {
                float g[N];
                if (vec_pair) {
                    w[k].get(g);
                } else if (!half) {
#pragma unroll
                    for (int j = 0; j < N; ++j) g[j] = f[j ^ 1];
                } else {
                    const T* xh = x + head(k) * hs;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        int pair, other = e + j;
                        float sign;
                        if (e + j < a.rot) pair_of(e + j, a.rot, half, pair, other, sign);
                        g[j] = to_f32<T>(xh[other]);
                    }
                }
#pragma unroll
                for (int j = 0; j < N; ++j) f[j] = e + j < a.rot ? turned<FMT>(f[j], c[j], g[j], s[j]) : f[j];
            }
        };
        if constexpr (FMT == QMM_KV_Q4_0) {
#pragma unroll
            for (int k = 0; k < kB; k += 2) {            // two heads' blocks at once; the second may be a repetition
                if (i + k >= heads_per) break;
                float f[2][N];
                unsigned codes[2];
                __half d[2];
                rotated(k, f[0]);
                rotated(k + 1, f[1]);
                quant4<2>(f, codes, d);
                if (!at.writes) continue;
                put4(a.c, at.base + head(k) * unit, at.row, e, codes[0], d[0]);
                if (i + k + 1 < heads_per) put4(a.c, at.base + head(k + 1) * unit, at.row, e, codes[1], d[1]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kB; ++k) {
                if (i + k >= heads_per) break;
                float f[N];
                rotated(k, f);
                put8<FMT>(a.c, at.base + head(k) * unit, at.row, e, f, at.writes);
            }
        }
    }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) k_kv_load(KvLoadArgs a, int64_t threads, int head_groups, int heads_per) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t id = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    if (id >= threads) return;
    int vec, hg;
    int64_t r, t;
    div_mod(id, a.c.D / N, r, vec);
    const int e = vec * N;
    const bool is_v = blockIdx.y;
    div_mod(r, head_groups, t, hg);
    const int h0 = hg * heads_per, h1 = min(h0 + heads_per, a.c.heads);
    const int64_t slot = a.slots[t];
    const bool bad = slot < -1 || slot >= (a.c.n_pages << a.c.page_shift);
    if (bad && e == 0) atomicOr(a.err, DEV_ERR_BAD_SLOT);
    T* y = static_cast<T*>(is_v ? a.V : a.K) + t * a.c.heads * a.c.D + e;
    if (bad || slot < 0) {
        float f[N];
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] = bad ? NAN : 0.f;
        Vec<T, N> v;
        v.set(f);
        for (int h = h0; h < h1; ++h) v.store(y + static_cast<int64_t>(h) * a.c.D);
        return;
    }
    constexpr int kB = 4;                // heads whose loads are in flight together
    const int64_t row = slot & ((1ll << a.c.page_shift) - 1);
    const int64_t unit = a.c.unit();
    const uint8_t* base = (is_v ? a.c.v : a.c.k) + (slot >> a.c.page_shift) * a.c.page_stride;
    const int64_t row_bytes = kv_code_bytes(FMT, a.c.D);
    const int64_t at = FMT == QMM_KV_Q4_0 ? row * row_bytes + e / 2 : row * a.c.D + e;
    const int64_t scale_at = (row_bytes << a.c.page_shift) + (row * (a.c.D / 32) + e / 32) * 2;   // Q8_0, Q4_0
#pragma unroll 1
    for (int h = h0; h < h1; h += kB) {
        using S = typename std::conditional<FMT == QMM_KV_BF16, __nv_bfloat16, __half>::type;
        Vec<S, N> v[kB];
        uint2 w[kB];
        __half d[kB];
#pragma unroll
        for (int k = 0; k < kB; ++k) {
            const uint8_t* p = base + min(h + k, h1 - 1) * unit;
            if constexpr (FMT == QMM_KV_Q8_0) {
                w[k] = *reinterpret_cast<const uint2*>(p + at);
                d[k] = *reinterpret_cast<const __half*>(p + scale_at);
            } else if constexpr (FMT == QMM_KV_Q4_0) {
                w[k].x = *reinterpret_cast<const unsigned*>(p + at);
                d[k] = *reinterpret_cast<const __half*>(p + scale_at);
            } else {
                v[k].load(reinterpret_cast<const S*>(p) + at);
            }
        }
#pragma unroll
        for (int k = 0; k < kB; ++k) {
            if (h + k >= h1) break;
            float f[N];
            if constexpr (FMT == QMM_KV_Q8_0) {
                // code + 128 in the low byte of 2^23, less 2^23 + 128: exact
                const float df = __half2float(d[k]);
                const unsigned u[2] = {w[k].x ^ 0x80808080u, w[k].y ^ 0x80808080u};
#pragma unroll
                for (int j = 0; j < N; ++j)
                    f[j] = df * (__uint_as_float(__byte_perm(u[j / 4], 0x4b000000u, 0x7440 + j % 4)) - 8388736.f);
            } else if constexpr (FMT == QMM_KV_Q4_0) {
                // code + 8 in the low bits of 2^23, less 2^23 + 8: exact
                const float df = __half2float(d[k]);
#pragma unroll
                for (int j = 0; j < N; ++j) f[j] = df * (__uint_as_float((w[k].x >> (4 * j) & 15u) | 0x4b000000u) - 8388616.f);
            } else {
                v[k].get(f);
            }
            Vec<T, N> out;
            out.set(f);
            out.store(y + static_cast<int64_t>(h + k) * a.c.D);
        }
    }
}

struct Shape {
    int64_t threads;
    int64_t blocks;
    int groups, per;
};

// Heads per thread: as many as leave about four blocks of 256 threads per SM, at
// most eight; one where the call is small.
Shape shape(int64_t T, int heads, int D, int per_thread = N) {
    int dev = 0;
    cudaGetDevice(&dev);
    const int64_t want = static_cast<int64_t>(sm_count(dev)) * 4 * kThreads;
    const int64_t all = T * 2 * (D / per_thread) * heads;
    Shape s;
    s.per = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({heads, 8, all / want})));
    s.groups = (heads + s.per - 1) / s.per;
    s.threads = T * (D / per_thread) * s.groups;        // of keys, and as many of values
    s.blocks = (s.threads + kThreads - 1) / kThreads;
    return s;
}

template <typename T> cudaError_t store(const KvStoreArgs& a, cudaStream_t s) {
    const int64_t S = sizeof(T);
    const bool al = reinterpret_cast<uintptr_t>(a.K) % 16 == 0 && reinterpret_cast<uintptr_t>(a.V) % 16 == 0 &&
                    a.k_ts * S % 16 == 0 && a.k_hs * S % 16 == 0 && a.v_ts * S % 16 == 0 && a.v_hs * S % 16 == 0;
    const bool pairs = a.pos && al && a.layout == QMM_ROPE_HALF && a.rot == a.c.D && a.c.D % 64 == 0;
    const Shape g = shape(a.T, a.c.heads, a.c.D, pairs ? 2 * N : N);
    if (g.blocks > 0x7fffffff) return cudaErrorInvalidValue;
    auto go = [&](auto kernel) {
        return launch_chained(kernel, dim3(static_cast<unsigned>(g.blocks), 2), kThreads, 0, s, a, g.threads, g.groups, g.per);
    };
    auto pick = [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        if (pairs) return go(k_kv_store_pairs<T, F>);
        if (a.pos) return al ? go(k_kv_store<T, F, true, true>) : go(k_kv_store<T, F, false, true>);
        return al ? go(k_kv_store<T, F, true, false>) : go(k_kv_store<T, F, false, false>);
    };
    switch (a.c.fmt) {
    case QMM_KV_F16: return pick(std::integral_constant<int, QMM_KV_F16>{});
    case QMM_KV_BF16: return pick(std::integral_constant<int, QMM_KV_BF16>{});
    case QMM_KV_Q4_0: return pick(std::integral_constant<int, QMM_KV_Q4_0>{});
    default: return pick(std::integral_constant<int, QMM_KV_Q8_0>{});
    }
}

template <typename T> cudaError_t load(const KvLoadArgs& a, cudaStream_t s) {
    const Shape g = shape(a.T, a.c.heads, a.c.D);
    if (g.blocks > 0x7fffffff) return cudaErrorInvalidValue;
    auto go = [&](auto kernel) {
        return launch_chained(kernel, dim3(static_cast<unsigned>(g.blocks), 2), kThreads, 0, s, a, g.threads, g.groups, g.per);
    };
    switch (a.c.fmt) {
    case QMM_KV_F16: return go(k_kv_load<T, QMM_KV_F16>);
    case QMM_KV_BF16: return go(k_kv_load<T, QMM_KV_BF16>);
    case QMM_KV_Q4_0: return go(k_kv_load<T, QMM_KV_Q4_0>);
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
