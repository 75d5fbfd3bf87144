// k_norm.cu -- qrmsnorm: RMS norm of rows, with the residual's addition before it.
//
//   h = x + r,  r' = h,  y = h / sqrt(mean(h^2) + eps) * (w + o)
//
// Bound by reading x and r and writing r' and y once each: a row stays in
// registers between the sum of squares and the product. A thread holds
// vectors of N elements (eight, or one where a row's size, strides or addresses
// do not allow 16-byte accesses); short rows take part of a warp each, long ones
// a block each, and rows that no block can hold are read twice.
#include <algorithm>
#include <type_traits>

#include "layer_common.cuh"
#include "quant.cuh"

namespace qmm {
namespace {

constexpr int kWide = 256;       // threads of a block of short rows

__device__ __forceinline__ float warp_sum(float v, int width) {
    for (int o = width / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// How a row's N elements are reached. kVec: 16-byte accesses. kShift: rows of any
// size that begin anywhere, alike in all arrays (an odd D, contiguous): a thread's vectors
// lie on the arrays' 16-byte grid, `shift` elements before where they would, so that only
// the first and the last of a row are partial. kOne: one by one.
enum Mode { kOne, kVec, kShift };

// N elements as they lie in memory, of a type known at run time (a branch that
// a whole grid takes alike). Of elements e .. e + N - 1 of a row those outside it are zeros.
template <int N> struct Raw;
template <> struct Raw<8> {
    uint4 a, b;
    template <int MODE> __device__ __forceinline__ void load(const void* p, int64_t i, int dt, int64_t e, int64_t D) {
        if (MODE == kShift && (e < 0 || e + 8 > D)) {
            unsigned* u = &a.x;
            a = b = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (e + j < 0 || e + j >= D) continue;
                if (dt == QMM_F32) (j < 4 ? u[j] : (&b.x)[j - 4]) = static_cast<const unsigned*>(p)[i + j];
                else u[j / 2] |= static_cast<unsigned>(static_cast<const unsigned short*>(p)[i + j]) << (j % 2 * 16);
            }
        } else if constexpr (MODE != kOne) {
            if (dt == QMM_F32) {
                const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
                a = q[0];
                b = q[1];
            } else {
                a = *reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(p) + i);
            }
        } else {
            unsigned* u = &a.x;
            if (dt == QMM_F32) {
#pragma unroll
                for (int j = 0; j < 8; ++j) (j < 4 ? u[j] : (&b.x)[j - 4]) = static_cast<const unsigned*>(p)[i + j];
            } else {
                const unsigned short* q = static_cast<const unsigned short*>(p) + i;
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = q[2 * j] | static_cast<unsigned>(q[2 * j + 1]) << 16;
            }
        }
    }
    __device__ __forceinline__ void get(float (&x)[8], int dt) const {
        const unsigned w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (dt == QMM_F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
        } else if (dt == QMM_F16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                x[2 * j] = f.x;
                x[2 * j + 1] = f.y;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[2 * j] = __uint_as_float(w[j] << 16);
                x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    }
};
template <> struct Raw<1> {
    float v;
    template <int MODE> __device__ __forceinline__ void load(const void* p, int64_t i, int dt, int64_t, int64_t) {
        v = dt == QMM_F32   ? static_cast<const float*>(p)[i]
            : dt == QMM_F16 ? __half2float(static_cast<const __half*>(p)[i])
                            : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    }
    __device__ __forceinline__ void get(float (&x)[1], int) const { x[0] = v; }
};

template <int N, int MODE>
__device__ __forceinline__ void put(void* p, int64_t i, int dt, const float (&x)[N], int64_t e, int64_t D) {
    if (MODE != kOne && (MODE == kVec || (e >= 0 && e + N <= D))) {
        if (dt == QMM_F32) {
            Vec<float, N> v;
            v.set(x);
            v.store(static_cast<float*>(p) + i);
        } else if (dt == QMM_F16) {
            Vec<__half, N> v;
            v.set(x);
            v.store(static_cast<__half*>(p) + i);
        } else {
            Vec<__nv_bfloat16, N> v;
            v.set(x);
            v.store(static_cast<__nv_bfloat16*>(p) + i);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (MODE == kShift && (e + j < 0 || e + j >= D)) continue;
            if (dt == QMM_F32) static_cast<float*>(p)[i + j] = x[j];
            else if (dt == QMM_F16) static_cast<__half*>(p)[i + j] = __float2half_rn(x[j]);
            else static_cast<__nv_bfloat16*>(p)[i + j] = __float2bfloat16_rn(x[j]);
        }
    }
}

// Eight elements a lane as Q8_0 blocks: a warp's 256 elements are 272 bytes, put
// together in shared memory and written in the widest accesses their address
// allows. `to`: the bytes of the warp's first block; lanes from `lanes` on hold nothing.
__device__ __forceinline__ void put_q8(uint8_t* to, uint8_t* stage, int lane, int lanes, const float (&x)[8]) {
    uint2 codes;
    __half d;
    quant8(x, codes, d);
    unsigned short* s = reinterpret_cast<unsigned short*>(stage + lane / 4 * 34);
    if (lane % 4 == 0) s[0] = __half_as_ushort(d);
    s += 1 + lane % 4 * 4;
    s[0] = static_cast<unsigned short>(codes.x);
    s[1] = static_cast<unsigned short>(codes.x >> 16);
    s[2] = static_cast<unsigned short>(codes.y);
    s[3] = static_cast<unsigned short>(codes.y >> 16);
    __syncwarp();
    const int bytes = lanes / 4 * 34;
    if (reinterpret_cast<uintptr_t>(to) % 16 == 0 && bytes % 16 == 0) {
        for (int i = lane; i < bytes / 16; i += 32) reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(stage)[i];
    } else {
        for (int i = lane; i < bytes / 2; i += 32)
            reinterpret_cast<unsigned short*>(to)[i] = reinterpret_cast<const unsigned short*>(stage)[i];
    }
    __syncwarp();
}

struct Row {
    int64_t x, r, ro, y;
    int shift;                       // kShift: of the row's vectors
};
// (rows are below 2^31; row / H by a multiplication, see launch_norm)
__device__ __forceinline__ Row row_of(const NormArgs& a, int64_t row) {
    unsigned t = static_cast<unsigned>(row), h = 0;
    if (a.H > 1) {
        t = __umulhi(static_cast<unsigned>(row), a.h_mul) >> a.h_shift;
        h = static_cast<unsigned>(row) - t * static_cast<unsigned>(a.H);
    }
    auto at = [&](int64_t ts, int64_t hs) { return static_cast<int64_t>(t) * ts + static_cast<int64_t>(h) * hs; };
    Row r;
    r.x = at(a.x_ts, a.x_hs);
    r.y = at(a.y_ts, a.y_hs);
    r.r = r.ro = 0;
    if (a.R) {
        r.r = at(a.r_ts, a.r_hs);
        r.ro = at(a.ro_ts, a.ro_hs);
    }
    r.shift = static_cast<int>((r.x + a.x_shift) & 7);
    return r;
}

// weight + offset
template <int N, int MODE> __device__ __forceinline__ void weights(const NormArgs& a, int64_t e, float (&w)[N]) {
    if (!a.W) {
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = 1.f;
        return;
    }
    if constexpr (MODE == kVec) {
        Vec<float, N> v;
        v.load(a.W + e);
        v.get(w);
    } else if (MODE == kShift && a.w_at16 && e >= 0 && e - (e & 3) + 12 <= a.D) {
        // three aligned vectors around them; where they lie in those is alike for a whole row
        float f[12];
        Vec<float, 12> v;
        v.load(a.W + (e - (e & 3)));
        v.get(f);
        auto from = [&](auto first) {
#pragma unroll
            for (int j = 0; j < N; ++j) w[j] = f[(j + decltype(first)::value) % 12];
        };
        switch (e & 3) {
        case 0: from(std::integral_constant<int, 0>{}); break;
        case 1: from(std::integral_constant<int, 1>{}); break;
        case 2: from(std::integral_constant<int, 2>{}); break;
        default: from(std::integral_constant<int, 3>{});
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = MODE == kOne || (e + j >= 0 && e + j < a.D) ? a.W[e + j] : 0.f;
    }
    if (a.w_off != 0.f) {
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] += a.w_off;
    }
}

// Two elements in one instruction where there are two.
template <int N> __device__ __forceinline__ void add_to(float (&h)[N], const float (&f)[N]) {
    if constexpr (N == 1) {
        h[0] += f[0];
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 v = add2(make_float2(h[j], h[j + 1]), make_float2(f[j], f[j + 1]));
            h[j] = v.x;
            h[j + 1] = v.y;
        }
    }
}
template <int N> __device__ __forceinline__ float2 squares(const float (&h)[N], float2 s) {
    if constexpr (N == 1) {
        s.x = fmaf(h[0], h[0], s.x);
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 2) s = fma2(make_float2(h[j], h[j + 1]), make_float2(h[j], h[j + 1]), s);
    }
    return s;
}
// y = (h * inv) * w
template <int N> __device__ __forceinline__ void scale(float (&h)[N], float inv, const float (&w)[N]) {
    if constexpr (N == 1) {
        h[0] = h[0] * inv * w[0];
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 v = mul2(mul2(make_float2(h[j], h[j + 1]), make_float2(inv, inv)), make_float2(w[j], w[j + 1]));
            h[j] = v.x;
            h[j + 1] = v.y;
        }
    }
}

// A row in `group` threads of a warp (a power of two), ITEMS vectors a thread.
template <int N, int MODE, bool RES, int ITEMS>
__global__ void __launch_bounds__(kWide) k_norm_warp(const __grid_constant__ NormArgs a, int group, int64_t rows) {
    grid_dep_launch();
    grid_dep_wait();
    __shared__ __align__(16) uint8_t stage[N == 8 ? kWide / 32 : 1][272];
    const int lane = threadIdx.x % 32, in = lane % group;
    const int64_t warp = blockIdx.x * static_cast<int64_t>(kWide / 32) + threadIdx.x / 32;
    const int per = 32 / group;
    const int64_t row = warp * per + lane / group;
    const bool live = row < rows;
    const Row at = row_of(a, live ? row : rows - 1);
    Raw<N> x[ITEMS], r[RES ? ITEMS : 1];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int e = (k * group + in) * N - (MODE == kShift ? at.shift : 0);
        if (e < a.D) {
            x[k].template load<MODE>(a.X, at.x + e, a.x_dt, e, a.D);
            if constexpr (RES) r[k].template load<MODE>(a.R, at.r + e, a.r_dt, e, a.D);
        }
    }
    float h[ITEMS][N];
    float2 sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int e = (k * group + in) * N - (MODE == kShift ? at.shift : 0);
        if (e < a.D) {
            x[k].get(h[k], a.x_dt);
            if constexpr (RES) {
                float f[N];
                r[k].get(f, a.r_dt);
                add_to(h[k], f);
                if (a.RO && live) put<N, MODE>(a.RO, at.ro + e, a.r_dt, h[k], e, a.D);
            }
            sq = squares(h[k], sq);
        }
    }
    const float inv = rsqrtf(warp_sum(sq.x + sq.y, group) / static_cast<float>(a.D) + a.eps);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int e = (k * group + in) * N - (MODE == kShift ? at.shift : 0);
        const bool mine = e < a.D;
        float w[N];
        if (mine) {
            weights<N, MODE>(a, e, w);
            scale(h[k], inv, w);
        }
        if constexpr (N == 8 && MODE != kShift) {
            if (a.y_fmt == QMM_NORM_Q8_0) {          // one row a warp
                const int left = (static_cast<int>(a.D) - k * 256) / 8;
                if (left <= 0) continue;
                uint8_t* to = static_cast<uint8_t*>(a.Y) + at.y + k * 272;
                if (!mine)
                    for (int j = 0; j < N; ++j) h[k][j] = 0.f;
                put_q8(to, stage[threadIdx.x / 32], lane, live ? min(32, left) : 0, h[k]);
                continue;
            }
        }
        if (mine && live) put<N, MODE>(a.Y, at.y + e, a.y_fmt, h[k], e, a.D);
    }
}

// A row a block.
template <int N, int MODE, bool RES, int ITEMS, int MOST>
__global__ void __launch_bounds__(MOST) k_norm_block(const __grid_constant__ NormArgs a) {
    grid_dep_launch();
    grid_dep_wait();
    __shared__ __align__(16) uint8_t stage[N == 8 ? 32 : 1][272];
    __shared__ float part[32];
    const int lane = threadIdx.x % 32, wid = threadIdx.x / 32, threads = static_cast<int>(blockDim.x);
    const Row at = row_of(a, blockIdx.x);
    Raw<N> x[ITEMS], r[RES ? ITEMS : 1];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int e = (k * threads + static_cast<int>(threadIdx.x)) * N - (MODE == kShift ? at.shift : 0);
        if (e < a.D) {
            x[k].template load<MODE>(a.X, at.x + e, a.x_dt, e, a.D);
            if constexpr (RES) r[k].template load<MODE>(a.R, at.r + e, a.r_dt, e, a.D);
        }
    }
    float h[ITEMS][N];
    float2 sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int e = (k * threads + static_cast<int>(threadIdx.x)) * N - (MODE == kShift ? at.shift : 0);
        if (e < a.D) {
            x[k].get(h[k], a.x_dt);
            if constexpr (RES) {
                float f[N];
                r[k].get(f, a.r_dt);
                add_to(h[k], f);
                if (a.RO) put<N, MODE>(a.RO, at.ro + e, a.r_dt, h[k], e, a.D);
            }
            sq = squares(h[k], sq);
        }
    }
    float ss = warp_sum(sq.x + sq.y, 32);
    if (lane == 0) part[wid] = ss;
    __syncthreads();
    ss = warp_sum(lane < threads / 32 ? part[lane] : 0.f, 32);
    const float inv = rsqrtf(ss / static_cast<float>(a.D) + a.eps);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int e = (k * threads + static_cast<int>(threadIdx.x)) * N - (MODE == kShift ? at.shift : 0);
        const bool mine = e < a.D;
        if (mine) {
            float w[N];
            weights<N, MODE>(a, e, w);
            scale(h[k], inv, w);
        }
        if constexpr (N == 8 && MODE != kShift) {
            if (a.y_fmt == QMM_NORM_Q8_0) {
                const int first = (k * threads + wid * 32) * 8, left = (static_cast<int>(a.D) - first) / 8;
                if (left <= 0) continue;
                uint8_t* to = static_cast<uint8_t*>(a.Y) + at.y + first / 32 * 34;
                if (!mine)
                    for (int j = 0; j < N; ++j) h[k][j] = 0.f;
                put_q8(to, stage[wid], lane, min(32, left), h[k]);
                continue;
            }
        }
        if (mine) put<N, MODE>(a.Y, at.y + e, a.y_fmt, h[k], e, a.D);
    }
}

// Rows too long for a block's registers: x and r are read again for the product
// (r' may be r or x, so that it is written with y).
template <int N, int MODE, bool RES>
__global__ void __launch_bounds__(1024) k_norm_long(const __grid_constant__ NormArgs a) {
    grid_dep_launch();
    grid_dep_wait();
    __shared__ __align__(16) uint8_t stage[N == 8 ? 32 : 1][272];
    __shared__ float part[32];
    const int lane = threadIdx.x % 32, wid = threadIdx.x / 32, threads = static_cast<int>(blockDim.x);
    const Row at = row_of(a, blockIdx.x);
    auto sum_of = [&](int64_t e, float (&h)[N]) {
        Raw<N> x, r;
        x.template load<MODE>(a.X, at.x + e, a.x_dt, e, a.D);
        if constexpr (RES) r.template load<MODE>(a.R, at.r + e, a.r_dt, e, a.D);
        x.get(h, a.x_dt);
        if constexpr (RES) {
            float f[N];
            r.get(f, a.r_dt);
            add_to(h, f);
        }
    };
    float2 sq = make_float2(0.f, 0.f);
    for (int64_t e = static_cast<int64_t>(threadIdx.x) * N - (MODE == kShift ? at.shift : 0); e < a.D; e += threads * N) {
        float h[N];
        sum_of(e, h);
        sq = squares(h, sq);
    }
    float ss = warp_sum(sq.x + sq.y, 32);
    if (lane == 0) part[wid] = ss;
    __syncthreads();
    ss = warp_sum(lane < threads / 32 ? part[lane] : 0.f, 32);
    const float inv = rsqrtf(ss / static_cast<float>(a.D) + a.eps);
    // a warp's lanes stay together: they share blocks of the 8-bit output
    for (int64_t first = wid * 32 * N; first < a.D + (MODE == kShift ? 7 : 0); first += threads * N) {
        const int64_t e = first + lane * N - (MODE == kShift ? at.shift : 0);
        const bool mine = e < a.D;
        float h[N];
#pragma unroll
        for (int j = 0; j < N; ++j) h[j] = 0.f;
        if (mine) {
            sum_of(e, h);
            if (RES && a.RO) put<N, MODE>(a.RO, at.ro + e, a.r_dt, h, e, a.D);
            float w[N];
            weights<N, MODE>(a, e, w);
            scale(h, inv, w);
        }
        if constexpr (N == 8 && MODE != kShift) {
            if (a.y_fmt == QMM_NORM_Q8_0) {
                put_q8(static_cast<uint8_t*>(a.Y) + at.y + first / 32 * 34, stage[wid], lane,
                       static_cast<int>(imin64(32, (a.D - first) / 8)), h);
                continue;
            }
        }
        if (mine) put<N, MODE>(a.Y, at.y + e, a.y_fmt, h, e, a.D);
    }
}

// Threads and vectors a thread. Few rows are spread over as many threads as they have
// vectors (latency); from four rows per SM on a thread takes four, whose loads
// are in flight together, and rows of up to four vectors a lane a warp alone. (Rows of a
// vector a lane, 8192 x 48 heads of 128 in f16: 56 us, 0.53 of copy, 240 instructions for a warp's
// two rows, issue slots 70 % busy, the wait for loads the longest of the others; two or four rows
// at a time were slower.)
template <int N, int MODE, bool RES> cudaError_t run(const NormArgs& a, cudaStream_t s) {
    const int64_t rows = a.T * a.H, vecs = (a.D + (MODE == kShift ? 7 : 0) + N - 1) / N;
    if (rows > 0x7fffffff) return cudaErrorInvalidValue;
    int dev = 0;
    cudaGetDevice(&dev);
    const int64_t sms = sm_count(dev);
    const bool many = rows >= 4 * sms;
    if (vecs <= (many ? 128 : 64)) {
        const bool q8 = a.y_fmt == QMM_NORM_Q8_0;
        int group = q8 ? 32 : 1;
        while (group < 32 && group < vecs) group *= 2;
        const int64_t per_block = kWide / group, blocks = (rows + per_block - 1) / per_block;
        auto go = [&](auto k, int64_t n) { return launch_chained(k, dim3(static_cast<unsigned>(n)), kWide, 0, s, a, group, rows); };
        return vecs <= 32   ? go(k_norm_warp<N, MODE, RES, 1>, blocks)
               : vecs <= 64 ? go(k_norm_warp<N, MODE, RES, 2>, blocks)
                            : go(k_norm_warp<N, MODE, RES, 4>, blocks);
    }
    const dim3 grid(static_cast<unsigned>(rows));
    auto go = [&](auto k, int items) {
        return launch_chained(k, grid, static_cast<int>((vecs + items * 32 - 1) / (items * 32)) * 32, 0, s, a);
    };
    if (!many && vecs <= 512) return go(k_norm_block<N, MODE, RES, 1, 512>, 1);
    if (!many && vecs <= 1024) return go(k_norm_block<N, MODE, RES, 2, 512>, 2);
    if (vecs <= 1024) return go(k_norm_block<N, MODE, RES, 4, 256>, 4);
    if (vecs <= 4096) return go(k_norm_block<N, MODE, RES, 4, 1024>, 4);
    if constexpr (N == 1) {
        if (vecs <= 16384) return go(k_norm_block<N, MODE, RES, 16, 1024>, 16);
    }
    return launch_chained(k_norm_long<N, MODE, RES>, grid, 1024, 0, s, a);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& args, cudaStream_t s) {
    NormArgs a = args;
    // n / H for n < 2^31 as (n * mul) >> (32 + shift): with mul = ceil(2^(32 + shift) / H), 2^shift < H
    // <= 2^(shift + 1), the product is off by less than n / 2^32 of a quotient's step, below 1 / H
    a.h_shift = 0;
    while ((int64_t(2) << a.h_shift) < a.H) ++a.h_shift;
    a.h_mul = static_cast<unsigned>(((uint64_t(1) << (32 + a.h_shift)) + static_cast<uint64_t>(a.H) - 1) / static_cast<uint64_t>(a.H));
    auto size = [](int dt) { return static_cast<int64_t>(dt == QMM_F32 ? 4 : 2); };
    const bool q8 = a.y_fmt == QMM_NORM_Q8_0;
    auto go = [&](auto n, auto mode) {
        constexpr int N = decltype(n)::value, MODE = decltype(mode)::value;
        return a.R ? run<N, MODE, true>(a, s) : run<N, MODE, false>(a, s);
    };
    auto ok = [&](const void* p, int64_t ts, int64_t hs, int64_t sz) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.T == 1 || ts * sz % 16 == 0) && (a.H == 1 || hs * sz % 16 == 0);
    };
    const bool vec = a.D % 8 == 0 && ok(a.X, a.x_ts, a.x_hs, size(a.x_dt)) && (!a.R || ok(a.R, a.r_ts, a.r_hs, size(a.r_dt))) &&
                     (!a.RO || ok(a.RO, a.ro_ts, a.ro_hs, size(a.r_dt))) && ok(a.W, 0, 0, 4) &&
                     (q8 || ok(a.Y, a.y_ts, a.y_hs, size(a.y_fmt)));
    if (vec) return go(std::integral_constant<int, 8>{}, std::integral_constant<int, kVec>{});
    if (q8) return go(std::integral_constant<int, 8>{}, std::integral_constant<int, kOne>{});
    // vectors of eight elements on a grid of 8 * size bytes: every array's rows begin alike
    a.w_at16 = reinterpret_cast<uintptr_t>(a.W) % 16 == 0;
    a.x_shift = static_cast<int>(reinterpret_cast<uintptr_t>(a.X) / size(a.x_dt) % 8);
    auto alike = [&](const void* p, int64_t ts, int64_t hs, int64_t sz) {
        return static_cast<int>(reinterpret_cast<uintptr_t>(p) / sz % 8) == a.x_shift && (a.T == 1 || (ts - a.x_ts) % 8 == 0) &&
               (a.H == 1 || (hs - a.x_hs) % 8 == 0);
    };
    if (a.D >= 32 && (!a.R || alike(a.R, a.r_ts, a.r_hs, size(a.r_dt))) && (!a.RO || alike(a.RO, a.ro_ts, a.ro_hs, size(a.r_dt))) &&
        alike(a.Y, a.y_ts, a.y_hs, size(a.y_fmt)))
        return go(std::integral_constant<int, 8>{}, std::integral_constant<int, kShift>{});
    return go(std::integral_constant<int, 1>{}, std::integral_constant<int, kOne>{});
}

}  // namespace qmm
