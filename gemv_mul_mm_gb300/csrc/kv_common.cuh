// kv_common.cuh -- what the rotary, cache and attention kernels share: element
// types, vector access, the rotary phase and the layout of a paged cache.
#pragma once

#include "qmm.h"
#include "qmm_internal.cuh"

namespace qmm {

// Row layouts of a paged key or value cache (bytes). Page p starts at
// p * page_stride; in it each head has one contiguous unit:
//   f16 / bf16   [page_size][D] values
//   q8_0         [page_size][D] int8 codes, then [page_size][D / 32] f16 scales
// (value = scale * code). Codes and scales apart keep every vector access
// aligned; the bytes per row are those of 34-byte Q8_0 blocks.
__host__ __device__ __forceinline__ size_t kv_row_bytes(int fmt, int64_t D) {
    return static_cast<size_t>(fmt == QMM_KV_Q8_0 ? D + D / 16 : 2 * D);
}

struct KvCache {
    uint8_t* k;
    uint8_t* v;
    int fmt;
    int page_shift;          // log2(page_size)
    int heads, D;
    int64_t n_pages;
    int64_t page_stride;     // bytes
    __host__ __device__ int64_t unit() const {
        return static_cast<int64_t>(kv_row_bytes(fmt, D)) << page_shift;
    }
};

// N consecutive elements of type T (2 or 4 bytes each) as one access of
// sizeof(T) * N bytes, up to 16 bytes; larger N takes several.
template <int BYTES> struct VecOf;
template <> struct VecOf<2> { using type = unsigned short; };
template <> struct VecOf<4> { using type = unsigned; };
template <> struct VecOf<8> { using type = uint2; };
template <> struct VecOf<16> { using type = uint4; };

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
// Rounded to nearest even, once.
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// N elements of type T as they lie in memory, moved in accesses of up to 16
// bytes (the address is aligned to min(16, N * sizeof(T)) bytes). Kernels load
// the vectors of several heads before they use the first: the stores between
// could alias, so the compiler does not.
template <typename T, int N> struct Vec {
    static constexpr int B = N * static_cast<int>(sizeof(T)) < 16 ? N * static_cast<int>(sizeof(T)) : 16;
    static constexpr int PER = B / static_cast<int>(sizeof(T));
    using V = typename VecOf<B>::type;
    V v[N / PER];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < N / PER; ++i) v[i] = reinterpret_cast<const V*>(p)[i];
    }
    __device__ __forceinline__ void load_unaligned(const T* p) {
        T* e = reinterpret_cast<T*>(v);
#pragma unroll
        for (int j = 0; j < N; ++j) e[j] = p[j];
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < N / PER; ++i) reinterpret_cast<V*>(p)[i] = v[i];
    }
    __device__ __forceinline__ void get(float (&x)[N]) const {
        const T* e = reinterpret_cast<const T*>(v);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = to_f32<T>(e[j]);
    }
    __device__ __forceinline__ void set(const float (&x)[N]) {
        T* e = reinterpret_cast<T*>(v);
#pragma unroll
        for (int j = 0; j < N; ++j) e[j] = from_f32<T>(x[j]);
    }
};

// q = a / b, r = a % b for 0 <= a, 0 < b; 32-bit where a allows it.
__device__ __forceinline__ void div_mod(int64_t a, int b, int64_t& q, int& r) {
    if (a >> 32) {
        q = a / b;
        r = static_cast<int>(a - q * b);
    } else {
        const unsigned u = static_cast<unsigned>(a), d = u / static_cast<unsigned>(b);
        q = d;
        r = static_cast<int>(u - d * static_cast<unsigned>(b));
    }
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\t"
        "mov.b64 {%0, %1}, d;}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// cos and sin of 2 pi frac(pos * turns / 2^64). The product wraps modulo 2^64,
// which drops whole turns exactly, so the angle is as good at position 10^6 as
// at 1 (an fp32 product pos * frequency is off by up to 4e-3 rad at 10^5). The
// top 32 bits of the fraction, as a signed half-turn count in [-1, 1), reach
// sincospif with one rounding (2^-25).
__device__ __forceinline__ void rope_cs(int32_t pos, uint64_t turns, float mscale, float& c, float& s) {
    const uint64_t ph = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns;
    const float half_turns = static_cast<float>(static_cast<int32_t>(ph >> 32)) * 4.656612873077393e-10f;  // 2^-31
    sincospif(half_turns, &s, &c);
    c *= mscale;
    s *= mscale;
}

// Programmatic dependent launch: the operators here are launched so that the
// next kernel on the stream may become resident while the one before it still
// runs (it saves about a microsecond per launch in a chain of short kernels).
// Each of their kernels lets its successor start at once and touches memory only
// after the wait, which returns when its predecessor has completed.
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<A&&>(args)...);
    if (e != cudaSuccess) {
        cudaGetLastError();   // reported to the caller, not left for the next one
        return e;
    }
    count_launch(1);
    return cudaSuccess;
}

// k_rope.cu
struct RopeArgs {
    const void* X;
    void* Y;
    int dtype;                     // QMM_F32 / QMM_F16 / QMM_BF16
    int64_t x_ts, x_hs, y_ts, y_hs;  // strides in elements
    const int32_t* pos;
    const uint64_t* turns;
    int rot, layout;
    float mscale;
    int64_t T, H, D;
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);

// k_kv.cu
struct KvStoreArgs {
    KvCache c;
    const void* K;
    const void* V;
    int dtype;
    int64_t k_ts, k_hs, v_ts, v_hs;
    const int64_t* slots;
    const int32_t* pos;            // nullptr: K is stored as given
    const uint64_t* turns;
    int rot, layout;
    float mscale;
    int64_t T;
    unsigned* err;
};
cudaError_t launch_kv_store(const KvStoreArgs& a, cudaStream_t s);

struct KvLoadArgs {
    KvCache c;
    const int64_t* slots;
    void* K;
    void* V;
    int dtype;
    int64_t T;
    unsigned* err;
};
cudaError_t launch_kv_load(const KvLoadArgs& a, cudaStream_t s);

// k_attn.cu
struct AttnArgs {
    KvCache c;
    const void* q;
    int dtype;                     // of q and out
    int64_t q_bs, q_hs;            // strides in elements
    const int32_t* table;          // [B][table_stride] page ids
    int64_t table_stride;
    int table_width;               // pages a row may name
    const int32_t* lens;
    int max_len;
    int64_t B;
    int Hq;
    float scale, softcap;
    int window;
    void* out;                     // [B][Hq][D]
    float* lse;                    // [B][Hq] or nullptr
    void* ws;
    unsigned* err;
};
struct AttnPlan {
    int splits;                    // most splits of one sequence
    int chunk;                     // keys per split
    int tiles;                     // 8-head tiles of a head group
    int head_chunks;               // head groups per key-value head
    bool hi;                       // the kernel with more terms
    size_t ws_bytes;               // what a split call asks for: no less than smaller sizes need
};
bool attn_dim_ok(int D);
cudaError_t attn_plan(int fmt, int dtype, int64_t B, int Hq, int Hkv, int D, int max_len, int window, int sms, AttnPlan* p);
cudaError_t launch_attn(const AttnArgs& a, const AttnPlan& p, cudaStream_t s);

}  // namespace qmm
