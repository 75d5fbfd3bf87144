// attn_kernel.cuh -- qattn_decode: attention of one new token a sequence over a
// paged key-value cache, split over the length and joined.
//
//   s_j = scale q . k_j  (softcap c: c tanh(s_j / c)),   lo <= j < len
//   o = sum_j e^{s_j} v_j / sum_j e^{s_j},   lse = ln sum_j e^{s_j}
//
// Every cached row is read once per group of query heads that share it, so the
// operator is bound by those bytes (K and V rows of the lengths in range).
//
// Tiles. A warp takes 16 * SUB keys at a time with up to 8 * NT query heads of
// one key-value head, and keeps the running maximum m, sum l and output O of
// the softmax in registers (fp32). Both products run on mma.sync m16n8k16 with
// the KEYS (first product) or the DIMS (second) on the 16-row side and the
// query heads on the 8-column side: S^T = K Q^T and O^T = V^T P^T. A group of
// up to eight heads then fills the columns, K and V are the A operands and are
// used by one warp only, so they go straight from global memory into the
// registers that feed the MMA -- no shared memory, no barrier in the loop. At 8
// heads the tensor work is 8 FLOP per cached byte, a small part of what
// mma.sync sustains; tcgen05's 128-row tiles would be 8/128 full here.
//
// Operand layout without transposes through memory:
//   * K: the sum over dims does not depend on their order, so lane (g, t) loads
//     8 consecutive dims 32c + 8t .. + 7 of keys g and g + 8, and the q fragment
//     is built in the same order.
//   * V: lane (g, t) loads VW consecutive dims of keys 2t, 2t+1, 2t+8, 2t+9;
//     pairs of keys are zipped by byte permutes. Row g of MMA tile j is dim
//     VW g + 2j, row g + 8 the dim after it.
//   * P: the accumulator layout of S^T becomes the B operand of the second
//     product through movmatrix (an 8 x 8 transpose in registers).
// Each warp issues the loads of its next K tile as soon as the first product
// has consumed the present one, and those of V after the second, so loads are
// in flight through the whole loop.
//
// Rounding. Products of a 16-bit cache are exact in fp32. q and the softmax
// weights p enter the MMAs as sums of 16-bit terms: two f16 terms carry 22
// bits, bf16 terms 8 bits each. With 16-bit activations p takes two terms (its
// rounding then stays well under the output's own); with fp32 activations q
// and p take as many as reach fp32 (f16: 2, bf16: 3). f16 terms need a bounded
// range: fp32 / bf16 q rows are scaled by a power of two that puts their
// largest magnitude in [2^9, 2^10), p is held as 2^14 e^{s - m}. Q8_0 codes are
// integers, exact in f16 and bf16: K's block scale multiplies the fp32 partial
// sums of its 32 dims, V's block scale multiplies p before it is split.
#pragma once

#include "kv_common.cuh"

namespace qmm {
namespace attn {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

template <int FMT, bool HI> struct Terms;    // MMA terms of q and p
template <> struct Terms<QMM_KV_F16, false> { static constexpr int q = 1, p = 2; };    // f16 q
template <> struct Terms<QMM_KV_F16, true> { static constexpr int q = 2, p = 2; };     // bf16, fp32 q
template <> struct Terms<QMM_KV_BF16, false> { static constexpr int q = 1, p = 2; };   // bf16 q
template <> struct Terms<QMM_KV_BF16, true> { static constexpr int q = 3, p = 3; };    // f16, fp32 q
template <> struct Terms<QMM_KV_Q8_0, false> { static constexpr int q = 1, p = 2; };   // f16 q
template <> struct Terms<QMM_KV_Q8_0, true> { static constexpr int q = 2, p = 3; };    // bf16, fp32 q

__host__ __device__ constexpr bool needs_hi(int fmt, int dtype) {
    return fmt == QMM_KV_BF16 ? dtype != QMM_BF16 : dtype != QMM_F16;
}

template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                    unsigned b1) {
    if constexpr (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ unsigned transpose8x8(unsigned x) {
    unsigned y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// x0, x1 rounded to 16 bits (low half: x0), their residues left in x0, x1.
template <bool BF> __device__ __forceinline__ unsigned take16(float& x0, float& x1) {
    unsigned r;
    if constexpr (BF) {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x1), "f"(x0));
        x0 -= __uint_as_float(r << 16);
        x1 -= __uint_as_float(r & 0xffff0000u);
    } else {
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x1), "f"(x0));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
        x0 -= f.x;
        x1 -= f.y;
    }
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four int8 codes (in byte order) as two f16 pairs, exactly: the biased code u =
// c + 128 in the low mantissa byte of 1024 is the f16 number 1024 + u.
__device__ __forceinline__ void codes_f16(unsigned x, unsigned& p0, unsigned& p1) {
    x ^= 0x80808080u;
    const unsigned a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));   // 1152
    const __half2 r0 = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
    const __half2 r1 = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
    p0 = *reinterpret_cast<const unsigned*>(&r0);
    p1 = *reinterpret_cast<const unsigned*>(&r1);
}

// Four int8 codes as two bf16 pairs, exactly: the low seven bits in the mantissa
// of 128 give 128 + low7; the sign bit in the exponent's last place gives 128
// or 256; their difference is the code.
__device__ __forceinline__ void codes_bf16(unsigned x, unsigned& p0, unsigned& p1) {
    const unsigned lo = x & 0x7f7f7f7fu, hi = x & 0x80808080u;
    const unsigned a0 = __byte_perm(lo, 0x43434343u, 0x4140), a1 = __byte_perm(lo, 0x43434343u, 0x4342);
    const unsigned b0 = __byte_perm(hi, 0x43434343u, 0x4140), b1 = __byte_perm(hi, 0x43434343u, 0x4342);
    const __nv_bfloat162 r0 =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a0), *reinterpret_cast<const __nv_bfloat162*>(&b0));
    const __nv_bfloat162 r1 =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a1), *reinterpret_cast<const __nv_bfloat162*>(&b1));
    p0 = *reinterpret_cast<const unsigned*>(&r0);
    p1 = *reinterpret_cast<const unsigned*>(&r1);
}

template <typename V> __device__ __forceinline__ V ldg(const uint8_t* p) { return *reinterpret_cast<const V*>(p); }

__device__ __forceinline__ float load_act(const void* p, int dtype, int64_t i) {
    if (dtype == QMM_F32) return static_cast<const float*>(p)[i];
    if (dtype == QMM_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_act(void* p, int dtype, int64_t i, float v) {
    if (dtype == QMM_F32) static_cast<float*>(p)[i] = v;
    else if (dtype == QMM_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// The range of one sequence: keys [lo, len), split in chunks that start at lo
// rounded down to 16. A length outside [0, max_len] is an error.
struct Range {
    int lo, lo16, len, splits;
    bool bad;
};
__device__ __forceinline__ Range range_of(const AttnArgs& a, int64_t b, int chunk) {
    Range r;
    r.len = a.lens[b];
    r.bad = r.len < 0 || r.len > a.max_len;
    if (r.bad) r.len = 0;
    r.lo = a.window > 0 && r.len > a.window ? r.len - a.window : 0;
    r.lo16 = r.lo & ~15;
    r.splits = (r.len - r.lo16 + chunk - 1) / chunk;
    return r;
}

// Partial results in the workspace: O [B * Hq][splits][D], then (m, l) pairs
// [B * Hq][splits]; m in units of log2.
__device__ __forceinline__ float* ws_o(const AttnArgs& a, int splits, int64_t bh, int s) {
    return static_cast<float*>(a.ws) + (bh * splits + s) * a.c.D;
}
__device__ __forceinline__ float2* ws_ml(const AttnArgs& a, int splits, int64_t bh, int s) {
    return reinterpret_cast<float2*>(static_cast<float*>(a.ws) + a.B * a.Hq * splits * a.c.D) + bh * splits + s;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int FMT, int D, bool HI, int NT, int SUB>
__device__ __forceinline__ void attn_block(const AttnArgs& a, int splits, int chunk, int head_chunks) {
    constexpr bool Q8 = FMT == QMM_KV_Q8_0;
    constexpr bool KBF = FMT == QMM_KV_BF16;          // operand type of K q and of V p
    constexpr bool VBF = FMT != QMM_KV_F16;
    constexpr int NQ = Terms<FMT, HI>::q, NP = Terms<FMT, HI>::p;
    constexpr int C = D / 32;                         // 32-dim blocks of a row
    constexpr int KT = 16 * SUB;                      // keys per tile
    constexpr int VW = !Q8 && D % 64 == 0 ? 8 : 4;    // dims per lane of a V row
    constexpr int VC = D / (8 * VW);                  // V chunks of 8 * VW dims
    constexpr float kBias = VBF ? 0.f : 14.f;
    using KVec = typename VecOf<Q8 ? 8 : 16>::type;
    using VVec = typename VecOf<Q8 ? 4 : 2 * VW>::type;
    constexpr int KW = sizeof(KVec) / 4;

    __shared__ float sm_o[kWarps][8 * NT][D + 4];     // the query rows first, the warps' outputs last
    __shared__ float sm_m[kWarps][8 * NT], sm_l[kWarps][8 * NT], sm_scale[8 * NT];

    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;
    // block -> (sequence, key-value head, chunk of its query heads, split)
    const int64_t blk = blockIdx.x;
    const int split = static_cast<int>(blk % splits);
    int64_t r = blk / splits;
    const int hc = static_cast<int>(r % head_chunks);
    r /= head_chunks;
    const int kh = static_cast<int>(r % a.c.heads);
    const int64_t b = r / a.c.heads;
    const int group = a.Hq / a.c.heads;
    const int h0 = kh * group + hc * 8 * NT;          // first query head
    const int nh = min(8 * NT, group - hc * 8 * NT);

    const Range rg = range_of(a, b, chunk);
    if (rg.splits == 0) {                             // nothing to attend to (or a bad length)
        if (split == 0) {
            if (rg.bad && threadIdx.x == 0) atomicOr(a.err, DEV_ERR_BAD_SLOT);
            for (int i = threadIdx.x; i < nh * D; i += kThreads)
                store_act(a.out, a.dtype, (b * a.Hq + h0) * D + i, rg.bad ? NAN : 0.f);
            if (a.lse && threadIdx.x < nh) a.lse[b * a.Hq + h0 + threadIdx.x] = rg.bad ? NAN : -INFINITY;
        }
        return;
    }
    if (split >= rg.splits) return;

    const int begin = rg.lo16 + split * chunk, end = min(begin + chunk, rg.len);
    const int shift = a.c.page_shift, page_mask = (1 << shift) - 1;
    const int page_lo = rg.lo >> shift, page_hi = (rg.len - 1) >> shift;
    const int32_t* table = a.table + b * a.table_stride;
    const int64_t unit = a.c.unit();
    const uint8_t* kbase = a.c.k + kh * unit;
    const uint8_t* vbase = a.c.v + kh * unit;
    bool bad = false;

    // Page ids of the 8-key groups of a tile: a group lies in one page (pages
    // hold 8 or more keys, tiles start at multiples of 16). Groups outside the
    // range name a page inside it, so that every address is that of a page the
    // sequence owns; their scores and V rows are masked below.
    auto page_ids = [&](int base, int (&id)[2 * SUB]) {
#pragma unroll
        for (int i = 0; i < 2 * SUB; ++i) id[i] = table[max(page_lo, min((base + 8 * i) >> shift, page_hi))];
    };
    auto page_at = [&](int id) -> int64_t {
        if (static_cast<unsigned>(id) >= static_cast<uint64_t>(a.c.n_pages)) {
            bad = true;
            id = 0;
        }
        return id * a.c.page_stride;
    };
    constexpr int ROW = Q8 ? D : 2 * D;               // bytes of a row's codes or values
    KVec kreg[SUB][2][C];
    VVec vreg[SUB][4][VC];
    // Q8_0 scales of keys g, g + 8 of each 16-key group
    __half kscale[Q8 ? SUB : 1][2][Q8 ? C : 1], vscale[Q8 ? SUB : 1][2][Q8 ? C : 1];
    auto load_scales = [&](const uint8_t* p, __half (&d)[Q8 ? C : 1]) {
        if constexpr (Q8) {
            constexpr int B = C % 4 == 0 ? 8 : C % 2 == 0 ? 4 : 2;
            using SV = typename VecOf<B>::type;
#pragma unroll
            for (int i = 0; i < 2 * C / B; ++i) {
                const SV v = reinterpret_cast<const SV*>(p)[i];
                const __half* e = reinterpret_cast<const __half*>(&v);
#pragma unroll
                for (int j = 0; j < B / 2; ++j) d[i * (B / 2) + j] = e[j];
            }
        }
    };
    auto load_k = [&](int base, const int (&id)[2 * SUB]) {
#pragma unroll
        for (int s = 0; s < SUB; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t* p = kbase + page_at(id[2 * s + i]);
                const int row = (base + 16 * s + 8 * i + g) & page_mask;
                const uint8_t* q = p + row * ROW + t * static_cast<int>(sizeof(KVec));
#pragma unroll
                for (int c = 0; c < C; ++c) kreg[s][i][c] = ldg<KVec>(q + c * (ROW / C));
                if constexpr (Q8) load_scales(p + (D << shift) + row * (2 * C), kscale[s][i]);
            }
    };
    auto load_v = [&](int base, const int (&id)[2 * SUB]) {
#pragma unroll
        for (int s = 0; s < SUB; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t* p = vbase + page_at(id[2 * s + i]);
                const int row = (base + 16 * s + 8 * i + 2 * t) & page_mask;
                const uint8_t* q = p + row * ROW + g * static_cast<int>(sizeof(VVec));
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int c = 0; c < VC; ++c)
                        vreg[s][2 * i + k][c] = ldg<VVec>(q + k * ROW + c * (ROW / VC));
                if constexpr (Q8) {
                    const int srow = (base + 16 * s + 8 * i + g) & page_mask;
                    load_scales(p + (D << shift) + srow * (2 * C), vscale[s][i]);
                }
            }
    };

    const int stride = kWarps * KT;
    int base = begin + warp * KT;
    int id0[2 * SUB], id1[2 * SUB];
    if (base < end) {
        page_ids(base, id0);
        page_ids(base + stride, id1);
        load_k(base, id0);
        load_v(base, id0);
    }

    // ---- the query fragments: B operand, column g = head, dims in K's order
    for (int i = threadIdx.x; i < 8 * NT * D; i += kThreads) {
        const int h = i / D, d = i % D;
        sm_o[0][h][d] = h < nh ? load_act(a.q, a.dtype, b * a.q_bs + (h0 + h) * a.q_hs + d) : 0.f;
    }
    __syncthreads();
    constexpr bool NORM = HI && !KBF;                 // f16 terms of fp32 / bf16 rows
    if (NORM) {
        for (int h = warp; h < 8 * NT; h += kWarps) {
            float m = 0.f;
            for (int d = lane; d < D; d += 32) m = fmaxf(m, fabsf(sm_o[0][h][d]));
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            // m in [2^e, 2^(e+1)) -> factor 2^(9 - e); none for zeros and Inf
            const int e = (__float_as_int(m) >> 23) - 127;
            const float f = m > 0.f && isfinite(m) ? exp2f(static_cast<float>(min(9 - e, 126))) : 1.f;
            if (lane == 0) sm_scale[h] = f;
        }
        __syncthreads();
    }
    unsigned qf[NT][NQ][4 * C];
    float sc[NT][2];                                  // score scale of heads 2t, 2t + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float f = NORM ? sm_scale[8 * n + g] : 1.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x0 = sm_o[0][8 * n + g][32 * c + 8 * t + 2 * j] * f;
                float x1 = sm_o[0][8 * n + g][32 * c + 8 * t + 2 * j + 1] * f;
#pragma unroll
                for (int q = 0; q < NQ; ++q) qf[n][q][4 * c + j] = take16<KBF>(x0, x1);
            }
#pragma unroll
        for (int k = 0; k < 2; ++k) sc[n][k] = NORM ? a.scale / sm_scale[8 * n + 2 * t + k] : a.scale;
    }

    float m[NT][2], l[NT][2], o[NT][VC][VW / 2][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int j = 0; j < VW / 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][c][j][i] = 0.f;
    }

#pragma unroll 1
    for (; base < end; base += stride) {
        int id2[2 * SUB];
        const bool more = base + stride < end;
        page_ids(base + 2 * stride, id2);
        // ---- S^T = K Q^T
        float sx[NT][SUB][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int s = 0; s < SUB; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) sx[n][s][i] = 0.f;
#pragma unroll
        for (int s = 0; s < SUB; ++s)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                unsigned x0[4], x1[4];                // dims 8t .. 8t + 7 of keys g and g + 8 as 16-bit pairs
                if constexpr (Q8) {
                    const unsigned* w0 = reinterpret_cast<const unsigned*>(&kreg[s][0][c]);
                    const unsigned* w1 = reinterpret_cast<const unsigned*>(&kreg[s][1][c]);
#pragma unroll
                    for (int k = 0; k < KW; ++k) {
                        codes_f16(w0[k], x0[2 * k], x0[2 * k + 1]);
                        codes_f16(w1[k], x1[2 * k], x1[2 * k + 1]);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x0[k] = reinterpret_cast<const unsigned*>(&kreg[s][0][c])[k];
                        x1[k] = reinterpret_cast<const unsigned*>(&kreg[s][1][c])[k];
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if constexpr (Q8) {
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int q = 0; q < NQ; ++q)
                                mma<KBF>(acc, x0[2 * j], x1[2 * j], x0[2 * j + 1], x1[2 * j + 1],
                                         qf[n][q][4 * c + 2 * j], qf[n][q][4 * c + 2 * j + 1]);
                        const float d0 = __half2float(kscale[s][0][c]), d1 = __half2float(kscale[s][1][c]);
                        sx[n][s][0] = fmaf(d0, acc[0], sx[n][s][0]);
                        sx[n][s][1] = fmaf(d0, acc[1], sx[n][s][1]);
                        sx[n][s][2] = fmaf(d1, acc[2], sx[n][s][2]);
                        sx[n][s][3] = fmaf(d1, acc[3], sx[n][s][3]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int q = 0; q < NQ; ++q)
                                mma<KBF>(sx[n][s], x0[2 * j], x1[2 * j], x0[2 * j + 1], x1[2 * j + 1],
                                         qf[n][q][4 * c + 2 * j], qf[n][q][4 * c + 2 * j + 1]);
                    }
                }
            }
        if (more) load_k(base + stride, id1);

        // ---- masks, running maximum, weights
        const bool partial = base < rg.lo || base + KT > end;
        float alpha[NT][2];
        bool grew = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int s = 0; s < SUB; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x = sx[n][s][i] * sc[n][i & 1];
                    if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
                    x *= kLog2e;
                    if (partial) {
                        const int key = base + 16 * s + 8 * (i >> 1) + g;
                        if (key < rg.lo || key >= end) x = -INFINITY;
                    }
                    sx[n][s][i] = x;
                    mt[i & 1] = fmaxf(mt[i & 1], x);
                }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                mt[k] = fmaxf(mt[k], __shfl_xor_sync(0xffffffffu, mt[k], 4));
                mt[k] = fmaxf(mt[k], __shfl_xor_sync(0xffffffffu, mt[k], 8));
                mt[k] = fmaxf(mt[k], __shfl_xor_sync(0xffffffffu, mt[k], 16));
                const float mn = fmaxf(m[n][k], mt[k]);
                grew |= mn > m[n][k];
                // before the first finite score m is -inf and O, l are zero: any
                // finite reference gives weights 0
                alpha[n][k] = mn == -INFINITY ? 1.f : ex2(m[n][k] - mn);
                m[n][k] = mn;
            }
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                l[n][0] *= alpha[n][0];
                l[n][1] *= alpha[n][1];
#pragma unroll
                for (int c = 0; c < VC; ++c)
#pragma unroll
                    for (int j = 0; j < VW / 2; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[n][c][j][i] *= alpha[n][i & 1];
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float r0 = m[n][0] == -INFINITY ? 0.f : m[n][0] - kBias;
            const float r1 = m[n][1] == -INFINITY ? 0.f : m[n][1] - kBias;
#pragma unroll
            for (int s = 0; s < SUB; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sx[n][s][i] = ex2(sx[n][s][i] - (i & 1 ? r1 : r0));
                    l[n][i & 1] += sx[n][s][i];
                }
        }

        // ---- O^T += V^T P^T. Rows outside the range may hold anything (0 * NaN).
        if (partial) {
#pragma unroll
            for (int s = 0; s < SUB; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = base + 16 * s + 8 * (i >> 1) + 2 * t + (i & 1);
                    if (key < rg.lo || key >= end) {
#pragma unroll
                        for (int c = 0; c < VC; ++c) vreg[s][i][c] = VVec{};
                    }
                    if constexpr (Q8) {
                        const int skey = base + 16 * s + 8 * (i >> 1) + g;
                        if ((i & 1) == 0 && (skey < rg.lo || skey >= end)) {
#pragma unroll
                            for (int c = 0; c < C; ++c) vscale[s][i >> 1][c] = __ushort_as_half(0);
                        }
                    }
                }
        }
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
            unsigned pf[NT][NP][2];
            if constexpr (!Q8) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float x[4] = {sx[n][s][0], sx[n][s][1], sx[n][s][2], sx[n][s][3]};
#pragma unroll
                    for (int q = 0; q < NP; ++q) {
                        pf[n][q][0] = transpose8x8(take16<VBF>(x[0], x[1]));
                        pf[n][q][1] = transpose8x8(take16<VBF>(x[2], x[3]));
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < VC; ++c) {
                if constexpr (Q8) {
                    const float d0 = __half2float(vscale[s][0][c]), d1 = __half2float(vscale[s][1][c]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float x[4] = {sx[n][s][0] * d0, sx[n][s][1] * d0, sx[n][s][2] * d1, sx[n][s][3] * d1};
#pragma unroll
                        for (int q = 0; q < NP; ++q) {
                            pf[n][q][0] = transpose8x8(take16<VBF>(x[0], x[1]));
                            pf[n][q][1] = transpose8x8(take16<VBF>(x[2], x[3]));
                        }
                    }
                }
                unsigned f[VW / 2][4];                // A operand of each 16-dim tile
                if constexpr (Q8) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {     // keys 2t, 2t + 1 (and + 8): bytes zipped, then widened
                        const unsigned w0 = *reinterpret_cast<const unsigned*>(&vreg[s][2 * i][c]);
                        const unsigned w1 = *reinterpret_cast<const unsigned*>(&vreg[s][2 * i + 1][c]);
                        codes_bf16(__byte_perm(w0, w1, 0x5140), f[0][2 * i], f[0][2 * i + 1]);
                        codes_bf16(__byte_perm(w0, w1, 0x7362), f[1][2 * i], f[1][2 * i + 1]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < VW / 2; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const unsigned w0 = reinterpret_cast<const unsigned*>(&vreg[s][2 * i][c])[j];
                            const unsigned w1 = reinterpret_cast<const unsigned*>(&vreg[s][2 * i + 1][c])[j];
                            f[j][2 * i] = __byte_perm(w0, w1, 0x5410);
                            f[j][2 * i + 1] = __byte_perm(w0, w1, 0x7632);
                        }
                }
#pragma unroll
                for (int j = 0; j < VW / 2; ++j)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int q = 0; q < NP; ++q)
                            mma<VBF>(o[n][c][j], f[j][0], f[j][1], f[j][2], f[j][3], pf[n][q][0], pf[n][q][1]);
            }
        }
        if (more) load_v(base + stride, id1);
#pragma unroll
        for (int i = 0; i < 2 * SUB; ++i) id1[i] = id2[i];
    }

    // ---- the block's warps joined
    bad = __any_sync(0xffffffffu, bad);
    if (bad && lane == 0) atomicOr(a.err, DEV_ERR_BAD_SLOT);
    __syncthreads();                                  // sm_o's query rows are consumed
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], 4);
            l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], 8);
            l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], 16);
            if (g == 0) {
                sm_m[warp][8 * n + 2 * t + k] = m[n][k];
                sm_l[warp][8 * n + 2 * t + k] = bad ? NAN : l[n][k];
            }
        }
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int j = 0; j < VW / 2; ++j) {
                const int d = 8 * VW * c + VW * g + 2 * j;
                *reinterpret_cast<float2*>(&sm_o[warp][8 * n + 2 * t][d]) = make_float2(o[n][c][j][0], o[n][c][j][2]);
                *reinterpret_cast<float2*>(&sm_o[warp][8 * n + 2 * t + 1][d]) = make_float2(o[n][c][j][1], o[n][c][j][3]);
            }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * D; i += kThreads) {
        const int h = i / D, d = i % D;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][h]);
        float ll = 0.f, oo = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = sm_m[w][h] == -INFINITY ? 0.f : ex2(sm_m[w][h] - mm);
            ll += sm_l[w][h] == 0.f ? 0.f : f * sm_l[w][h];
            oo = fmaf(f, sm_o[w][h][d], oo);
        }
        const int64_t bh = b * a.Hq + h0 + h;
        if (rg.splits == 1) {
            // all scores -inf: 0 / 0, as the formula gives
            store_act(a.out, a.dtype, bh * D + d, oo / ll);
            if (a.lse && d == 0) a.lse[bh] = (mm - kBias) * kLn2 + logf(ll);
        } else {
            ws_o(a, splits, bh, split)[d] = oo;
            if (d == 0) *ws_ml(a, splits, bh, split) = make_float2(mm, ll);
        }
    }
}

template <int FMT, int D, bool HI, int NT, int SUB, int MINB>
__global__ void __launch_bounds__(kThreads, MINB)
    k_attn(const __grid_constant__ AttnArgs a, int splits, int chunk, int head_chunks) {
    grid_dep_launch();
    attn_block<FMT, D, HI, NT, SUB>(a, splits, chunk, head_chunks);
}

// One format's launcher (a translation unit each): the kernel for the head dim,
// activation type and head tiles, on `blocks` blocks.
template <int FMT> cudaError_t launch_fmt(const AttnArgs& a, const AttnPlan& p, int64_t blocks, int head_chunks, cudaStream_t s);

}  // namespace attn
}  // namespace qmm
