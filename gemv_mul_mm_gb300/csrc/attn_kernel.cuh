// attn_kernel.cuh -- qattn_decode: attention of one new token a sequence over a
// paged key-value cache, split over the length and joined.
//
//   s_j = scale q . k_j  (softcap c: c tanh(s_j / c)),   lo <= j < len
//   o = sum_j e^{s_j} v_j / sum_j e^{s_j},   lse = ln sum_j e^{s_j}
//
// Every cached row is read once per group of query heads that share it, so the
// operator is bound by those bytes (K and V rows of the lengths in range).
//
// Tiles. A warp takes 16 keys at a time with up to 8 * NT query heads of one
// key-value head, and keeps the running maximum m, sum l and output O of the
// softmax in registers (fp32). Both products run on mma.sync m16n8k16 with the
// KEYS (first product) or the DIMS (second) on the 16-row side and the query
// heads on the 8-column side: S^T = K Q^T and O^T = V^T P^T. A group of up to
// eight heads then fills the columns. At 8 heads the tensor work is 8 FLOP per
// cached byte, a small part of what mma.sync sustains; tcgen05's 128-row tiles
// would be 8/128 full here.
//
// Loads. Each warp has a ring of STAGES tiles in shared memory, filled by its
// own 16-byte asynchronous copies: no barrier between warps, and the bytes in
// flight do not depend on registers. Rows are padded by 16 bytes, so that the
// 8 x 8 matrices that ldmatrix reads touch every bank once. ldmatrix gives K's
// operand as it is and V's transposed. For Q8_0 a 16-bit matrix element is two
// codes: lane (g, t) gets codes 4t .. 4t + 3 of key g (K), or dims 2g, 2g + 1
// of keys 2t, 2t + 1 (V, transposed), and the byte permutes that widen the
// codes put them in the order that the MMA wants; q is laid out to match.
// P passes from the accumulator layout of S^T to the B operand of the second
// product by movmatrix (an 8 x 8 transpose in registers).
//
// Rounding. Products of a 16-bit cache are exact in fp32. q and the softmax
// weights p enter the MMAs as sums of 16-bit terms: two f16 terms carry 22
// bits, bf16 terms 8 bits each. With 16-bit activations p takes two terms (its
// rounding then stays well under the output's own); with fp32 activations q
// and p take as many as reach fp32 (f16: 2, bf16: 3). f16 terms need a bounded
// range: fp32 / bf16 q rows are scaled by a power of two that puts their
// largest magnitude in [2^9, 2^10), and weights are held as 2^14 e^{s - m}.
//
// Q8_0 codes enter exactly, as the f16 integers they are (u = c + 128 in the low
// byte of 1024, less 1152). K's block scale multiplies the fp32 partial sum of
// the 32 dims. The MMA cuts its sum off 24 bits below the largest term, so that
// nothing large may stand in it that the result does not hold: the biased codes
// themselves, with 128 sum q taken off at the start, are a subtraction fewer,
// but where one channel of a block stands out the other codes are small, and
// scores came out 10 to 20 times as far off as an fp32 sum with a channel of 50
// times the others, 100 to 300 times with one of 500. (Nor were they faster: 64 x
// 8192 tokens, f16 q, 203 us against 191 to 203, fp32 q 219 against 223.) The
// small terms of q are summed first, for the same reason.
// V's codes enter the second product the same way, and V's block scale d
// multiplies the two terms of p: t1 = rn(ph d), then
// t2 = rn(pl d + (ph d - t1)), where the bracket is exact in one fma. A power
// of two, from the running largest exponent of V's scales, keeps d near 1.
//
// The running maximum moves only where a score exceeds it (a vote over the
// warp), so most tiles do without the maximum over lanes and the rescaling.
#pragma once

#include <type_traits>

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
template <> struct Terms<QMM_KV_Q8_0, true> { static constexpr int q = 2, p = 2; };    // bf16, fp32 q

__host__ __device__ constexpr bool needs_hi(int fmt, int dtype) {
    return fmt == QMM_KV_BF16 ? dtype != QMM_BF16 : dtype != QMM_F16;
}

// d += a b
template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                    unsigned b1) {
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ unsigned transpose8x8(unsigned x) {
    unsigned y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
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

// Four int8 codes as two f16 pairs, (bytes 0, 2) and (bytes 1, 3), exactly: the
// biased code u = c + 128 in the low mantissa byte of 1024 is 1024 + u.
__device__ __forceinline__ void codes_f16(unsigned x, unsigned& p0, unsigned& p1) {
    const unsigned a = (x & 0x00ff00ffu) ^ 0x64806480u, b = __byte_perm(x, 0u, 0x4341) ^ 0x64806480u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));   // 1152
    const __half2 r0 = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
    const __half2 r1 = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
    p0 = *reinterpret_cast<const unsigned*>(&r0);
    p1 = *reinterpret_cast<const unsigned*>(&r1);
}

__device__ __forceinline__ __half2 as_half2(unsigned x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ unsigned as_u32(__half2 x) { return *reinterpret_cast<const unsigned*>(&x); }

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
// [B * Hq][splits]; m, the score that O and l are relative to.
__device__ __forceinline__ float* ws_o(const AttnArgs& a, int splits, int64_t bh, int s) {
    return static_cast<float*>(a.ws) + (bh * splits + s) * a.c.D;
}
__device__ __forceinline__ float2* ws_ml(const AttnArgs& a, int splits, int64_t bh, int s) {
    return reinterpret_cast<float2*>(static_cast<float*>(a.ws) + a.B * a.Hq * splits * a.c.D) + bh * splits + s;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Scores are kept in log2 units, scale and log2 e in one factor; capped ones in
// natural units (the cap times log2 e, rounded, would scale all of them alike)
// and their differences are multiplied by log2 e.
__device__ __forceinline__ float unit_of(const AttnArgs& a) { return a.softcap > 0.f ? kLog2e : 1.f; }
__device__ __forceinline__ float lse_of(const AttnArgs& a, float m, float l) {
    return (a.softcap > 0.f ? m : m * kLn2) + logf(l);
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes global -> shared.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The same with bytes 16; bytes 0 writes zeros and reads nothing.
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const uint8_t* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N of this thread's newest groups are in flight.
template <int N> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(unsigned (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(unsigned (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Shared-memory layout of a block: the warps' rings; after the loop, the
// warps' outputs in the same place.
template <int FMT, int D, int NT, int STAGES> struct Layout {
    static constexpr bool Q8 = FMT == QMM_KV_Q8_0;
    static constexpr int C = D / 32;
    static constexpr int ROW = Q8 ? D : 2 * D;              // bytes of a row's codes or values
    static constexpr int RS = ROW + 16;                     // row pitch
    static constexpr int KT = 16;                           // keys per stage
    static constexpr int V0 = KT * RS;                      // K rows, V rows, K scales, V scales
    static constexpr int S0 = 2 * KT * RS, SV = 2 * C * KT; // (bytes of K's scales)
    static constexpr int STAGE = S0 + (Q8 ? 2 * SV : 0);
    static constexpr int RING = STAGES * STAGE;             // of one warp
    static constexpr int OD = D + 4;
    static constexpr int JOIN = kWarps * 8 * NT * OD * 4;
    static constexpr int BYTES = kWarps * RING > JOIN ? kWarps * RING : JOIN;
};

template <int FMT, int D, bool HI, int NT, int STAGES>
__device__ __forceinline__ void attn_block(const AttnArgs& a, int splits, int chunk, int head_chunks) {
    using Lay = Layout<FMT, D, NT, STAGES>;
    constexpr bool Q8 = FMT == QMM_KV_Q8_0;
    constexpr bool BF = FMT == QMM_KV_BF16;           // operand type of both products: bf16, else f16
    constexpr int NQ = Terms<FMT, HI>::q, NP = Terms<FMT, HI>::p;
    constexpr int C = D / 32;                         // 32-dim blocks of a row
    constexpr int KT = Lay::KT;                       // keys per tile
    constexpr int ROW = Lay::ROW, RS = Lay::RS;
    constexpr int MT = D / 16;                        // 16-dim tiles of the output

    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float sm_q[8 * NT][D + 4];
    __shared__ float sm_m[kWarps][8 * NT], sm_l[kWarps][8 * NT], sm_scale[8 * NT];
    __shared__ uint2 sm_qf[Q8 ? NT * NQ * MT : 1][32];

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

    // the query rows, read before anything waits for the lengths
    constexpr int QN = 8 * NT * D / kThreads;
    float qv[QN];
#pragma unroll
    for (int i = 0; i < QN; ++i) {
        const int j = i * kThreads + threadIdx.x, h = j / D, d = j % D;
        qv[i] = h < nh ? load_act(a.q, a.dtype, b * a.q_bs + (h0 + h) * a.q_hs + d) : 0.f;
    }
    // and the pages of this warp's first tiles, as they are without a window
    const int32_t* table = a.table + b * a.table_stride;
    int first_page[STAGES];
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
        const int64_t key = static_cast<int64_t>(split) * chunk + (warp + i * kWarps) * Lay::KT;
        first_page[i] = table[imin64(key >> a.c.page_shift, a.table_width - 1)];
    }
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
    const uint8_t* kbase = a.c.k + kh * a.c.unit();
    const int64_t v_minus_k = a.c.v - a.c.k;
    bool bad = false;

    // Pages of a tile: one for its 16 keys, or with pages of 8 one for each half
    // (tiles start at multiples of 16). Halves outside the range name a page
    // inside it, so that every address is that of a page the sequence owns.
    const bool small_pages = shift < 4;
    auto page_id = [&](int key) { return table[max(page_lo, min(key >> shift, page_hi))]; };
    auto page_ids = [&](int base, int (&id)[2]) {
        id[0] = page_id(base);
        if (small_pages) id[1] = page_id(base + 8);
    };
    auto page_at = [&](int id) {                      // this head's K rows in a page
        if (static_cast<uint64_t>(static_cast<unsigned>(id)) >= static_cast<uint64_t>(a.c.n_pages)) {
            bad = true;
            id = 0;
        }
        return kbase + static_cast<uint64_t>(static_cast<unsigned>(id)) * static_cast<uint64_t>(a.c.page_stride);
    };
    const uint32_t ring = smem_addr(smem) + warp * Lay::RING;
    constexpr int CPR = ROW / 16;                     // 16-byte pieces of a row
    // this lane's first piece of a tile
    const uint32_t dst_lane = lane / CPR * RS + lane % CPR * 16;
    // Copies one tile to a stage. Its rows (of either half) are contiguous in
    // the cache. Rows outside the range become zeros (what the cache holds
    // there must not reach the products: 0 * NaN).
    auto load_tile = [&](int base, const int (&id)[2], uint32_t stage) {
        const uint8_t* page[2];
        page[0] = page_at(id[0]);
        page[1] = small_pages ? page_at(id[1]) : page[0];
        const int row0 = base & page_mask, row1 = (base + 8) & page_mask;
        if constexpr (Q8) {
            if (lane < 4 * C) {                       // scales: C pieces per half, of K then of V
                const int col = lane % C;
                const uint8_t* p = (lane / C & 1 ? page[1] + row1 * (2 * C) : page[0] + row0 * (2 * C)) + (D << shift) + col * 16;
                const uint32_t dst = stage + Lay::S0 + lane % (2 * C) * 16;
                copy16(lane < 2 * C ? dst : dst + Lay::SV, lane < 2 * C ? p : p + v_minus_k);
            }
        }
        const uint8_t* pk[2] = {page[0] + row0 * ROW + lane * 16, page[1] + (row1 - 8) * ROW + lane * 16};
        const bool partial = base < rg.lo || base + KT > end;
        auto copies = [&](auto some, auto two) {      // some rows are zeros; two pages
#pragma unroll
            for (int i = 0; i < ROW / 32; ++i) {
                const int q = 32 * i + lane, row = q / CPR;
                const int half = !decltype(two)::value ? 0 : (ROW / 2) % 32 == 0 ? 32 * i / (ROW / 2) : row / 8;
                const uint32_t dst = 32 % CPR == 0 ? stage + dst_lane + i * (32 / CPR) * RS
                                     : CPR == 32   ? stage + dst_lane + i * RS
                                                   : stage + row * RS + q % CPR * 16;
                const uint8_t* src = pk[half] + i * 512;
                if constexpr (decltype(some)::value) {
                    const int n = base + row >= rg.lo && base + row < end ? 16 : 0;
                    copy16_or_zero(dst, src, n);
                    copy16_or_zero(dst + Lay::V0, src + v_minus_k, n);
                } else {
                    copy16(dst, src);
                    copy16(dst + Lay::V0, src + v_minus_k);
                }
            }
        };
        if (partial) copies(std::true_type{}, std::true_type{});
        else if (small_pages) copies(std::false_type{}, std::true_type{});
        else copies(std::false_type{}, std::false_type{});
    };
    constexpr int stride = kWarps * KT;
    int base = begin + warp * KT;
    int id[2];                                        // pages of the next tile to load
    int ahead = base;                                 // its first key
    const bool known = rg.lo16 == 0 && !small_pages;
    if (known) id[0] = first_page[0];
    else page_ids(ahead, id);
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
        if (ahead < end) {
            load_tile(ahead, id, ring + i * Lay::STAGE);
            ahead += stride;
            if (known) id[0] = first_page[i + 1];
            else page_ids(ahead, id);
        }
        copies_commit();
    }

    // ---- the query fragments: B operand, column g = head
#pragma unroll
    for (int i = 0; i < QN; ++i) {
        const int j = i * kThreads + threadIdx.x;
        sm_q[j / D][j % D] = qv[i];
    }
    __syncthreads();
    constexpr bool NORM = HI && !BF;                  // f16 terms of fp32 / bf16 rows
    if (NORM) {
        for (int h = warp; h < 8 * NT; h += kWarps) {
            float m = 0.f;
            for (int d = lane; d < D; d += 32) m = fmaxf(m, fabsf(sm_q[h][d]));
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            // m in [2^e, 2^(e+1)) -> factor 2^(9 - e); none for zeros and Inf
            const int e = (__float_as_int(m) >> 23) - 127;
            const float f = m > 0.f && isfinite(m) ? exp2f(static_cast<float>(min(9 - e, 126))) : 1.f;
            if (lane == 0) sm_scale[h] = f;
        }
        __syncthreads();
    }
    // The fragments stay in registers, or with Q8_0, whose registers decide how
    // many blocks fit an SM, in shared memory, where the block's warps share them.
    uint2 qf[Q8 ? 1 : NT][Q8 ? 1 : NQ][Q8 ? 1 : MT];
    float sc[NT][2];                                  // score scale of heads 2t, 2t + 1, to log2 units unless capped
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float f = NORM ? sm_scale[8 * n + g] : 1.f;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            if (Q8 && j % kWarps != warp) continue;
            unsigned w[NQ][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                // dims 2t, 2t + 1 (+ 8) of the 16, or with Q8_0 4t, 4t + 2 (+ 1)
                const int d = 16 * j + (Q8 ? 4 * t + k : 2 * t + 8 * k);
                float x0 = sm_q[8 * n + g][d] * f, x1 = sm_q[8 * n + g][d + (Q8 ? 2 : 1)] * f;
#pragma unroll
                for (int q = 0; q < NQ; ++q) w[q][k] = take16<BF>(x0, x1);
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                if constexpr (Q8) sm_qf[(n * NQ + q) * MT + j][lane] = make_uint2(w[q][0], w[q][1]);
                else qf[n][q][j] = make_uint2(w[q][0], w[q][1]);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            sc[n][k] = a.scale * (a.softcap > 0.f ? 1.f : kLog2e);
            if (NORM) sc[n][k] /= sm_scale[8 * n + 2 * t + k];
        }
    }
    if constexpr (Q8) __syncthreads();
    auto q_frag = [&](int n, int q, int j) {
        if constexpr (Q8) return sm_qf[(n * NQ + q) * MT + j][lane];
        else return qf[n][q][j];
    };

    // Weights are 2^(score - ref) <= 2^kTop: f16 terms use the top of their
    // range. Before the first score, ref is kNone, the lowest float (with an
    // infinity a masked score would be NaN): a score of just that value leaves
    // ref alone and is told from none by l.
    constexpr float kTop = BF ? 0.f : 14.f, kNone = -3.402823466e38f;
    const float unit = unit_of(a), top = a.softcap > 0.f ? kTop * kLn2 : kTop;
    float ref[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        ref[n][0] = ref[n][1] = kNone;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][j][i] = 0.f;
    }
    // Q8_0: V's scales, of either sign, are below v_lim = 2^E in magnitude and are
    // multiplied by v_mul = 2^k, k = -E within f16's range; O carries that factor
    __half2 v_lim = __float2half2_rn(0.f), v_mul = __float2half2_rn(1.f);

    // matrix mi of an ldmatrix: lanes 8 mi .. 8 mi + 7 give its rows
    const int mi = lane / 8, mr = lane % 8;
    const uint32_t k_lane = (mr + 8 * (mi & 1)) * RS + 16 * (mi >> 1);
    const uint32_t v_lane = Lay::V0 + (Q8 ? k_lane : (mr + 8 * (mi >> 1)) * RS + 16 * (mi & 1));
    uint32_t stage = ring, fill = ring + (STAGES - 1) * Lay::STAGE;
    const uint32_t ring_end = ring + Lay::RING, smem_base = smem_addr(smem);

    // One tile. SLOW: some keys are masked, or scores are capped.
    auto tile = [&](auto slow_tag) {
        constexpr bool SLOW = decltype(slow_tag)::value;
        [[maybe_unused]] const uint8_t* scales = smem + (stage - smem_base) + Lay::S0;
        // ---- S^T = K Q^T
        float sx[NT][4];
        if constexpr (Q8) {
            constexpr int B = C % 4 == 0 ? 8 : C % 2 == 0 ? 4 : 2;
            using SV = typename VecOf<B>::type;
            __half kscale[2][C];                  // of keys g, g + 8
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2 * C / B; ++k) {
                    const SV x = reinterpret_cast<const SV*>(scales + (g + 8 * i) * (2 * C))[k];
#pragma unroll
                    for (int j = 0; j < B / 2; ++j) kscale[i][k * (B / 2) + j] = reinterpret_cast<const __half*>(&x)[j];
                }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                unsigned w[4];                    // (key g, g + 8) of dims 0 .. 15, then of 16 .. 31
                ldsm4(w, stage + k_lane + 32 * c);
                unsigned x[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    codes_f16(w[2 * j], x[j][0], x[j][2]);
                    codes_f16(w[2 * j + 1], x[j][1], x[j][3]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = NQ - 1; q >= 0; --q)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint2 f = q_frag(n, q, 2 * c + j);
                            mma<BF>(acc, x[j][0], x[j][1], x[j][2], x[j][3], f.x, f.y);
                        }
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const float d = __half2float(kscale[i >> 1][c]);
                        const float2 x = fma2(make_float2(d, d), make_float2(acc[i], acc[i + 1]),
                                              c == 0 ? make_float2(0.f, 0.f) : make_float2(sx[n][i], sx[n][i + 1]));
                        sx[n][i] = x.x;
                        sx[n][i + 1] = x.y;
                    }
                }
            }
        } else {
            float acc[NT][NQ][4];                     // a sum for each term: the small ones keep their bits
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int q = 0; q < NQ; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][q][i] = 0.f;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                unsigned x[4];
                ldsm4(x, stage + k_lane + 32 * j);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int q = 0; q < NQ; ++q) mma<BF>(acc[n][q], x[0], x[1], x[2], x[3], q_frag(n, q, j).x, q_frag(n, q, j).y);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sx[n][i] = acc[n][NQ - 1][i];
#pragma unroll
                    for (int q = NQ - 2; q >= 0; --q) sx[n][i] += acc[n][q][i];
                }
        }

        // ---- scores, less ref, in log2 units
        if constexpr (SLOW) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x = sx[n][i] * sc[n][i & 1];
                    if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
                    const int key = base + 8 * (i >> 1) + g;
                    if (key < rg.lo || key >= end) x = -INFINITY;
                    sx[n][i] = x;
                }
        }
        auto rel = [&](int n, int i) {
            // not fused: ref is a rounded score, and against the exact product the
            // rounding itself would be the difference once scores pass 2^24
            return SLOW ? (sx[n][i] - ref[n][i & 1]) * unit : __fmul_rn(sx[n][i], sc[n][i & 1]) - ref[n][i & 1];
        };
        float y[NT][4];
        bool grew = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[n][i] = rel(n, i);
                grew |= y[n][i] > kTop;
            }
        [[maybe_unused]] unsigned vd[2][Q8 ? C : 1];   // V scales of keys (2t, 2t + 1) and (2t + 8, 2t + 9)
        __half2 v_top = v_lim;
        if constexpr (Q8) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t* p = scales + Lay::SV + (2 * t + 8 * i) * (2 * C);
                if constexpr (C % 2 == 0) {
                    constexpr int B = C % 4 == 0 ? 8 : 4;
                    using SV = typename VecOf<B>::type;
#pragma unroll
                    for (int k = 0; k < 2 * C / B; ++k) {
                        const SV x = reinterpret_cast<const SV*>(p)[k], z = reinterpret_cast<const SV*>(p + 2 * C)[k];
#pragma unroll
                        for (int j = 0; j < B / 4; ++j) {
                            const unsigned u = reinterpret_cast<const unsigned*>(&x)[j];
                            const unsigned v = reinterpret_cast<const unsigned*>(&z)[j];
                            vd[i][k * (B / 2) + 2 * j] = __byte_perm(u, v, 0x5410);
                            vd[i][k * (B / 2) + 2 * j + 1] = __byte_perm(u, v, 0x7632);
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        vd[i][c] = reinterpret_cast<const unsigned short*>(p)[c] |
                                      static_cast<unsigned>(reinterpret_cast<const unsigned short*>(p + 2 * C)[c]) << 16;
                }
                if constexpr (SLOW) {             // rows outside the range are zeros, their scales are not
                    const int key = base + 8 * i + 2 * t;
                    const unsigned keep = (key >= rg.lo && key < end ? 0xffffu : 0u) |
                                          (key + 1 >= rg.lo && key + 1 < end ? 0xffff0000u : 0u);
#pragma unroll
                    for (int c = 0; c < C; ++c) vd[i][c] &= keep;
                }
#pragma unroll
                for (int c = 0; c < C; ++c) v_top = __hmax2(v_top, __habs2(as_half2(vd[i][c])));
            }
            grew |= !__hbleu2(v_top, v_lim);
        }
        if (__any_sync(0xffffffffu, grew)) {
            float up = 1.f;                           // change of O's factor
            if constexpr (Q8) {
                const unsigned w = as_u32(v_top);
                const unsigned big = __reduce_max_sync(0xffffffffu, max(w & 0xffffu, w >> 16));
                if (big > (as_u32(v_lim) & 0xffffu)) {
                    // scales are below 2^(field - 14) by their exponent field;
                    // one step more, so that few tiles raise it again
                    const int e = min(static_cast<int>(big >> 10) - 13, 16);
                    const __half2 mul = __float2half2_rn(exp2f(static_cast<float>(max(-15, min(15, -e)))));
                    up = __low2float(mul) / __low2float(v_mul);
                    v_mul = mul;
                    v_lim = __float2half2_rn(exp2f(static_cast<float>(e)));
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float alpha[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float mt = SLOW ? fmaxf(sx[n][k], sx[n][k + 2]) : fmaxf(__fmul_rn(sx[n][k], sc[n][k]), __fmul_rn(sx[n][k + 2], sc[n][k]));
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                    // From 2^24 on floats lie 2 and more apart and mt - top may
                    // round down, the largest weight past f16's range. There the
                    // maximum itself is the reference: weights lie that far apart
                    // too, and the largest is 1.
                    float now = mt - top;
                    if ((mt - now) * unit > kTop + 1.f) now = mt;
                    now = fmaxf(ref[n][k], now);
                    alpha[k] = ex2((ref[n][k] - now) * unit);
                    ref[n][k] = now;
                    l[n][k] *= alpha[k];
                    alpha[k] *= up;
                }
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][j][i] *= alpha[i & 1];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[n][i] = rel(n, i);
            }
        }
        // ---- weights, as the B operand of the second product: O^T += V^T P^T.
        // A weight below 2^-32 of the largest has lost most of its bits to f16's
        // subnormals. With activations whose type shows that (WIDE), a tile that
        // has such weights takes them in bands of 2^24, each scaled into range.
        constexpr bool WIDE = HI && !BF;
        constexpr float kLow = -18.f, kBand = 24.f;
        // band k of weights: [kLow - 24 k, kLow - 24 (k - 1)), the first without an
        // upper end
        auto in_band = [&](float x, int k) {
            const float lo = kLow - kBand * static_cast<float>(k);
            return x >= lo && (k == 0 || x < lo + kBand);
        };
        unsigned bands = 1;                           // those that have a weight in this tile
        if constexpr (WIDE) {
            bool low = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) low |= y[n][i] < kLow && y[n][i] >= kLow - 3 * kBand;
            if (__any_sync(0xffffffffu, low)) {
#pragma unroll 1
                for (int k = 1; k < 4; ++k) {
                    bool in = false;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) in |= in_band(y[n][i], k);
                    bands |= (__any_sync(0xffffffffu, in) ? 1u : 0u) << k;
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (WIDE) l[n][i & 1] += ex2(y[n][i]);
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            if (WIDE && !(bands >> k & 1)) {
                if (bands >> k == 0) break;
                continue;
            }
            // the MMA's sum cuts off what does not fit in 24 bits: over thousands of
            // tiles that is a bias of 1e-5 and more. With HI each tile's product
            // is summed apart and added to O with rounding.
            [[maybe_unused]] const float down = WIDE ? ex2(-kBand * static_cast<float>(k)) : 1.f;
            auto add = [&](int n, int j, const unsigned (&f)[4], const unsigned (&p)[NP][2]) {
                if constexpr (HI) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = NP - 1; q >= 0; --q) mma<BF>(d, f[0], f[1], f[2], f[3], p[q][0], p[q][1]);
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const float2 x = fma2(make_float2(d[i], d[i + 1]), make_float2(down, down),
                                              make_float2(o[n][j][i], o[n][j][i + 1]));
                        o[n][j][i] = x.x;
                        o[n][j][i + 1] = x.y;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < NP; ++q) mma<BF>(o[n][j], f[0], f[1], f[2], f[3], p[q][0], p[q][1]);
                }
            };
            unsigned pf[NT][NP][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = ex2(WIDE ? y[n][i] + kBand * static_cast<float>(k) : y[n][i]);
                    if (!WIDE) l[n][i & 1] += x[i];
                    if (WIDE && bands > 1 && !in_band(y[n][i], k)) x[i] = isnan(x[i]) ? x[i] : 0.f;
                }
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    pf[n][q][0] = transpose8x8(take16<BF>(x[0], x[1]));
                    pf[n][q][1] = transpose8x8(take16<BF>(x[2], x[3]));
                }
            }
            if constexpr (Q8) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    unsigned pd[NT][2][2];            // p times the block's scale
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const __half2 d = __hmul2(as_half2(vd[i][c]), v_mul);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const __half2 hi = as_half2(pf[n][0][i]), t1 = __hmul2_rn(hi, d);
                            pd[n][0][i] = as_u32(t1);
                            pd[n][1][i] = as_u32(__hfma2(as_half2(pf[n][1][i]), d, __hfma2(hi, d, __hneg2(t1))));
                        }
                    }
                    unsigned w[4];
                    ldsm4_trans(w, stage + v_lane + 32 * c);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        unsigned f[4];
                        codes_f16(w[2 * j], f[0], f[1]);
                        codes_f16(w[2 * j + 1], f[2], f[3]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) add(n, 2 * c + j, f, pd[n]);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    unsigned f[4];
                    ldsm4_trans(f, stage + v_lane + 32 * j);
#pragma unroll
                    for (int n = 0; n < NT; ++n) add(n, j, f, pf[n]);
                }
            }
            if constexpr (!WIDE) break;
        }
    };

#pragma unroll 1
    for (; base < end; base += stride) {
        __syncwarp();                                 // every lane is done with the stage filled next
        if (ahead < end) {
            load_tile(ahead, id, fill);
            ahead += stride;
            page_ids(ahead, id);
        }
        copies_commit();
        copies_wait<STAGES - 1>();
        __syncwarp();                                 // the tile's copies by all lanes are visible
        if (base < rg.lo || base + KT > end || a.softcap > 0.f) tile(std::true_type{});
        else tile(std::false_type{});
        fill = stage;
        stage += Lay::STAGE;
        if (stage == ring_end) stage = ring;
    }

    // ---- the block's warps joined
    copies_wait<0>();
    bad = __any_sync(0xffffffffu, bad);
    if (bad && lane == 0) atomicOr(a.err, DEV_ERR_BAD_SLOT);
    __syncthreads();                                  // every warp's ring is consumed
    float* sm_o = reinterpret_cast<float*>(smem);     // [warp][head][OD]
    constexpr int OD = Lay::OD;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], 4);
            l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], 8);
            l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], 16);
            if (g == 0) {
                sm_m[warp][8 * n + 2 * t + k] = l[n][k] == 0.f ? -INFINITY : ref[n][k];
                sm_l[warp][8 * n + 2 * t + k] = bad ? NAN : l[n][k];
            }
        }
        float* p = sm_o + (warp * 8 * NT + 8 * n + 2 * t) * OD;
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // row g of a tile is dim g, row g + 8 dim g + 8 (Q8_0: 2g and 2g + 1)
                const int d = 16 * j + (Q8 ? 2 * g + (i >> 1) : g + 8 * (i >> 1));
                p[(i & 1) * OD + d] = o[n][j][i] * (Q8 ? 1.f / __low2float(v_mul) : 1.f);
            }
    }
    __syncthreads();
    // m and l of the block, and each warp's factor in sm_m
    if (threadIdx.x < 8 * NT) {
        const int h = threadIdx.x;
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][h]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = sm_m[w][h] == -INFINITY ? 0.f : ex2((sm_m[w][h] - mm) * unit);
            ll += sm_l[w][h] == 0.f ? 0.f : f * sm_l[w][h];
            sm_m[w][h] = f;
        }
        sm_l[0][h] = ll;
        if (h < nh) {
            const int64_t bh = b * a.Hq + h0 + h;
            if (rg.splits > 1) *ws_ml(a, splits, bh, split) = make_float2(mm, ll);
            else if (a.lse) a.lse[bh] = lse_of(a, mm, ll);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * (D / 4); i += kThreads) {
        const int h = i / (D / 4), d = i % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = sm_m[w][h];
            const float4 v = *reinterpret_cast<const float4*>(&sm_o[(w * 8 * NT + h) * OD + d]);
            x.x = fmaf(f, v.x, x.x);
            x.y = fmaf(f, v.y, x.y);
            x.z = fmaf(f, v.z, x.z);
            x.w = fmaf(f, v.w, x.w);
        }
        const int64_t bh = b * a.Hq + h0 + h;
        if (rg.splits > 1) {
            *reinterpret_cast<float4*>(ws_o(a, splits, bh, split) + d) = x;
        } else {
            const float ll = sm_l[0][h];              // all scores -inf: 0 / 0, as the formula gives
            store_act(a.out, a.dtype, bh * D + d, x.x / ll);
            store_act(a.out, a.dtype, bh * D + d + 1, x.y / ll);
            store_act(a.out, a.dtype, bh * D + d + 2, x.z / ll);
            store_act(a.out, a.dtype, bh * D + d + 3, x.w / ll);
        }
    }
}

template <int FMT, int D, bool HI, int NT, int STAGES, int MINB>
__global__ void __launch_bounds__(kThreads, MINB)
    k_attn(const __grid_constant__ AttnArgs a, int splits, int chunk, int head_chunks) {
    grid_dep_launch();
    grid_dep_wait();
    attn_block<FMT, D, HI, NT, STAGES>(a, splits, chunk, head_chunks);
}

// One format's launcher (a translation unit each): the kernel for the head dim,
// activation type and head tiles. With blocks 0 nothing is launched and
// *resident gets the number of its blocks that fit an SM together.
struct Launch {
    AttnArgs a;
    AttnPlan p;
    int64_t blocks;
    cudaStream_t stream;
    int* resident;
};
template <int FMT> cudaError_t launch_fmt(const Launch& l, int D, bool hi, int tiles);

}  // namespace attn
}  // namespace qmm
