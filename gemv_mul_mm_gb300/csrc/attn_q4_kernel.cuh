// attn_q4_kernel.cuh -- qattn_decode over a q4_0 cache. The formulas, the split
// and the join, the ring of a warp's tiles, the softmax and the two products on
// mma.sync are those of attn_kernel.cuh; what differs is here.
//
// A cached value takes 18 / 32 bytes: half of q8_0's traffic for as many values, so
// that a warp's instructions per value, and the latency of their chain, decide. Tiles of 32 keys (two halves of 16 in the MMAs) share
// one step of the loop and of the running maximum, and give two chains of
// dependent instructions to interleave. Pages of 32 keys and more hold whole tiles, which
// are copied without a look at pages inside; smaller ones take a kernel of their own.
//
// Measured, 64 sequences of 8192 tokens, 8 key-value heads of 128, 4 query heads each: 134 us
// with f16 activations (0.66 of the copy bandwidth, 4.5 TB/s; some 680 instructions a tile
// of 32 keys, 63 % of the issue slots), 156 us with fp32; one sequence of 131072: 39 and 44 us.
// A window of 4096 of the 8192 takes 84 and 95 us, of 1024 27 and 31; a softcap (every tile then
// takes the slow path) 190 and 216. 16 query heads (4 key-value heads) do 126 and 97 TFLOP/s.
//
// Codes. ldmatrix reads a row's 32-dim block as eight 16-bit elements, four codes
// each: lane (g, t) gets codes 8t .. 8t + 7 of key g (K), or dims 4g .. 4g + 3 of
// keys 2t and 2t + 1 (V, transposed). A mask and an or put two codes n = code + 8
// into the mantissas of a f16 pair: 1024 + n, or from the bits above
// 1024 + 16 n; one subtraction or fma makes them the exact f16 integers n - 8. Nine
// instructions for eight codes. The pairs are (0, 4), (1, 5), (2, 6), (3, 7) of a
// lane's eight; q's fragments and the output's rows are laid out to match.
//
// (As subnormals, n 2^-24, codes would need no arithmetic at all and 8 sum q taken off at
// the start, but the MMA aligns its products by their exponent fields, and what it cuts off
// then is 2^-17 of the sum of magnitudes: scores and results 100 times as far off.)
//
// Scales as over q8_0: K's multiplies the fp32 sum of a 32-dim block, V's the two
// f16 terms of the weights, after a power of two for each block of dims where its scales
// pass 2 or stay below 2^-3 (then 1 to 2 % slower: 134 -> 136, 156 -> 159 us). The MMAs have
// eight columns, and up to four query heads fill half of them: the other four then take the second
// terms, of the weights and of fp32 queries, of the same heads (PACK: half the MMAs; 140 -> 134
// and 176 -> 156 us). With 16-bit activations (bf16 rows are f16 values once scaled by a power of
// two) the MMAs sum O, with fp32 ones each tile's part is added with rounding.
#pragma once

#include "attn_kernel.cuh"

namespace qmm {
namespace attn {

// A tile is two 16-key halves; a warp's ring has two tiles (see attn_launch.cuh).
constexpr int SUB = 2, kRing4 = 2;

template <int D, int NT> struct Layout4 {
    static constexpr int STAGES = kRing4;
    static constexpr int C = D / 32;                        // 32-dim blocks of a row
    static constexpr int ROW = D / 2;                       // bytes of a row's codes
    // row pitch: an odd number of 16 bytes, so that eight rows of a matrix touch every bank once
    static constexpr int RS = ROW / 16 % 2 ? ROW : ROW + 16;
    static constexpr int KT = 16 * SUB;                     // keys per stage
    static constexpr int V0 = KT * RS;                      // K rows, V rows, K scales, V scales
    static constexpr int S0 = 2 * KT * RS, SV = 2 * C * KT;
    static constexpr int STAGE = S0 + 2 * SV;
    static constexpr int RING = STAGES * STAGE;             // of one warp
    static constexpr int OD = D + 4;
    static constexpr int JOIN = kWarps * 8 * NT * OD * 4;
    static constexpr int BYTES = kWarps * RING > JOIN ? kWarps * RING : JOIN;
};

// (x & mask) | bits in one instruction.
__device__ __forceinline__ unsigned and_or(unsigned x, unsigned mask, unsigned bits) {
    unsigned r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
    return r;
}

// Eight codes as four f16 pairs, (0, 4), (1, 5), (2, 6), (3, 7), exactly.
__device__ __forceinline__ void codes4_f16(unsigned w, unsigned (&p)[4]) {
    const __half2 m1032 = __half2half2(__ushort_as_half(0xe408));     // -1032
    const __half2 r16 = __half2half2(__ushort_as_half(0x2c00));       // 1 / 16
    const __half2 m72 = __half2half2(__ushort_as_half(0xd480));       // -72
    const unsigned v = w >> 8;
    p[0] = as_u32(__hadd2(as_half2(and_or(w, 0x000f000fu, 0x64006400u)), m1032));
    p[1] = as_u32(__hfma2(as_half2(and_or(w, 0x00f000f0u, 0x64006400u)), r16, m72));
    p[2] = as_u32(__hadd2(as_half2(and_or(v, 0x000f000fu, 0x64006400u)), m1032));
    p[3] = as_u32(__hfma2(as_half2(and_or(v, 0x00f000f0u, 0x64006400u)), r16, m72));
}

// ONE: pages of 32 keys and more, so that a tile lies in one page.
// PACK: at most four query heads, as columns 0 .. 3 and, their second terms, 4 .. 7.
template <int D, bool HI, int NT, bool ONE, bool PACK>
__device__ __forceinline__ void attn_block_q4(const AttnArgs& a, int splits, int chunk, int head_chunks) {
    using Lay = Layout4<D, NT>;
    constexpr int STAGES = Lay::STAGES;
    static_assert(!PACK || NT == 1);
    // f16 terms of q and of the weights that take an MMA each
    constexpr int NQ = HI && !PACK ? 2 : 1, NP = PACK ? 1 : 2;
    constexpr int C = Lay::C, KT = Lay::KT, ROW = Lay::ROW, RS = Lay::RS;
    constexpr int MT = D / 16;                        // 16-dim tiles of the output

    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float sm_q[8 * NT][D + 4];
    __shared__ float sm_m[kWarps][8 * NT], sm_l[kWarps][8 * NT], sm_scale[8 * NT];
    __shared__ uint2 sm_qf[NT * NQ * MT][32];

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
    auto load_q = [&](auto type) {
        using T = decltype(type);
        const T* q = static_cast<const T*>(a.q) + b * a.q_bs + h0 * a.q_hs;
#pragma unroll
        for (int i = 0; i < QN; ++i) {
            const int j = i * kThreads + threadIdx.x, h = PACK ? j / D % 4 : j / D;
            qv[i] = h < nh ? to_f32<T>(q[h * a.q_hs + j % D]) : 0.f;
        }
    };
    if constexpr (HI) load_q(0.f);
    else if (a.dtype == QMM_F16) load_q(__half());
    else load_q(__nv_bfloat16());
    const int32_t* table = a.table + b * a.table_stride;
    // and the pages of this warp's first tiles, as they are without a window
    int first_page[STAGES];
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
        const int64_t key = static_cast<int64_t>(split) * chunk + (warp + i * kWarps) * KT;
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

    // Pages of a 16-key half: one, or with pages of 8 one for each eight keys.
    // Keys outside the range name a page inside it, so that every address is that of
    // a page the sequence owns.
    const bool small_pages = shift < 4;
    auto page_id = [&](int key) { return table[max(page_lo, min(key >> shift, page_hi))]; };
    auto page_ids = [&](int base, int (&id)[SUB][2]) {
        if constexpr (ONE) {                          // (a tile begins in the page of its first key in range)
            if (base < end) id[0][0] = table[base >> shift];
        } else {
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                id[u][0] = page_id(base + 16 * u);
                if (small_pages) id[u][1] = page_id(base + 16 * u + 8);
            }
        }
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
    // A whole tile inside one page, as most are: its rows are contiguous, and so are its scales.
    const uint32_t dst_lane = lane / CPR * RS + lane % CPR * 16;
    constexpr int SP = KT * C / 8;                    // pieces of K's scales, and of V's
    const uint8_t* const k_lane = kbase + lane * 16;
    const uint8_t* const s_lane = k_lane + (ROW << shift) + (lane >= SP ? v_minus_k - SP * 16 : 0);
    const int64_t page_stride = a.c.page_stride;
    auto load_whole = [&](int base, int id, uint32_t stage) {
        if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.c.n_pages)) {
            bad = true;
            id = 0;
        }
        const int64_t at = static_cast<int64_t>(static_cast<unsigned>(id)) * page_stride;
        const int row = base & page_mask;
        const uint8_t *k = k_lane + at + row * ROW, *v = k + v_minus_k, *sc = s_lane + at + row * (2 * C);
#pragma unroll
        for (int i = 0; i < KT * CPR / 32; ++i) {
            const int q = 32 * i + lane;
            const uint32_t dst = stage + (32 % CPR == 0 ? dst_lane + i * (32 / CPR) * RS : q / CPR * RS + q % CPR * 16);
            copy16(dst, k + i * 512);
            copy16(dst + Lay::V0, v + i * 512);
        }
#pragma unroll
        for (int i = 0; i < (2 * SP + 31) / 32; ++i) {
            const int q = 32 * i + lane;
            if (2 * SP % 32 && q >= 2 * SP) break;
            if constexpr (SP % 32 == 0) copy16(stage + Lay::S0 + q * 16, sc + (i >= SP / 32 ? v_minus_k - SP * 16 : 0) + i * 512);
            else if constexpr (2 * SP <= 32) copy16(stage + Lay::S0 + q * 16, sc);
            else copy16(stage + Lay::S0 + q * 16, k_lane + at + (ROW << shift) + row * (2 * C) + (q >= SP ? v_minus_k - SP * 16 : 0) + i * 512);
        }
    };
    // Rows outside the range are copied like the others: they are masked by their
    // key (K) and have weights and scales of zero (V), and codes are never NaN.
    auto load_tile = [&](int base, const int (&id)[SUB][2], uint32_t stage) {
        if constexpr (ONE) {
            load_whole(base, id[0][0], stage);
        } else {
#pragma unroll
            for (int u = 0; u < SUB; ++u) {               // pages of 16 or 8 keys
                const int first = base + 16 * u, row0 = first & page_mask, row1 = (first + 8) & page_mask;
                const uint8_t* page0 = page_at(id[u][0]);
                const uint8_t* page1 = small_pages ? page_at(id[u][1]) : page0;
                if (lane < 4 * C) {                       // scales: C pieces per eight keys, of K then of V
                    const uint8_t* p = (lane / C & 1 ? page1 + row1 * (2 * C) : page0 + row0 * (2 * C)) + (ROW << shift) + lane % C * 16;
                    copy16(stage + Lay::S0 + u * 32 * C + lane % (2 * C) * 16 + (lane < 2 * C ? 0 : Lay::SV), lane < 2 * C ? p : p + v_minus_k);
                }
                const uint8_t* k0 = page0 + row0 * ROW + lane * 16;
                const uint8_t* k1 = page1 + (row1 - 8) * ROW + lane * 16;
#pragma unroll
                for (int i = 0; i < (ROW + 31) / 32; ++i) {
                    const int q = 32 * i + lane, row = q / CPR;
                    if (ROW % 32 && q >= ROW) break;
                    const uint32_t dst = stage + 16 * u * RS + (32 % CPR == 0 ? dst_lane + i * (32 / CPR) * RS : row * RS + q % CPR * 16);
                    const uint8_t* src = ((ROW / 2) % 32 == 0 ? 32 * i >= ROW / 2 : row >= 8) ? k1 : k0;
                    copy16(dst, src + i * 512);
                    copy16(dst + Lay::V0, src + v_minus_k + i * 512);
                }
            }
        }
    };
    constexpr int stride = kWarps * KT;
    int base = begin + warp * KT;
    int id[SUB][2];                                   // pages of the next tile to load
    int ahead = base;                                 // its first key
    const bool known = ONE && rg.lo16 == 0;
    if (known) id[0][0] = first_page[0];
    else page_ids(ahead, id);
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
        if (ahead < end) {
            load_tile(ahead, id, ring + i * Lay::STAGE);
            ahead += stride;
            if (known) id[0][0] = first_page[i + 1];
            else page_ids(ahead, id);
        }
        copies_commit();
    }

    // ---- the query fragments in shared memory: B operand, column g = head
#pragma unroll
    for (int i = 0; i < QN; ++i) {
        const int j = i * kThreads + threadIdx.x;
        sm_q[j / D][j % D] = qv[i];
    }
    __syncthreads();
    const bool norm = HI || a.dtype != QMM_F16;       // rows scaled into the middle of f16's range
    if (norm) {
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
    float sc[NT][2];                                  // score scale of heads 2t, 2t + 1, to log2 units unless capped
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float f = norm ? sm_scale[8 * n + g] : 1.f;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            if (j % kWarps != warp) continue;
            unsigned w[NQ][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                // codes 2 (j % 2) + k and that + 4 of the lane's eight
                const int d = j / 2 * 32 + 8 * t + 2 * (j % 2) + k;
                float x0 = sm_q[8 * n + g][d] * f, x1 = sm_q[8 * n + g][d + 4] * f;
#pragma unroll
                for (int q = 0; q < NQ; ++q) w[q][k] = take16<false>(x0, x1);
                if constexpr (PACK && HI) {
                    const unsigned second = take16<false>(x0, x1);
                    w[0][k] = g < 4 ? w[0][k] : second;
                }
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q) sm_qf[(n * NQ + q) * MT + j][lane] = make_uint2(w[q][0], w[q][1]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            sc[n][k] = a.scale * (a.softcap > 0.f ? 1.f : kLog2e);
            if (norm) sc[n][k] /= sm_scale[8 * n + 2 * t + k];
        }
    }
    __syncthreads();

    // Weights are 2^(score - ref) <= 2^kTop (see attn_kernel.cuh)
    constexpr float kTop = 14.f, kNone = -3.402823466e38f;
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
    // V's scales, of either sign, are multiplied by a power of two that keeps them
    // below 2 (the weights' terms below 2^15) and a block's largest at 2^-3 or more, one for each
    // 32-dim block: a block of small scales keeps its bits beside one of large ones. O carries the
    // factor. None is applied where all are 1.
    __half2 v_mul[C];
    bool v_scaled = true;
#pragma unroll
    for (int c = 0; c < C; ++c) v_mul[c] = __float2half2_rn(32768.f);

    // matrix mi of an ldmatrix: lanes 8 mi .. 8 mi + 7 give its rows; keys 0 .. 7 and
    // 8 .. 15 of a block, then of the next block (or, of an odd last one, the same again)
    const int mi = lane / 8, mr = lane % 8;
    const uint32_t m_row = (mr + 8 * (mi & 1)) * RS, m_lane = m_row + 16 * (mi >> 1);
    uint32_t stage = ring, fill = ring + (STAGES - 1) * Lay::STAGE;
    const uint32_t ring_end = ring + Lay::RING, smem_base = smem_addr(smem);

    // One tile. SLOW: some keys are masked, or scores are capped.
    auto tile = [&](auto slow_tag) {
        constexpr bool SLOW = decltype(slow_tag)::value;
        const uint8_t* scales = smem + (stage - smem_base) + Lay::S0;
        // ---- S^T = K Q^T
        float sx[SUB][NT][4];
        __half kscale[SUB][2][C];                     // of keys g, g + 8
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            constexpr int B = C % 4 == 0 ? 8 : C % 2 == 0 ? 4 : 2;
            using SVec = typename VecOf<B>::type;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2 * C / B; ++k) {
                    const SVec x = reinterpret_cast<const SVec*>(scales + (16 * u + g + 8 * i) * (2 * C))[k];
#pragma unroll
                    for (int j = 0; j < B / 2; ++j) kscale[u][i][k * (B / 2) + j] = reinterpret_cast<const __half*>(&x)[j];
                }
        }
#pragma unroll
        for (int c2 = 0; c2 < C; c2 += 2) {
            unsigned w[SUB][4];
#pragma unroll
            for (int u = 0; u < SUB; ++u) ldsm4(w[u], stage + u * 16 * RS + (c2 + 1 < C ? m_lane : m_row) + 16 * c2);
#pragma unroll
            for (int c = c2; c < c2 + 2 && c < C; ++c) {
                uint2 f[NT][NQ][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
#pragma unroll
                        for (int j = 0; j < 2; ++j) f[n][q][j] = sm_qf[(n * NQ + q) * MT + 2 * c + j][lane];
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    unsigned x0[4], x1[4];            // keys g, g + 8
                    codes4_f16(w[u][2 * (c - c2)], x0);
                    codes4_f16(w[u][2 * (c - c2) + 1], x1);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int q = NQ - 1; q >= 0; --q)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                mma<false>(acc, x0[2 * j], x1[2 * j], x0[2 * j + 1], x1[2 * j + 1], f[n][q][j].x, f[n][q][j].y);
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const float d = __half2float(kscale[u][i >> 1][c]);
                            const float2 x = fma2(make_float2(d, d), make_float2(acc[i], acc[i + 1]),
                                                  c == 0 ? make_float2(0.f, 0.f) : make_float2(sx[u][n][i], sx[u][n][i + 1]));
                            sx[u][n][i] = x.x;
                            sx[u][n][i + 1] = x.y;
                        }
                    }
                }
            }
        }

        if constexpr (PACK && HI) {                   // both terms' scores
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) sx[u][0][i] += __shfl_xor_sync(0xffffffffu, sx[u][0][i], 2);
        }

        // ---- scores, less ref, in log2 units
        if constexpr (SLOW) {
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x = sx[u][n][i] * sc[n][i & 1];
                        if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
                        const int key = base + 16 * u + 8 * (i >> 1) + g;
                        if (key < rg.lo || key >= end) x = -INFINITY;
                        sx[u][n][i] = x;
                    }
        }
        auto rel = [&](int u, int n, int i) {         // not fused (see attn_kernel.cuh)
            return SLOW ? (sx[u][n][i] - ref[n][i & 1]) * unit : __fmul_rn(sx[u][n][i], sc[n][i & 1]) - ref[n][i & 1];
        };
        float y[SUB][NT][4];
        float most = -INFINITY;
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[u][n][i] = rel(u, n, i);
                    most = fmaxf(most, y[u][n][i]);
                }
        const bool grew = most > kTop;
        // V scales of keys (2t, 2t + 1) and (2t + 8, 2t + 9) as stored
        auto v_scales = [&](unsigned (&vd)[SUB][2][C]) {
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t* p = scales + Lay::SV + (16 * u + 2 * t + 8 * i) * (2 * C);
                    if constexpr (C % 2 == 0) {
                        constexpr int B = C % 4 == 0 ? 8 : 4;
                        using SVec = typename VecOf<B>::type;
#pragma unroll
                        for (int k = 0; k < 2 * C / B; ++k) {
                            const SVec x = reinterpret_cast<const SVec*>(p)[k], z = reinterpret_cast<const SVec*>(p + 2 * C)[k];
#pragma unroll
                            for (int j = 0; j < B / 4; ++j) {
                                const unsigned s0 = reinterpret_cast<const unsigned*>(&x)[j];
                                const unsigned s1 = reinterpret_cast<const unsigned*>(&z)[j];
                                vd[u][i][k * (B / 2) + 2 * j] = __byte_perm(s0, s1, 0x5410);
                                vd[u][i][k * (B / 2) + 2 * j + 1] = __byte_perm(s0, s1, 0x7632);
                            }
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < C; ++c)
                            vd[u][i][c] = reinterpret_cast<const unsigned short*>(p)[c] |
                                          static_cast<unsigned>(reinterpret_cast<const unsigned short*>(p + 2 * C)[c]) << 16;
                    }
                    if constexpr (SLOW) {                 // rows outside the range are zeros, their scales are not
                        const int key = base + 16 * u + 8 * i + 2 * t;
                        const unsigned keep = (key >= rg.lo && key < end ? 0xffffu : 0u) |
                                              (key + 1 >= rg.lo && key + 1 < end ? 0xffff0000u : 0u);
#pragma unroll
                        for (int c = 0; c < C; ++c) vd[u][i][c] &= keep;
                    }
                }
        };
        unsigned vd[SUB][2][C];                       // those scales times v_mul
        v_scales(vd);
        if (v_scaled) {
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < C; ++c) vd[u][i][c] = as_u32(__hmul2(as_half2(vd[u][i][c]), v_mul[c]));
        }
        unsigned v_bits = 0u;
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < C; ++c) v_bits |= vd[u][i][c];
        const bool v_grew = v_bits & 0x40004000u;     // an exponent of 2 and more
        if (__any_sync(0xffffffffu, grew || v_grew)) {
            float up[C];                              // change of O's factors
#pragma unroll
            for (int c = 0; c < C; ++c) up[c] = 1.f;
            if (__any_sync(0xffffffffu, v_grew)) {
                v_scales(vd);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    __half2 m = __float2half2_rn(0.f);
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int i = 0; i < 2; ++i) m = __hmax2(m, __habs2(as_half2(vd[u][i][c])));
                    const unsigned w = as_u32(m);
                    const unsigned big = __reduce_max_sync(0xffffffffu, max(w & 0xffffu, w >> 16));
                    // below 2^(field - 14) by the exponent's field: from 2^-3 up to 2 they stay,
                    // larger ones go below 1, smaller ones to 1/4 .. 1/2. (Products of a scale and a
                    // weight are held to 2^-25: what a scale is below 1, they lose in bits.)
                    const int field = static_cast<int>(big >> 10);
                    const int e = field >= 16 ? 14 - field : field >= 12 ? 0 : 13 - field;
                    const __half2 mul = __hmin2(v_mul[c], __float2half2_rn(exp2f(static_cast<float>(max(-15, min(15, e))))));
                    up[c] = __low2float(mul) / __low2float(v_mul[c]);
                    v_mul[c] = mul;
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int i = 0; i < 2; ++i) vd[u][i][c] = as_u32(__hmul2(as_half2(vd[u][i][c]), mul));
                }
                v_scaled = false;
#pragma unroll
                for (int c = 0; c < C; ++c) v_scaled |= __low2float(v_mul[c]) != 1.f;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float alpha[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float mt = -INFINITY;
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
                        mt = fmaxf(mt, SLOW ? fmaxf(sx[u][n][k], sx[u][n][k + 2])
                                            : fmaxf(__fmul_rn(sx[u][n][k], sc[n][k]), __fmul_rn(sx[u][n][k + 2], sc[n][k])));
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
                    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                    // from 2^24 on the maximum itself is the reference (see attn_kernel.cuh)
                    float now = mt - top;
                    if ((mt - now) * unit > kTop + 1.f) now = mt;
                    now = fmaxf(ref[n][k], now);
                    alpha[k] = ex2((ref[n][k] - now) * unit);
                    ref[n][k] = now;
                    l[n][k] *= alpha[k];
                }
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][j][i] *= alpha[i & 1] * up[j / 2];
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[u][n][i] = rel(u, n, i);
            }
        }
        // ---- weights, as the B operand of the second product: O^T += V^T P^T. A weight
        // times V's scale is held to 2^-25, so that a small one keeps few bits, and where those of the
        // large ones meet values of zero it is all there is. With wide activations, a tile that has
        // weights below 2^-21 of the largest takes them in bands of 2^21, each scaled into
        // range: with scales of 2^-3 the least of a band is still off by no more than 2^-15. It costs
        // nothing where scores stay within 14 of the largest (64 x 8192, fp32 q: 157 us); scores that spread
        // by 3.2 take 238 us, by 6.4 323. (Bands from 2^-32 on took 194 and 279, and left weights of
        // 2^-24 with errors of up to 2^-12, those of 2^-32 with 2^-4.)
        constexpr float kLow = -7.f, kBand = 21.f;
        constexpr int kBands = 5;                     // down to 2^-105 of the largest
        auto in_band = [&](float x, int k) {
            const float lo = kLow - kBand * static_cast<float>(k);
            return x >= lo && (k == 0 || x < lo + kBand);
        };
        unsigned bands = 1;                           // those that have a weight in this tile
        if constexpr (HI) {
            float least = INFINITY;
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) least = fminf(least, y[u][n][i]);
            if (__any_sync(0xffffffffu, least < kLow)) {
#pragma unroll 1
                for (int k = 1; k < kBands; ++k) {
                    bool in = false;
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) in |= in_band(y[u][n][i], k);
                    bands |= (__any_sync(0xffffffffu, in) ? 1u : 0u) << k;
                }
            }
        }
#pragma unroll 1
        for (int k = 0; k < kBands; ++k) {
            if (HI && !(bands >> k & 1)) {
                if (bands >> k == 0) break;
                continue;
            }
            [[maybe_unused]] const float down = HI ? ex2(-kBand * static_cast<float>(k)) : 1.f;
            unsigned pf[SUB][NT][2][2];
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = ex2(HI ? y[u][n][i] + kBand * static_cast<float>(k) : y[u][n][i]);
                        if (HI && bands > 1 && !in_band(y[u][n][i], k)) x[i] = isnan(x[i]) ? x[i] : 0.f;
                        if (HI) l[n][i & 1] = fmaf(x[i], down, l[n][i & 1]);
                        else l[n][i & 1] += x[i];
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        unsigned lo = take16<false>(x[0], x[1]), hi = take16<false>(x[2], x[3]);
                        if (PACK && q == 1 && t < 2) lo = hi = 0u;
                        pf[u][n][q][0] = transpose8x8(lo);
                        pf[u][n][q][1] = transpose8x8(hi);
                    }
                }
            [[maybe_unused]] unsigned minus[SUB][2];  // -hi, or 0 where hi d is wanted itself
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) minus[u][i] = g < 4 ? 0u : pf[u][0][0][i] ^ 0x80008000u;
#pragma unroll
            for (int c2 = 0; c2 < C; c2 += 2) {
                unsigned w[SUB][4];
#pragma unroll
                for (int u = 0; u < SUB; ++u)
                    ldsm4_trans(w[u], stage + Lay::V0 + u * 16 * RS + (c2 + 1 < C ? m_lane : m_row) + 16 * c2);
#pragma unroll
                for (int c = c2; c < c2 + 2 && c < C; ++c) {
                    unsigned pd[SUB][NT][NP][2];      // p times the block's scale, in two terms
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const __half2 d = as_half2(vd[u][i][c]);
                                const __half2 hi = as_half2(pf[u][n][0][i]), lo = as_half2(pf[u][n][1][i]);
                                if constexpr (PACK) {     // columns 0 .. 3: hi d + 0; the others what that has left
                                    const __half2 t1 = __hmul2_rn(as_half2(minus[u][i]), d);
                                    pd[u][n][0][i] = as_u32(__hfma2(lo, d, __hfma2(hi, d, t1)));
                                } else {
                                    const __half2 t1 = __hmul2_rn(hi, d);
                                    pd[u][n][0][i] = as_u32(t1);
                                    pd[u][n][1][i] = as_u32(__hfma2(lo, d, __hfma2(hi, d, __hneg2(t1))));
                                }
                            }
                    // the MMA's sum cuts off what does not fit in 24 bits: with HI the tile's
                    // products are summed apart and added to O with rounding
                    float apart[HI ? NT : 1][2][4];
                    if constexpr (HI) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 8; ++i) apart[n][i / 4][i % 4] = 0.f;
                    }
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        unsigned f0[4], f1[4];        // keys 0 .. 7, 8 .. 15 of the half
                        codes4_f16(w[u][2 * (c - c2)], f0);
                        codes4_f16(w[u][2 * (c - c2) + 1], f1);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int q = NP - 1; q >= 0; --q)
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    mma<false>(HI ? apart[n][j] : o[n][2 * c + j], f0[2 * j], f0[2 * j + 1], f1[2 * j], f1[2 * j + 1],
                                               pd[u][n][q][0], pd[u][n][q][1]);
                    }
                    if constexpr (HI) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
#pragma unroll
                                for (int i = 0; i < 4; i += 2) {
                                    float* to = &o[n][2 * c + j][i];
                                    const float2 x = fma2(make_float2(apart[n][j][i], apart[n][j][i + 1]), make_float2(down, down),
                                                          make_float2(to[0], to[1]));
                                    to[0] = x.x;
                                    to[1] = x.y;
                                }
                    }
                }
            }
            if constexpr (!HI) break;
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
    float v_div[C];
#pragma unroll
    for (int c = 0; c < C; ++c) v_div[c] = 1.f / __low2float(v_mul[c]);
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
                // rows g and g + 8 of a tile: codes 2 (j % 2) and the next of four
                const int d = j / 2 * 32 + 4 * g + 2 * (j % 2) + (i >> 1);
                p[(i & 1) * OD + d] = o[n][j][i] * v_div[j / 2];
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
            float4 v = *reinterpret_cast<const float4*>(&sm_o[(w * 8 * NT + h) * OD + d]);
            if constexpr (PACK) {
                const float4 low = *reinterpret_cast<const float4*>(&sm_o[(w * 8 * NT + h + 4) * OD + d]);
                v = make_float4(v.x + low.x, v.y + low.y, v.z + low.z, v.w + low.w);
            }
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

template <int D, bool HI, int NT, int MINB, bool ONE, bool PACK>
__global__ void __launch_bounds__(kThreads, MINB)
    k_attn_q4(const __grid_constant__ AttnArgs a, int splits, int chunk, int head_chunks) {
    grid_dep_launch();
    grid_dep_wait();
    attn_block_q4<D, HI, NT, ONE, PACK>(a, splits, chunk, head_chunks);
}

}  // namespace attn
}  // namespace qmm
