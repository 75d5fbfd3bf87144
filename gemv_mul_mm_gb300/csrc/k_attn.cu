// k_attn.cu -- qattn_decode: the split over the length, the launch and the join.
#include <algorithm>
#include <cmath>

#include "attn_kernel.cuh"

namespace qmm {
namespace attn {
namespace {

constexpr int kJoinThreads = 256;

// o = sum_s e^(m_s - m) O_s / sum_s e^(m_s - m) l_s of one head of one sequence
// per block, in split order within each of the block's lanes' groups
// (deterministic). A group of D / 4 threads adds every GROUPS-th split.
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(const __grid_constant__ AttnArgs a, int splits, int chunk) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t bh = blockIdx.x;
    const Range r = range_of(a, bh / a.Hq, chunk);
    if (r.splits <= 1) return;
    __shared__ float sm[kJoinThreads * 4];
    __shared__ float sm_m[kJoinThreads], sm_l[kJoinThreads];
    const int D = a.c.D, per = D / 4, groups = kJoinThreads / per;
    const int grp = threadIdx.x / per, v = threadIdx.x % per;
    const float2* ml = ws_ml(a, splits, bh, 0);
    const float unit = unit_of(a);
    if (grp < groups) {
        const float4* O = reinterpret_cast<const float4*>(ws_o(a, splits, bh, 0)) + v;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float m = -INFINITY, l = 0.f;
#pragma unroll 4
        for (int s = grp; s < r.splits; s += groups) {
            const float2 p = ml[s];
            const float4 x = O[static_cast<int64_t>(s) * per];
            const float top = fmaxf(m, p.x);
            const float old = m == -INFINITY ? 0.f : ex2((m - top) * unit), f = p.x == -INFINITY ? 0.f : ex2((p.x - top) * unit);
            m = top;
            l = l * old + (p.y == 0.f ? 0.f : f * p.y);
            acc.x = fmaf(f, x.x, acc.x * old);
            acc.y = fmaf(f, x.y, acc.y * old);
            acc.z = fmaf(f, x.z, acc.z * old);
            acc.w = fmaf(f, x.w, acc.w * old);
        }
        reinterpret_cast<float4*>(sm)[grp * per + v] = acc;
        if (v == 0) {
            sm_m[grp] = m;
            sm_l[grp] = l;
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kJoinThreads) {
        float m = -INFINITY, o = 0.f, l = 0.f;
        for (int i = 0; i < groups; ++i) m = fmaxf(m, sm_m[i]);
        for (int i = 0; i < groups; ++i) {
            const float f = sm_m[i] == -INFINITY ? 0.f : ex2((sm_m[i] - m) * unit);
            o = fmaf(f, sm[i * D + d], o);
            l += sm_l[i] == 0.f ? 0.f : f * sm_l[i];
        }
        store_act(a.out, a.dtype, bh * D + d, o / l);
        if (a.lse && d == 0) a.lse[bh] = lse_of(a, m, l);
    }
}

cudaError_t launch_one(const Launch& l, int fmt, int D) {
    switch (fmt) {
    case QMM_KV_F16: return launch_fmt<QMM_KV_F16>(l, D, l.p.hi, l.p.tiles);
    case QMM_KV_BF16: return launch_fmt<QMM_KV_BF16>(l, D, l.p.hi, l.p.tiles);
    case QMM_KV_Q4_0: return launch_fmt<QMM_KV_Q4_0>(l, D, l.p.hi, l.p.tiles);
    default: return launch_fmt<QMM_KV_Q8_0>(l, D, l.p.hi, l.p.tiles);
    }
}

}  // namespace
}  // namespace attn

bool attn_dim_ok(int D) { return D == 64 || D == 96 || D == 128 || D == 192 || D == 256; }

cudaError_t attn_plan(int fmt, int dtype, int64_t B, int Hq, int Hkv, int D, int max_len, int window, int sms, AttnPlan* p) {
    const int group = Hq / Hkv;
    // Query heads per block: 16 halve the reads of a group of more than 8 (above
    // dim 128 there are no registers for them).
    p->tiles = group > 8 && D <= 128 ? 2 : 1;
    p->head_chunks = (group + 8 * p->tiles - 1) / (8 * p->tiles);
    p->hi = attn::needs_hi(fmt, dtype);
    p->pack = fmt == QMM_KV_Q4_0 && group <= 4;
    int resident = 0;
    attn::Launch l{};
    l.p = *p;
    l.resident = &resident;
    const cudaError_t e = attn::launch_one(l, fmt, D);
    if (e != cudaSuccess) return e;
    const int64_t items = B * Hkv * p->head_chunks;
    const int tile = fmt == QMM_KV_Q4_0 ? 32 : 16;               // a window begins inside one
    const int64_t keys = window > 0 ? std::min<int64_t>(max_len, static_cast<int64_t>(window) + tile - 1) : max_len;
    const int64_t step = attn::kWarps * tile;                    // keys that a block's warps take at once
    const int64_t steps = (keys + step - 1) / step;
    // The split count n with the least expected time, in steps of 64 keys (an SM
    // takes 0.5 to 0.7 us for one, and q8_0 a quarter more for each block
    // missing from a full SM): the steps of the busiest SM, plus a block's
    // fixed part (8: query, first loads, warps joined), which further waves hide
    // where memory bounds them and a neighbour is resident, plus the join. Candidates give every SM a whole number of
    // blocks, or are powers of two. Lengths are known on the device only: a
    // batch is taken to be anything between its bound and half of it. A
    // smaller count wins within 3 %.
    // Over q4_0 a step is 128 keys and takes an SM 0.9 us with one block, 1.8 with three, and
    // the fixed parts, in those steps, are half and a quarter of the above.
    const bool q4 = fmt == QMM_KV_Q4_0;
    const double fixed = q4 ? 4.0 : 8.0, join = q4 ? 2.0 : 4.0;
    auto busiest = [&](double blocks, int64_t per) {
        const double load = blocks / sms, waves = std::ceil(load / resident);
        const double idle = (fmt == QMM_KV_Q8_0 || q4) && load < resident ? resident - std::ceil(load) : 0.0;
        return (load <= resident ? std::ceil(load) : load + 0.5) * (1.0 + 0.25 * idle) * static_cast<double>(per) + fixed +
               (fmt == QMM_KV_Q8_0 || resident <= (q4 ? 2 : 1) ? 8.0 : 2.0) * (waves - 1);
    };
    auto cost = [&](int64_t n, int64_t per) {
        const double full = busiest(static_cast<double>(items) * n, per);
        const double half = B >= 4 ? busiest(0.5 * static_cast<double>(items) * n, per) : full;
        return 0.5 * (full + half) + (n > 1 ? join + 0.02 * static_cast<double>(n) : 0.0);
    };
    // Without HI the MMAs sum a block's keys, cutting off bits (see the kernel):
    // 16384 keys are 1.2e-5 of the result, little against a 16-bit output's own
    // rounding, and more are not taken.
    const int64_t least = p->hi ? 1 : (steps * step + 16383) / 16384;
    // More than 64 blocks per SM are not made (only sequences of a million
    // keys and batches that nearly fill the memory would take them): the workspace
    // has a bound that grows with the sizes, though the count itself does not.
    const int64_t blocks = static_cast<int64_t>(64) * sms;
    int64_t best = least;
    double best_cost = cost(best, (steps + best - 1) / best);
    const int64_t most = std::max(least, std::min<int64_t>({steps, 512, blocks / items}));
    for (int i = 0; i < 18; ++i) {
        int64_t s = i < 9 ? int64_t(2) << i : (i - 8) * sms / items;
        if (q4) s = std::min(s, most);
        if (s < 2 || s <= least || s > most) continue;
        const int64_t per = (steps + s - 1) / s, n = (steps + per - 1) / per;
        const double c = cost(n, per);
        if (n < best ? c <= best_cost * 1.03 : c < best_cost * 0.97) {
            best_cost = c;
            best = n;
        }
    }
    const int64_t per = (steps + best - 1) / best;
    p->chunk = static_cast<int>(per * step);
    p->splits = static_cast<int>(best);
    // Partial results at most: those of the most splits that this batch and any
    // smaller one, these lengths and any shorter ones, can have.
    const int64_t heads = B * Hq, any = std::max(least, std::min<int64_t>(steps, 512));
    const int64_t parts = std::min(heads * any, std::max(heads * least, (blocks * group + p->head_chunks - 1) / p->head_chunks));
    p->ws_bytes = any > 1 ? static_cast<size_t>(parts) * (D * 4 + 8) : 0;
    return cudaSuccess;
}

cudaError_t launch_attn(const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
    const int64_t blocks = a.B * a.c.heads * p.head_chunks * p.splits;
    if (blocks > 0x7fffffff || a.B * a.Hq > 0x7fffffff) return cudaErrorInvalidValue;
    const attn::Launch l{a, p, blocks, s, nullptr};
    const cudaError_t e = attn::launch_one(l, a.c.fmt, a.c.D);
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_chained(attn::k_attn_join, dim3(static_cast<unsigned>(a.B * a.Hq)), attn::kJoinThreads, 0, s, a, p.splits,
                          p.chunk);
}

}  // namespace qmm
