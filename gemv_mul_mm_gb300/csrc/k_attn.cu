// k_attn.cu -- qattn_decode: the split over the length, the launch and the join.
#include <algorithm>

#include "attn_kernel.cuh"

namespace qmm {
namespace attn {
namespace {

constexpr int kJoinThreads = 256;

// o = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s of one head of one sequence
// per block, in split order within each of the block's lanes' groups
// (deterministic). A group of D / 4 threads adds every GROUPS-th split.
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(const __grid_constant__ AttnArgs a, int splits, int chunk) {
    grid_dep_wait();
    const int64_t bh = blockIdx.x;
    const Range r = range_of(a, bh / a.Hq, chunk);
    if (r.splits <= 1) return;
    __shared__ float sm[kJoinThreads * 4];
    __shared__ float sl[kJoinThreads];
    const int D = a.c.D, per = D / 4, groups = kJoinThreads / per;
    const int grp = threadIdx.x / per, v = threadIdx.x % per;
    const float2* ml = ws_ml(a, splits, bh, 0);
    float m = -INFINITY;
    for (int s = threadIdx.x % 32; s < r.splits; s += 32) m = fmaxf(m, ml[s].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    if (grp < groups) {
        const float4* O = reinterpret_cast<const float4*>(ws_o(a, splits, bh, 0)) + v;
#pragma unroll 4
        for (int s = grp; s < r.splits; s += groups) {
            const float2 p = ml[s];
            const float4 x = O[static_cast<int64_t>(s) * per];
            const float f = p.x == -INFINITY ? 0.f : ex2(p.x - m);
            l += p.y == 0.f ? 0.f : f * p.y;
            acc.x = fmaf(f, x.x, acc.x);
            acc.y = fmaf(f, x.y, acc.y);
            acc.z = fmaf(f, x.z, acc.z);
            acc.w = fmaf(f, x.w, acc.w);
        }
        reinterpret_cast<float4*>(sm)[grp * per + v] = acc;
        if (v == 0) sl[grp] = l;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kJoinThreads) {
        float o = 0.f, ll = 0.f;
        for (int i = 0; i < groups; ++i) {
            o += sm[i * D + d];
            ll += sl[i];
        }
        store_act(a.out, a.dtype, bh * D + d, o / ll);
        if (a.lse && d == 0) a.lse[bh] = m * kLn2 + logf(ll);
    }
}

}  // namespace
}  // namespace attn

bool attn_dim_ok(int D) { return D == 64 || D == 96 || D == 128 || D == 256; }

AttnPlan attn_plan(int fmt, int dtype, int64_t B, int Hq, int Hkv, int D, int max_len, int window, int sms) {
    (void)fmt;
    (void)dtype;
    AttnPlan p;
    const int group = Hq / Hkv;
    p.tiles = group > 8 && D <= 128 ? 2 : 1;
    const int head_chunks = (group + 8 * p.tiles - 1) / (8 * p.tiles);
    const int64_t items = B * Hkv * head_chunks;
    const int64_t keys = std::max<int64_t>(1, window > 0 ? std::min<int64_t>(max_len, window + 15) : max_len);
    const int64_t step = 64;                           // four warps of 16 keys
    const int64_t steps = (keys + step - 1) / step;
    const int64_t slots = static_cast<int64_t>(sms) * 3;
    // The split count with the least cost in steps: waves of blocks, times the
    // steps of a block and its fixed part (query, join). Only counts that fill
    // a whole number of waves can be best.
    int64_t best = 1;
    double best_cost = 1e300;
    for (int64_t w = 0; w <= 6; ++w) {
        const int64_t s = w == 0 ? 1 : std::min<int64_t>({w * slots / items, steps, 512});
        if (s < 1) continue;
        const int64_t per = (steps + s - 1) / s;
        const int64_t n = (steps + per - 1) / per;
        const double waves = static_cast<double>((items * n + slots - 1) / slots);
        const double cost = waves * (per + 4.0) + (n > 1 ? 4.0 + 0.02 * n : 0.0);
        if (cost < best_cost) {
            best_cost = cost;
            best = n;
        }
    }
    const int64_t per = (steps + best - 1) / best;
    p.chunk = static_cast<int>(per * step);
    p.splits = static_cast<int>((keys + p.chunk - 1) / p.chunk);
    p.ws_bytes = p.splits > 1 ? static_cast<size_t>(B) * Hq * p.splits * (D * 4 + 8) : 0;
    return p;
}

cudaError_t launch_attn(const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
    const int group = a.Hq / a.c.heads;
    const int head_chunks = (group + 8 * p.tiles - 1) / (8 * p.tiles);
    const int64_t blocks = a.B * a.c.heads * head_chunks * p.splits;
    if (blocks > 0x7fffffff || a.B * a.Hq > 0x7fffffff) return cudaErrorInvalidValue;
    cudaError_t e;
    switch (a.c.fmt) {
    case QMM_KV_F16: e = attn::launch_fmt<QMM_KV_F16>(a, p, blocks, head_chunks, s); break;
    case QMM_KV_BF16: e = attn::launch_fmt<QMM_KV_BF16>(a, p, blocks, head_chunks, s); break;
    default: e = attn::launch_fmt<QMM_KV_Q8_0>(a, p, blocks, head_chunks, s); break;
    }
    if (e != cudaSuccess || p.splits == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B * a.Hq));
    cfg.blockDim = dim3(attn::kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attn::k_attn_join, a, p.splits, p.chunk);
    count_launch(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace qmm
