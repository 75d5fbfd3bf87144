// attn_launch.cuh -- the kernel choice of one cache format (included by one
// translation unit per format).
#pragma once

#include "attn_kernel.cuh"

namespace qmm {
namespace attn {

template <int FMT, int D, bool HI, int NT>
cudaError_t go(const AttnArgs& a, const AttnPlan& p, int64_t blocks, int head_chunks, cudaStream_t s) {
    k_attn<FMT, D, HI, NT, 1, 1><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a, p.splits, p.chunk, head_chunks);
    count_launch(1);
    return cudaGetLastError();
}

template <int FMT, int D>
cudaError_t pick(const AttnArgs& a, const AttnPlan& p, int64_t blocks, int head_chunks, cudaStream_t s) {
    const bool hi = needs_hi(FMT, a.dtype);
    if constexpr (D <= 128) {
        if (p.tiles == 2) return hi ? go<FMT, D, true, 2>(a, p, blocks, head_chunks, s) : go<FMT, D, false, 2>(a, p, blocks, head_chunks, s);
    }
    return hi ? go<FMT, D, true, 1>(a, p, blocks, head_chunks, s) : go<FMT, D, false, 1>(a, p, blocks, head_chunks, s);
}

template <int FMT>
cudaError_t launch_fmt(const AttnArgs& a, const AttnPlan& p, int64_t blocks, int head_chunks, cudaStream_t s) {
    switch (a.c.D) {
    case 64: return pick<FMT, 64>(a, p, blocks, head_chunks, s);
    case 96: return pick<FMT, 96>(a, p, blocks, head_chunks, s);
    case 128: return pick<FMT, 128>(a, p, blocks, head_chunks, s);
    default: return pick<FMT, 256>(a, p, blocks, head_chunks, s);
    }
}

template cudaError_t launch_fmt<QMM_ATTN_FMT>(const AttnArgs&, const AttnPlan&, int64_t, int, cudaStream_t);

}  // namespace attn
}  // namespace qmm
