// attn_launch.cuh -- the kernel choice of one cache format (included by one
// translation unit per format).
#pragma once

#include <atomic>

#include "attn_kernel.cuh"

namespace qmm {
namespace attn {

// Shared memory beyond 48 KB has to be allowed once per kernel and device.
template <int FMT, int D, bool HI, int NT, int STAGES, int MINB>
cudaError_t go_with(const AttnArgs& a, const AttnPlan& p, int64_t blocks, int head_chunks, cudaStream_t s) {
    constexpr int bytes = Layout<FMT, D, NT, STAGES>::BYTES;
    auto kernel = k_attn<FMT, D, HI, NT, STAGES, MINB>;
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    kernel<<<static_cast<unsigned>(blocks), kThreads, bytes, s>>>(a, p.splits, p.chunk, head_chunks);
    count_launch(1);
    return cudaGetLastError();
}

template <int FMT, int D, bool HI, int NT>
cudaError_t go(const AttnArgs& a, const AttnPlan& p, int64_t blocks, int head_chunks, cudaStream_t s) {
    return go_with<FMT, D, HI, NT, 3, 2>(a, p, blocks, head_chunks, s);
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
