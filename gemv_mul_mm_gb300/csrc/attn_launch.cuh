// attn_launch.cuh -- the kernel choice of one cache format (included by one
// translation unit per format; that of q4_0 defines QMM_ATTN_Q4).
#pragma once

#include <atomic>

#include "attn_kernel.cuh"

namespace qmm {
namespace attn {

// Shared memory beyond 48 KB has to be allowed once per kernel and device; the
// resident blocks are looked up at the same time (`fits`, one of each kernel).
constexpr int kDevices = 64;
template <typename K> cudaError_t launch_kernel(const Launch& l, K kernel, int bytes, std::atomic<int> (&fits)[kDevices]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int n = dev < kDevices ? fits[dev].load(std::memory_order_acquire) : 0;
    if (n == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, bytes);
        if (e == cudaSuccess && n < 1) e = cudaErrorInvalidConfiguration;
        if (e != cudaSuccess) {
            cudaGetLastError();
            return e;
        }
        if (dev < kDevices) fits[dev].store(n, std::memory_order_release);
    }
    if (l.resident) *l.resident = n;
    if (l.blocks == 0) return cudaSuccess;
    return launch_chained(kernel, dim3(static_cast<unsigned>(l.blocks)), kThreads, bytes, l.stream, l.a, l.p.splits, l.p.chunk,
                          l.p.head_chunks);
}

#ifdef QMM_ATTN_Q4
template <int D, bool HI, int NT, int MINB, bool PACK> cudaError_t go_with(const Launch& l) {
    static std::atomic<int> fits[kDevices], fits_small[kDevices];
    constexpr int bytes = Layout4<D, NT>::BYTES;
    // (a plan, without blocks, has no page size)
    if (l.blocks && (1 << l.a.c.page_shift) < Layout4<D, NT>::KT)
        return launch_kernel(l, k_attn_q4<D, HI, NT, MINB, false, PACK>, bytes, fits_small);
    return launch_kernel(l, k_attn_q4<D, HI, NT, MINB, true, PACK>, bytes, fits);
}

// Blocks per SM, keys per tile and depth of the ring, measured on 64 sequences of 8192
// tokens and on one of 131072 (f16 activations, 8 key-value heads of 128). A warp's chain of
// instructions bounds the kernel, three warps a scheduler: 63 % of the issue slots, no pipe above
// half. Tiles of 32 keys, two stages and three blocks take 134 and 39 us, four blocks
// 135 and 43. (With an MMA for each term, 140 and 40 us, tiles of 16 keys took 154 and 47, of
// 64 155 and 43, three stages 142 and 42.) Dim 64 fits four blocks (64 x 8192: 88 us; three 89).
template <int FMT, int D, bool HI, int NT> cudaError_t go(const Launch& l) {
    constexpr int minb = D > 128 || NT == 2 ? 2 : D == 64 ? 4 : 3;
    if constexpr (NT == 1) {
        if (l.p.pack) return go_with<D, HI, 1, minb, true>(l);
    }
    return go_with<D, HI, NT, minb, false>(l);
}
#else
template <int FMT, int D, bool HI, int NT, int STAGES, int MINB> cudaError_t go_with(const Launch& l) {
    static std::atomic<int> fits[kDevices];
    return launch_kernel(l, k_attn<FMT, D, HI, NT, STAGES, MINB>, Layout<FMT, D, NT, STAGES>::BYTES, fits);
}

// Depth of a warp's ring and blocks per SM, measured on 64 sequences of 8192
// tokens (GB/s over the measured copy bandwidth). f16 and bf16 fill the memory
// system with three stages and two blocks per SM (1.00; 0.96 with tiles of 32
// keys in two stages). q8_0 issues on 62 % of its cycles and waits on its own
// results the rest, so that it takes as many blocks as registers and shared
// memory hold: four with two stages (0.83 to 0.88 with f16 and 0.76 with fp32
// activations; three with three stages were 0.03 to 0.04 less), at dim 256 and
// with 16 heads two (dim 256: 0.82; 0.71 with three stages, where only one fits).
template <int FMT, int D, bool HI, int NT> cudaError_t go(const Launch& l) {
    if constexpr (FMT != QMM_KV_Q8_0) return go_with<FMT, D, HI, NT, 3, 2>(l);
    else if constexpr (D <= 128 && NT == 1) return go_with<FMT, D, HI, NT, 2, 4>(l);
    else return go_with<FMT, D, HI, NT, 2, 2>(l);
}
#endif

template <int FMT, int D> cudaError_t pick(const Launch& l, bool hi, int tiles) {
    if constexpr (D <= 128) {
        if (tiles == 2) return hi ? go<FMT, D, true, 2>(l) : go<FMT, D, false, 2>(l);
    }
    return hi ? go<FMT, D, true, 1>(l) : go<FMT, D, false, 1>(l);
}

template <int FMT> cudaError_t launch_fmt(const Launch& l, int D, bool hi, int tiles) {
    switch (D) {
    case 64: return pick<FMT, 64>(l, hi, tiles);
    case 96: return pick<FMT, 96>(l, hi, tiles);
    case 128: return pick<FMT, 128>(l, hi, tiles);
    case 192: return pick<FMT, 192>(l, hi, tiles);
    default: return pick<FMT, 256>(l, hi, tiles);
    }
}

template cudaError_t launch_fmt<QMM_ATTN_FMT>(const Launch&, int, bool, int);

}  // namespace attn
}  // namespace qmm
