// What the translation units of the orthogonalisation's products share.
#pragma once

#include <algorithm>
#include <atomic>

#include "orth.h"
#include "orth_gemm.cuh"

namespace bl {
namespace orth {

template <int KIND, bool A_MN, bool B_MN, int PLANES, int CTAS>
cudaError_t launch_tiles(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &md, const CUtensorMap &mo, const Args &a,
                         int sms, cudaStream_t s) {
    constexpr int kSmem = Ring<PLANES, CTAS>::kSmem;
    const auto kernel = product_kernel<KIND, A_MN, B_MN, PLANES, CTAS>;
    static std::atomic<int> groups[64];         // CTAs, or pairs of CTAs, that the device runs at once
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int most = dev < 64 ? groups[dev].load(std::memory_order_acquire) : 0;
    if (most == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        most = sms;
        if constexpr (CTAS > 1) {
            cudaLaunchConfig_t c{};
            c.gridDim = dim3(sms / CTAS * CTAS);
            c.blockDim = dim3(kThreads);
            c.dynamicSmemBytes = kSmem;
            cudaLaunchAttribute at{};
            at.id = cudaLaunchAttributeClusterDimension;
            at.val.clusterDim.x = CTAS;
            at.val.clusterDim.y = at.val.clusterDim.z = 1;
            c.attrs = &at;
            c.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&most, kernel, &c);
            if (e != cudaSuccess) return e;
            most = std::max(1, std::min(most, sms / CTAS));
        }
        if (dev < 64) groups[dev].store(most, std::memory_order_release);
    }
    return launch_pdl_cluster(kernel, std::min(a.total, most) * CTAS, kThreads, kSmem, CTAS, s, ma, mb, md, mo, a);
}

template <int PLANES>
cudaError_t launch(Layout layout, int ctas, const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &md,
                   const CUtensorMap &mo, const Args &a, int sms, cudaStream_t s) {
    switch (layout) {
        case GRAM_LINES:
            return ctas == 1 ? launch_tiles<GRAM, false, false, PLANES, 1>(ma, mb, md, mo, a, sms, s)
                             : launch_tiles<GRAM, false, false, PLANES, 2>(ma, mb, md, mo, a, sms, s);
        case GRAM_WIDTH:
            return ctas == 1 ? launch_tiles<GRAM, true, true, PLANES, 1>(ma, mb, md, mo, a, sms, s)
                             : launch_tiles<GRAM, true, true, PLANES, 2>(ma, mb, md, mo, a, sms, s);
        case SQUARE_A:
            return ctas == 1 ? launch_tiles<SQUARE, false, false, PLANES, 1>(ma, mb, md, mo, a, sms, s)
                             : launch_tiles<SQUARE, false, false, PLANES, 2>(ma, mb, md, mo, a, sms, s);
        case APPLY_LEFT:
            return ctas == 1 ? launch_tiles<APPLY, false, true, PLANES, 1>(ma, mb, md, mo, a, sms, s)
                             : launch_tiles<APPLY, false, true, PLANES, 2>(ma, mb, md, mo, a, sms, s);
        default:
            return ctas == 1 ? launch_tiles<APPLY, false, false, PLANES, 1>(ma, mb, md, mo, a, sms, s)
                             : launch_tiles<APPLY, false, false, PLANES, 2>(ma, mb, md, mo, a, sms, s);
    }
}

}  // namespace orth
}  // namespace bl
