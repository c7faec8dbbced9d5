// Tensor maps (what TMA is told of a matrix in memory), encoded by the driver.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace bl {

// Whether rows of `elem`-byte values, ld apart, start on the 16-byte boundaries that TMA wants.
inline bool for_tma(const void *p, int64_t ld, int64_t elem) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * elem % 16 == 0;
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess)
            return EncodeFn(nullptr);
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Planes of rows x inner values, copied in boxes of box_rows lines of line_bytes (128 or 64, the
// swizzle's width too); what lies outside reads as zero and is not written. Planes are `plane`
// values apart; with one plane any multiple of 16 bytes will do.
inline bool make_map(CUtensorMap *map, CUtensorMapDataType type, int elem, const void *base, int64_t inner, int64_t rows, int64_t planes,
              int64_t ld, int64_t plane, int box_rows, int line_bytes = 128) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(planes)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * elem), static_cast<cuuint64_t>(plane * elem)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(line_bytes / elem), static_cast<cuuint32_t>(box_rows), 1}, step[3] = {1, 1, 1};
    return fn(map, type, 3, const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              line_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace bl
