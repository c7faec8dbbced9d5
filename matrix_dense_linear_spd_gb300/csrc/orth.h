// Launches of the orthogonalisation's products, compiled in a translation unit for each number of planes.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace bl {
namespace orth {

struct Args;

// How a product reads its operands (see orth_gemm.cuh).
enum Layout : int { GRAM_LINES = 0, GRAM_WIDTH = 1, SQUARE_A = 2, APPLY_LEFT = 3, APPLY_RIGHT = 4 };

cudaError_t launch_one(Layout layout, int ctas, const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &md, const CUtensorMap &mo,
                       const Args &a, int sms, cudaStream_t s);
cudaError_t launch_two(Layout layout, int ctas, const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &md, const CUtensorMap &mo,
                       const Args &a, int sms, cudaStream_t s);

// Small matrices, in one launch; needs no workspace.
bool fits_small(int64_t lines, int64_t width);
cudaError_t launch_small(int dtype, int64_t lines, int64_t width, int64_t batch, const void *g, int64_t ldg, int64_t stride_g, void *x,
                         int64_t ldx, int64_t stride_x, int steps, const double *coefficients, int sms, cudaStream_t s);

}  // namespace orth
}  // namespace bl
