// The orthogonalisation's products of two planes of f16.
#include "orth_launch.cuh"

namespace bl {
namespace orth {

cudaError_t launch_two(Layout layout, int ctas, const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &md, const CUtensorMap &mo,
                       const Args &a, int sms, cudaStream_t s) {
    return launch<2>(layout, ctas, ma, mb, md, mo, a, sms, s);
}

}  // namespace orth
}  // namespace bl
