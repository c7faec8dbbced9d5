// The orthogonalisation's products of one plane of f16.
#include "orth_launch.cuh"

namespace bl {
namespace orth {

cudaError_t launch_one(Layout layout, int ctas, const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &md, const CUtensorMap &mo,
                       const Args &a, int sms, cudaStream_t s) {
    return launch<1>(layout, ctas, ma, mb, md, mo, a, sms, s);
}

}  // namespace orth
}  // namespace bl
