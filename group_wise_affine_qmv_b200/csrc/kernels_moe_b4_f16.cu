// kernels_moe_b4_f16.cu -- mixture-of-experts kernels for 4-bit codes with f16 activations
// (moe_kernel.cuh; one file per instantiation set so that they compile in parallel).
#include "moe_kernel.cuh"

namespace aq {
namespace moe {

template <>
cudaError_t launch_b<4, false>(const Args& a, int group, cudaStream_t s) {
    return launch_g<4, f16_t>(a, group, s);
}

}  // namespace moe
}  // namespace aq
