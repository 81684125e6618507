// kernels_moe_b2_bf16.cu -- mixture-of-experts kernels for 2-bit codes with bf16 activations
// (moe_kernel.cuh; one file per instantiation set so that they compile in parallel).
#include "moe_kernel.cuh"

namespace aq {
namespace moe {

template <>
cudaError_t launch_b<2, true>(const Args& a, int group, cudaStream_t s) {
    return launch_g<2, bf16_t>(a, group, s);
}

}  // namespace moe
}  // namespace aq
