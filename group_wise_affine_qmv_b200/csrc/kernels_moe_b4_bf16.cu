// kernels_moe_b4_bf16.cu -- mixture-of-experts kernels for 4-bit codes with bf16 activations
// (moe_kernel.cuh; one file per instantiation set so that they compile in parallel).
#include "moe_kernel.cuh"

namespace aq {
namespace moe {

template <>
cudaError_t launch_b<4, true>(const Args& a, int group, cudaStream_t s) {
    return launch_g<4, bf16_t>(a, group, s);
}

}  // namespace moe
}  // namespace aq
