// kernels_moe_b8_f16.cu -- mixture-of-experts kernels for 8-bit codes with f16 activations
// (moe_kernel.cuh; one file per instantiation set so that they compile in parallel).
#include "moe_kernel.cuh"

namespace aq {
namespace moe {

template <>
cudaError_t launch_b<8, false>(const Args& a, int group, cudaStream_t s) {
    return launch_g<8, f16_t>(a, group, s);
}

}  // namespace moe
}  // namespace aq
