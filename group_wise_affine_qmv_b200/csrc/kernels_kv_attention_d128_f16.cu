// kernels_kv_attention_d128_f16.cu -- head size 128 with f16 queries, scales and biases (kernels in
// kv_attention_kernel.cuh; one file per instantiation set so that they compile in parallel).
#include "kv_attention_kernel.cuh"

namespace aq {
namespace kv {

template <>
cudaError_t launch_d<128, false>(const AttnArgs& a, const AttnShape& s, int group, cudaStream_t st) {
    return launch_g<128, f16_t>(a, s, group, st);
}

}  // namespace kv
}  // namespace aq
