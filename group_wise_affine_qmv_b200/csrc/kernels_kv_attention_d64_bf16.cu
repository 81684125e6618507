// kernels_kv_attention_d64_bf16.cu -- head size 64 with bf16 queries, scales and biases (kernels in
// kv_attention_kernel.cuh; one file per instantiation set so that they compile in parallel).
#include "kv_attention_kernel.cuh"

namespace aq {
namespace kv {

template <>
cudaError_t launch_d<64, true>(const AttnArgs& a, const AttnShape& s, int group, cudaStream_t st) {
    return launch_g<64, bf16_t>(a, s, group, st);
}

}  // namespace kv
}  // namespace aq
