// kernels_moe.cu -- the choice of the mixture-of-experts layer's instantiation.
#include "moe.h"

namespace aq {
namespace moe {

extern template cudaError_t launch_b<2, true>(const Args&, int, cudaStream_t);
extern template cudaError_t launch_b<2, false>(const Args&, int, cudaStream_t);
extern template cudaError_t launch_b<4, true>(const Args&, int, cudaStream_t);
extern template cudaError_t launch_b<4, false>(const Args&, int, cudaStream_t);
extern template cudaError_t launch_b<8, true>(const Args&, int, cudaStream_t);
extern template cudaError_t launch_b<8, false>(const Args&, int, cudaStream_t);

cudaError_t launch(const Args& a, int bits, int group, bool bf16, cudaStream_t s) {
    switch (bits) {
        case 2: return bf16 ? launch_b<2, true>(a, group, s) : launch_b<2, false>(a, group, s);
        case 4: return bf16 ? launch_b<4, true>(a, group, s) : launch_b<4, false>(a, group, s);
        case 8: return bf16 ? launch_b<8, true>(a, group, s) : launch_b<8, false>(a, group, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
}  // namespace aq
