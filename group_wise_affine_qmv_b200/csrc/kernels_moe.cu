// kernels_moe.cu -- launch shape of the mixture-of-experts layer, and the choice of its instantiation.
#include "moe.h"

namespace aq {
namespace moe {

extern template cudaError_t launch_b<2, true>(const Args&, int, cudaStream_t);
extern template cudaError_t launch_b<2, false>(const Args&, int, cudaStream_t);
extern template cudaError_t launch_b<4, true>(const Args&, int, cudaStream_t);
extern template cudaError_t launch_b<4, false>(const Args&, int, cudaStream_t);
extern template cudaError_t launch_b<8, true>(const Args&, int, cudaStream_t);
extern template cudaError_t launch_b<8, false>(const Args&, int, cudaStream_t);

cudaError_t launch(Args& a, int bits, int group, bool bf16, cudaStream_t s) {
    // the down kernel's CTAs per block of 32 columns: enough for about three CTAs per SM, no more than
    // there can be entries
    const int blocks = (a.K + 31) / 32;
    a.cs = 1;
    while (a.cs < 8 && blocks * a.cs * 2 <= 148 * 4 && a.cs * 2 <= a.T * a.topk && a.cs * 2 <= a.E) a.cs *= 2;
    switch (bits) {
        case 2: return bf16 ? launch_b<2, true>(a, group, s) : launch_b<2, false>(a, group, s);
        case 4: return bf16 ? launch_b<4, true>(a, group, s) : launch_b<4, false>(a, group, s);
        case 8: return bf16 ? launch_b<8, true>(a, group, s) : launch_b<8, false>(a, group, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
}  // namespace aq
