// kernels_kv_attention.cu -- launch shape of the attention over a 4-bit cache, and the choice of its
// instantiation.
#include "kv_cache.h"

namespace aq {
namespace kv {

template <int D, bool BF>
cudaError_t launch_d(const AttnArgs& a, const AttnShape& s, int group, cudaStream_t st);
extern template cudaError_t launch_d<64, true>(const AttnArgs&, const AttnShape&, int, cudaStream_t);
extern template cudaError_t launch_d<64, false>(const AttnArgs&, const AttnShape&, int, cudaStream_t);
extern template cudaError_t launch_d<128, true>(const AttnArgs&, const AttnShape&, int, cudaStream_t);
extern template cudaError_t launch_d<128, false>(const AttnArgs&, const AttnShape&, int, cudaStream_t);
extern template cudaError_t launch_d<256, true>(const AttnArgs&, const AttnShape&, int, cudaStream_t);
extern template cudaError_t launch_d<256, false>(const AttnArgs&, const AttnShape&, int, cudaStream_t);

namespace {
constexpr int SMS = 148;
}  // namespace

AttnShape attn_shape(int64_t B, int64_t rows, int64_t Hkv, int D, int64_t max_tokens) {
    AttnShape s;
    s.nt = rows <= 8 ? 1 : (rows <= 16 || D == 256) ? 2 : 4;
    s.rtiles = (int)((rows + 8 * s.nt - 1) / (8 * s.nt));
    const int64_t items = B * Hkv * s.rtiles;
    // CTAs that fit the device at once (the kernel's launch bounds)
    const int64_t all = (int64_t)SMS * ctas_per_sm(D, s.nt);
    const int64_t most = items * ((max_tokens + unit_tokens(D, s.nt) - 1) / unit_tokens(D, s.nt));
    // Short tables: an item per CTA, which spares the combine launch.  The rule goes by the table's width, which a
    // captured step fixes, not by the lengths.  Tables of 512 (this form) and 528 tokens (the other), 16 heads on 8 of 128,
    // bf16: one sequence of 128 tokens 5.4 and 6.7 us, of 512 9.2 and 7.3; 8 sequences of 300 8.3 and 9.4, of 512 9.7 and
    // 9.6; 32 of 300 12.3 and 16.0, of 512 16.0 and 18.0; one of 512, D 256 15.7 and 8.3.  Wider tables cost what 528 does, within 1 us.
    if (max_tokens <= 512 && items <= 0x7fffffff) {
        s.split = 0;
        s.grid = (int)(items < 1 ? 1 : items);
        s.o_floats = s.ml_floats = 0;
        return s;
    }
    s.split = 1;
    s.grid = (int)(most < all ? (most < 1 ? 1 : most) : all);
    s.o_floats = (size_t)2 * s.grid * 8 * s.nt * D;
    s.ml_floats = (size_t)2 * s.grid * 8 * s.nt * 2;
    return s;
}

cudaError_t launch_attention(const AttnArgs& a, const AttnShape& s, int D, int group, bool bf16, cudaStream_t st) {
    switch (D) {
        case 64: return bf16 ? launch_d<64, true>(a, s, group, st) : launch_d<64, false>(a, s, group, st);
        case 128: return bf16 ? launch_d<128, true>(a, s, group, st) : launch_d<128, false>(a, s, group, st);
        case 256: return bf16 ? launch_d<256, true>(a, s, group, st) : launch_d<256, false>(a, s, group, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace kv
}  // namespace aq
