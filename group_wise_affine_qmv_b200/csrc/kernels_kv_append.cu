// kernels_kv_append.cu -- new keys and values into the 4-bit paged cache.
//
// Per token, head and group of G elements, the quantizer of kernels_quant.cu bit for bit, in IEEE
// fp32: scale = (max - min) / 15, bias = min, q = clamp(rint((w - bias) / scale), 0, 15); scale and
// bias are stored rounded to the 16-bit type.  The optional outputs are fma(scale, q, bias) of the
// stored scale and bias, rounded once.
//
// Bound by memory: a thread owns eight elements, which are one 16-byte load, one 32-bit word of
// codes and one 16-byte store, and a group's minimum and maximum are shuffles among its G/8 lanes,
// so every byte moves once and nothing goes through shared memory.
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "kv_cache.h"
#include "sm100_ptx.cuh"

namespace aq {
namespace kv {
namespace {

constexpr int THREADS = 256;

template <typename XT>
__global__ void __launch_bounds__(THREADS) append_kernel(const __grid_constant__ AppendArgs a, int tokens_per_block) {
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();   // k, v and slots may come from the kernel before; the cache may still be read by it
    const int side = blockIdx.y;
    const Side& c = a.side[side];
    const int per_head = a.D >> 3;                 // 8-element pieces
    const int per_tok = a.H * per_head;
    const int glanes = 1 << (a.log2g - 3);         // lanes of a group: 4, 8 or 16
    const int64_t t0 = (int64_t)blockIdx.x * tokens_per_block;
    const int64_t t1 = t0 + tokens_per_block < a.T ? t0 + tokens_per_block : a.T;
    const int total = (int)(t1 - t0) * per_tok;
    for (int i0 = 0; i0 < total; i0 += THREADS) {   // block-uniform: every lane takes part in the shuffles
        int i = i0 + (int)threadIdx.x;
        const bool live = i < total;                // a whole group is live or not: total is a multiple of G/8
        if (!live) i = total - 1;
        const int tl = i / per_tok;
        const int rem = i - tl * per_tok;
        const int h = rem / per_head;
        const int d8 = rem - h * per_head;
        const int64_t t = t0 + tl;
        const uint16_t* xp = a.x[side] + t * a.x_tok[side] + h * a.x_head[side] + d8 * 8;
        uint4 u;
        if (a.xvec[side]) {
            u = __ldcg(reinterpret_cast<const uint4*>(xp));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = (uint32_t)__ldcg(xp + 2 * j) | ((uint32_t)__ldcg(xp + 2 * j + 1) << 16);
            u = make_uint4(w[0], w[1], w[2], w[3]);
        }
        const int64_t slot = __ldcg(a.slots + t);
        float v[8];
        unpack8(u, v, XT{});
        float mn = v[0], mx = v[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) {
            mn = fminf(mn, v[j]);
            mx = fmaxf(mx, v[j]);
        }
        for (int o = glanes >> 1; o > 0; o >>= 1) {
            mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        const float scale = __fdiv_rn(__fsub_rn(mx, mn), 15.0f);
        float q[8];
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            q[j] = 0.0f;
            if (scale != 0.0f) q[j] = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(v[j], mn), scale)), 0.0f), 15.0f);
            word |= (uint32_t)q[j] << (4 * j);
        }
        if (!live) continue;
        const uint16_t sh = float_to_half_bits(scale, XT{}), bh = float_to_half_bits(mn, XT{});
        if (slot >= 0 && slot < a.nslots) {
            const int64_t pg = slot / a.S;
            const int64_t sl = slot - pg * a.S;
            c.wq[pg * c.w_page + h * c.w_head + sl * c.w_slot + d8] = word;
            if ((d8 & (glanes - 1)) == 0) {
                const int g = (d8 * 8) >> a.log2g;
                c.scales[pg * c.s_page + h * c.s_head + sl * c.s_slot + g] = sh;
                c.biases[pg * c.b_page + h * c.b_head + sl * c.b_slot + g] = bh;
            }
        } else if (slot >= a.nslots && rem == 0) {
            atomicOr(a.err, DEVERR_INDEX);
        }
        if (a.out[side]) {
            const float s = half_bits_to_float(sh, XT{}), b = half_bits_to_float(bh, XT{});
            uint16_t* op = a.out[side] + t * a.o_tok[side] + h * a.o_head[side] + d8 * 8;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = (uint32_t)float_to_half_bits(fmaf(s, q[2 * j], b), XT{}) |
                       ((uint32_t)float_to_half_bits(fmaf(s, q[2 * j + 1], b), XT{}) << 16);
            if (a.ovec[side]) {
                *reinterpret_cast<uint4*>(op) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    op[2 * j] = (uint16_t)w[j];
                    op[2 * j + 1] = (uint16_t)(w[j] >> 16);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, bool bf16, cudaStream_t s) {
    // a block takes whole tokens, about one pass of its threads; more where the tokens are many
    const int64_t per_tok = (int64_t)a.H * (a.D / 8);
    int64_t tpb = (THREADS + per_tok - 1) / per_tok;
    if (tpb * per_tok > THREADS && tpb > 1) tpb = THREADS / per_tok;
    while ((a.T + tpb - 1) / tpb > 0x7fffffff) tpb *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.T + tpb - 1) / tpb), 2);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return bf16 ? cudaLaunchKernelEx(&cfg, append_kernel<bf16_t>, a, (int)tpb)
                : cudaLaunchKernelEx(&cfg, append_kernel<f16_t>, a, (int)tpb);
}

}  // namespace kv
}  // namespace aq
