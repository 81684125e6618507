// kernels_kv_append.cu -- new keys and values into the 4-bit paged cache.
//
// Per token, head and group of G elements, in IEEE fp32: scale = (max - min) R, R the fp32 number next to
// 1/15, bias = min, q = rint((w - bias) / scale); scale and bias are stored rounded to the 16-bit type.
// The optional outputs are fma(scale, q, bias) of the stored scale and bias, rounded once.  The quantizer
// of kernels_quant.cu divides by 15 instead: its stored scales are the same but where the last bit of an fp32
// number decides a rounding to 16, its codes but where w lies halfway between two and that bit decides.
//
// Bound by memory: a thread owns eight elements, which are one 16-byte load, one 32-bit word of
// codes and one 16-byte store, and a group's minimum and maximum are shuffles among its G/8 lanes,
// so every byte moves once and nothing goes through shared memory.  What then counts is
// instructions: eight IEEE divisions a thread by one divisor took most of the time, so the quotient
// is formed from the correctly rounded reciprocal r of the scale (one per group) as
//     q0 = t r,  q = q0 + (t - q0 scale) r      (both steps fused)
// which Markstein ("Computation of elementary functions on the IBM RISC System/6000", 1990) proves
// to be the correctly rounded t / scale as long as nothing under- or overflows; scales outside
// [2^-96, 2^96] take the division itself.
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "kv_cache.h"
#include "sm100_ptx.cuh"

namespace aq {
namespace kv {
namespace {

constexpr int THREADS = 256;

// two 16-bit values, rounded to nearest even
__device__ __forceinline__ uint32_t pack_pair(float x, float y, bf16_t) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_pair(float x, float y, f16_t) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// A thread keeps one piece (head and eight elements) and walks the block's tokens, so the index
// arithmetic is done once: `side_by_side` tokens at a time, `piece0` the block's first piece.
template <typename XT>
__global__ void __launch_bounds__(THREADS) append_kernel(const __grid_constant__ AppendArgs a, int pieces, int side_by_side,
                                                         int tokens_per_block) {
    const int side = blockIdx.y;
    const Side& c = a.side[side];
    const int per_head = a.D >> 3;                 // 8-element pieces
    const int glanes = 1 << (a.log2g - 3);         // lanes of a group: 4, 8 or 16
    const int tl = (int)threadIdx.x / pieces;      // which of the tokens side by side
    const int piece = blockIdx.z * pieces + (int)threadIdx.x - tl * pieces;
    // a whole group of lanes is live or not: pieces and H * D / 8 are multiples of G / 8
    const bool live = tl < side_by_side && piece < a.H * per_head;
    const int h = piece / per_head;
    const int d8 = piece - h * per_head;
    const int g = (d8 * 8) >> a.log2g;
    const bool lead = (d8 & (glanes - 1)) == 0;    // stores the group's scale and bias
    const uint16_t* xh = a.x[side] + h * a.x_head[side] + d8 * 8;
    uint16_t* oh = a.out[side] ? a.out[side] + h * a.o_head[side] + d8 * 8 : nullptr;
    uint32_t* wh = c.wq + h * c.w_head + d8;
    uint16_t* sh = c.scales + h * c.s_head + g;
    uint16_t* bh = c.biases + h * c.b_head + g;
    const int64_t t0 = (int64_t)blockIdx.x * tokens_per_block;
    const int64_t t1 = t0 + tokens_per_block < a.T ? t0 + tokens_per_block : a.T;
    ptx::pdl_wait();   // k, v and slots may come from the kernel before; the cache may still be read by it
    ptx::pdl_launch_dependents();
    for (int64_t tb = t0; tb < t1; tb += side_by_side) {   // block-uniform: every lane takes part in the shuffles
        const int64_t t = tb + tl;
        const bool on = live && t < t1;
        uint4 u = make_uint4(0, 0, 0, 0);
        int64_t slot = -1;
        if (on) {
            const uint16_t* xp = xh + t * a.x_tok[side];
            if (a.xvec[side]) {
                u = __ldcg(reinterpret_cast<const uint4*>(xp));
            } else {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = (uint32_t)__ldcg(xp + 2 * j) | ((uint32_t)__ldcg(xp + 2 * j + 1) << 16);
                u = make_uint4(w[0], w[1], w[2], w[3]);
            }
            slot = __ldcg(a.slots + t);
        }
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
        const float scale = __fmul_rn(__fsub_rn(mx, mn), 1.0f / 15.0f);
        // codes as small whole floats; the sums 2^23 + 2^22 + q round to nearest, ties to even
        constexpr float MAGIC = 12582912.0f;
        float q[8];
        if (scale >= 0x1p-96f && scale <= 0x1p96f) {
            const float rcp = __frcp_rn(scale);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = __fsub_rn(v[j], mn);
                const float q0 = __fmul_rn(t, rcp);
                q[j] = __fsub_rn(__fadd_rn(__fmaf_rn(__fmaf_rn(-q0, scale, t), rcp, q0), MAGIC), MAGIC);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                q[j] = scale != 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(v[j], mn), scale)), 0.0f), 15.0f) : 0.0f;
        }
        // four codes are one whole number below 2^16
        uint32_t half[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            half[j] = __float_as_uint(fmaf(fmaf(q[4 * j + 3], 16.0f, q[4 * j + 2]), 256.0f, fmaf(q[4 * j + 1], 16.0f, q[4 * j])) + 8388608.0f);
        const uint32_t word = __byte_perm(half[0], half[1], 0x5410);
        if (!on) continue;
        const uint32_t sb = pack_pair(scale, mn, XT{});
        if (slot >= 0 && slot < a.nslots) {
            // 64-bit division only where a slot's index needs it
            const int64_t pg = a.nslots <= 0xffffffffll ? (int64_t)((uint32_t)slot / (uint32_t)a.S) : slot / a.S;
            const int64_t sl = slot - pg * a.S;
            wh[pg * c.w_page + sl * c.w_slot] = word;
            if (lead) {
                sh[pg * c.s_page + sl * c.s_slot] = (uint16_t)sb;
                bh[pg * c.b_page + sl * c.b_slot] = (uint16_t)(sb >> 16);
            }
        } else if (slot >= a.nslots && piece == 0) {
            atomicOr(a.err, DEVERR_INDEX);
        }
        if (oh) {
            const float s = half_bits_to_float((uint16_t)sb, XT{}), b = half_bits_to_float((uint16_t)(sb >> 16), XT{});
            uint16_t* op = oh + t * a.o_tok[side];
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack_pair(fmaf(s, q[2 * j], b), fmaf(s, q[2 * j + 1], b), XT{});
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
    // a block's threads are the pieces of a few tokens side by side (blockIdx.z: blocks of pieces where
    // one token has more than a block's threads); it walks up to eight such rows of tokens when there
    // are many, so that its set-up is paid once
    const int per_tok = a.H * (a.D / 8);
    const int pieces = per_tok < THREADS ? per_tok : THREADS;
    const int sbs = THREADS / pieces;
    int64_t rows = (a.T + sbs - 1) / sbs, walk = rows / (148 * 8);
    walk = walk < 1 ? 1 : walk > 8 ? 8 : walk;
    while ((rows + walk - 1) / walk > 0x7fffffff) walk *= 2;
    const int64_t tpb = walk * sbs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.T + tpb - 1) / tpb), 2, (unsigned)((per_tok + pieces - 1) / pieces));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return bf16 ? cudaLaunchKernelEx(&cfg, append_kernel<bf16_t>, a, pieces, sbs, (int)tpb)
                : cudaLaunchKernelEx(&cfg, append_kernel<f16_t>, a, pieces, sbs, (int)tpb);
}

}  // namespace kv
}  // namespace aq
