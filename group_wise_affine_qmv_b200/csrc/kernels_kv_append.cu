// kernels_kv_append.cu -- new keys and values into the 4-bit paged cache.
//
// Per token, head and group of G elements, in IEEE fp32: scale = (max - min) R, R the fp32 number next to
// 1/15, bias = min, q = rint((w - bias) / scale); scale and bias are stored rounded to the 16-bit type.
// The optional outputs are fma(scale, q, bias) of the stored scale and bias, rounded once.  The quantizer
// of kernels_quant.cu divides by 15 instead: its stored scales are the same but where the last bit of an fp32
// number decides a rounding to 16, its codes but where w lies halfway between two and that bit decides.
//
// Every byte moves once and nothing goes through shared memory; what then counts is instructions (8191
// tokens, 8 heads of 128, f16, with the outputs: issue slots 74% busy, 16.1 us, 4.8 TB/s where memory alone would
// take 11.8 us).  So
//  - a thread owns sixteen elements, two words of codes, and walks tokens (eight elements: 25.9 us: the set-up and
//    the slot's addresses were half of all instructions); the next token is fetched while one is at work;
//  - a group's maximum and minimum are packed maxima of the 16-bit pairs, exact, and of (max, -min) as one pair in
//    the shuffles among its lanes;
//  - the quotients come from the correctly rounded reciprocal r of the scale (one per group) as
//        q0 = t r,  q = q0 + (t - q0 scale) r      (both steps fused)
//    which Markstein ("Computation of elementary functions on the IBM RISC System/6000", 1990) proves to be the
//    correctly rounded t / scale as long as nothing under- or overflows; scales outside [2^-96, 2^96] take the
//    division itself (eight IEEE divisions by one divisor took most of the time);
//  - codes are packed as they stand in the low bits of 2^23 + 2^22 + q.
#include <cuda_runtime.h>

#include "device_common.cuh"
#include "kv_cache.h"
#include "sm100_ptx.cuh"

namespace aq {
namespace kv {
namespace {

constexpr int THREADS = 256;
constexpr int PIECE = 16;              // elements of a thread

// two 16-bit values, rounded to nearest even
__device__ __forceinline__ uint32_t pack_pair(float x, float y, bf16_t) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_pair(float x, float y, f16_t) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// the largest and the negated smallest of two pairs each, as a pair
__device__ __forceinline__ uint32_t max_pair(uint32_t x, uint32_t y, bf16_t) {
    const __nv_bfloat162 v = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t max_pair(uint32_t x, uint32_t y, f16_t) {
    const __half2 v = __hmax2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// A thread keeps one piece (head and sixteen elements) and walks the block's tokens, so the index
// arithmetic is done once: `side_by_side` tokens at a time, blockIdx.z * pieces the block's first piece.
template <typename XT>
__global__ void __launch_bounds__(THREADS) append_kernel(const __grid_constant__ AppendArgs a, int pieces, int side_by_side,
                                                         int tokens_per_block) {
    const int side = blockIdx.y;
    const Side& c = a.side[side];
    const int per_head = a.D / PIECE;
    const int glanes = (1 << a.log2g) / PIECE;     // lanes of a group: 2, 4 or 8
    const int tl = (int)threadIdx.x / pieces;      // which of the tokens side by side
    const int piece = blockIdx.z * pieces + (int)threadIdx.x - tl * pieces;
    // a whole group of lanes is live or not: pieces and H * D / 16 are multiples of G / 16
    const bool live = tl < side_by_side && piece < a.H * per_head;
    const int h = piece / per_head;
    const int dp = piece - h * per_head;
    const int g = (dp * PIECE) >> a.log2g;
    const bool lead = (dp & (glanes - 1)) == 0;    // stores the group's scale and bias
    const uint16_t* xh = a.x[side] + h * a.x_head[side] + dp * PIECE;
    uint16_t* oh = a.out[side] ? a.out[side] + h * a.o_head[side] + dp * PIECE : nullptr;
    uint32_t* wh = c.wq + h * c.w_head + dp * (PIECE / 8);
    uint16_t* sh = c.scales + h * c.s_head + g;
    uint16_t* bh = c.biases + h * c.b_head + g;
    const int64_t t0 = (int64_t)blockIdx.x * tokens_per_block;
    const int64_t t1 = t0 + tokens_per_block < a.T ? t0 + tokens_per_block : a.T;
    ptx::pdl_wait();   // k, v and slots may come from the kernel before; the cache may still be read by it
    ptx::pdl_launch_dependents();
    // the token after the one at work is on its way
    constexpr int PAIRS = PIECE / 2;
    uint32_t ahead[PAIRS];
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) ahead[j] = 0;
    int64_t slot_ahead = -1;
    auto fetch = [&](int64_t t) {
        if (!live || t >= t1) return;
        const uint16_t* xp = xh + t * a.x_tok[side];
        if (a.xvec[side]) {
#pragma unroll
            for (int j = 0; j < PAIRS; j += 4) {
                const uint4 u = __ldcg(reinterpret_cast<const uint4*>(xp + 2 * j));
                ahead[j] = u.x; ahead[j + 1] = u.y; ahead[j + 2] = u.z; ahead[j + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) ahead[j] = (uint32_t)__ldcg(xp + 2 * j) | ((uint32_t)__ldcg(xp + 2 * j + 1) << 16);
        }
        slot_ahead = __ldcg(a.slots + t);
    };
    fetch(t0 + tl);
    for (int64_t tb = t0; tb < t1; tb += side_by_side) {   // block-uniform: every lane takes part in the shuffles
        const int64_t t = tb + tl;
        const bool on = live && t < t1;
        uint32_t u[PAIRS];
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) u[j] = ahead[j];
        const int64_t slot = slot_ahead;
        fetch(t + side_by_side);
        // (max, -min) as one pair of the inputs' type, exact: one maximum and one shuffle a step
        constexpr uint32_t SIGNS = 0x80008000u;
        uint32_t hi = u[0], lo = u[0] ^ SIGNS;
#pragma unroll
        for (int j = 1; j < PAIRS; ++j) {
            hi = max_pair(hi, u[j], XT{});
            lo = max_pair(lo, u[j] ^ SIGNS, XT{});
        }
        uint32_t m = max_pair(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632), XT{});
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
            if (o < glanes) m = max_pair(m, __shfl_xor_sync(0xffffffffu, m, o), XT{});
        const float mx = half_bits_to_float((uint16_t)m, XT{}), mn = -half_bits_to_float((uint16_t)(m >> 16), XT{});
        const float scale = __fmul_rn(__fsub_rn(mx, mn), 1.0f / 15.0f);
        // codes as 2^23 + 2^22 + q: that sum rounds to nearest, ties to even
        constexpr float MAGIC = 12582912.0f;
        float q[PIECE];
        if (scale >= 0x1p-96f && scale <= 0x1p96f) {
            const float rcp = __frcp_rn(scale);
#pragma unroll
            for (int j = 0; j < PIECE; ++j) {
                const float t_ = __fsub_rn(half_bits_to_float((uint16_t)(u[j >> 1] >> (16 * (j & 1))), XT{}), mn);
                const float q0 = __fmul_rn(t_, rcp);
                q[j] = __fadd_rn(__fmaf_rn(__fmaf_rn(-q0, scale, t_), rcp, q0), MAGIC);
            }
        } else {
#pragma unroll
            for (int j = 0; j < PIECE; ++j) {
                const float t_ = __fsub_rn(half_bits_to_float((uint16_t)(u[j >> 1] >> (16 * (j & 1))), XT{}), mn);
                q[j] = MAGIC + (scale != 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(t_, scale)), 0.0f), 15.0f) : 0.0f);
            }
        }
        if (!on) continue;
        // their bits end in the code: a word is the sum of the eight shifted, less what the rest of the bits adds
        uint32_t word[PIECE / 8];
#pragma unroll
        for (int w = 0; w < PIECE / 8; ++w) {
            constexpr uint32_t REST = 0x4B400000u * 0x11111111u;
            word[w] = 0u - REST;
#pragma unroll
            for (int j = 0; j < 8; ++j) word[w] += __float_as_uint(q[8 * w + j]) << (4 * j);
        }
        const uint32_t sb = pack_pair(scale, mn, XT{});
        if (slot >= 0 && slot < a.nslots) {
            // 64-bit division only where a slot's index needs it
            const int64_t pg = a.nslots <= 0xffffffffll ? (int64_t)((uint32_t)slot / (uint32_t)a.S) : slot / a.S;
            const int64_t sl = slot - pg * a.S;
            *reinterpret_cast<uint2*>(wh + pg * c.w_page + sl * c.w_slot) = make_uint2(word[0], word[1]);
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
            uint32_t w[PAIRS];
#pragma unroll
            for (int j = 0; j < PAIRS; ++j)
                w[j] = pack_pair(fmaf(s, q[2 * j] - MAGIC, b), fmaf(s, q[2 * j + 1] - MAGIC, b), XT{});
            if (a.ovec[side]) {
#pragma unroll
                for (int j = 0; j < PAIRS; j += 4) *reinterpret_cast<uint4*>(op + 2 * j) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < PAIRS; ++j) {
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
    // one token has more than a block's threads); it walks up to eight such rows of tokens, so that its set-up is
    // paid once and one wave of blocks does (16.1 us; twice the blocks and half the walk 16.6, half the blocks 17.4)
    constexpr int PER_SIDE = 148 * 4 / 2;    // four blocks fit an SM
    const int per_tok = a.H * (a.D / PIECE);
    const int pieces = per_tok < THREADS ? per_tok : THREADS;
    const int sbs = THREADS / pieces;
    int64_t rows = (a.T + sbs - 1) / sbs, walk = (rows + PER_SIDE - 1) / PER_SIDE;
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
