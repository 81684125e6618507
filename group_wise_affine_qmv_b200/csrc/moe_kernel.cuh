// moe_kernel.cuh -- a mixture-of-experts layer for a few tokens.
//
//     e_1 .. e_k = the top-k of logits[t], w = their softmax weights
//     h[t, j]    = w_j silu(x[t] . Wg[e_j]^T) * (x[t] . Wu[e_j]^T)
//     y[t]       = r[t] + sum_j h[t, j] . Wd[e_j]^T
//
// Three kernels, each a programmatic dependent of the one before: a small one for what depends on the
// tokens alone (routing, and x in the form the next kernel multiplies), gate/up, and down.  Every
// weight that some token chose is read once per 16 of its tokens; at a few dozen tokens that traffic is
// what counts, so the two large kernels are streams of packed codes that never pause, and what is left
// to care about is instructions per code:
//  - Codes go to the tensor cores (mma.sync.m16n8k16, 16 weight rows x 16 codes, 8 tokens) as f16
//    subnormals: a byte of a half, masked to one code, is already the f16 number code * 2^-24 (times 4 or
//    16 where the code sits higher in the byte).  A pair of 8-bit codes takes one PRMT, a pair of 4-bit
//    codes one AND and half a shift; the exact products and fp32 sums differ from those of the codes by
//    powers of two only.  x is scaled by a power of two per token into f16's range (exact for elements
//    down to 2^-24 of the token's largest, 2^-22 with 2-bit codes; smaller ones are off by at most 2^-33 of it), its elements permuted and scaled to meet their codes' positions.
//  - A group costs s D + b X, two FMAs per row and token; X, the sum over the group, comes from one more MMA
//    per k step whose codes are all one.  (Sums kept in memory by the kernel before and loaded per group took
//    a third of the down kernel's time: 460 against 390 us for 32 tokens and 128 experts.)
//  - A warp streams stages of 128 bytes x 32 weight rows through its own ring in shared memory with
//    16-byte asynchronous copies; the ring runs on across items, so the next item's codes are in flight
//    while one is finished.  Experts and token lists are fetched an item ahead.
//  - Scales and biases of an item's rows are one dense run each, which a bulk copy brings whole.  (Copied
//    stage by stage, 4 bytes a row, each 32-byte sector crosses from L2 eight times, as much traffic as the
//    codes: 128 experts of 8 bits, 8 tokens, 225 against 139 us without the arithmetic.)  Rows with too many
//    groups for that, and items that four warps share, copy them stage by stage.
//  - gate/up: an item is 16 gate rows and the same 16 up rows of one expert, for up to 16 tokens.  A warp
//    does an item alone, all of K, and ends with both sums of an activation in one lane.  Where there
//    are too few items to fill the device the four warps of a CTA share one, a quarter of the stages each.
//  - The activations pass on as f16 with a power of two per 16 of them (11 bits of mantissa where y has 8, two
//    such numbers where y is f16 or f32: parts_of), and the largest of a row's powers (an atomic maximum: order does not matter), on which the
//    down kernel puts them, by one multiplication a pair, to multiply subnormal codes again.
//  - x and the activations are read through L1: with few tokens all warps of the device walk the same lines, which
//    from L2 cost up to 1.5 us a stage (one token: 53 against 42 us).
//  - down: a CTA owns 32 columns of y for all tokens and walks the entries, its warps splitting N by
//    stages; a cluster of up to eight CTAs splits the entries and adds its tiles in rank order.  It stages
//    its first weights while the gate/up kernel still runs.  No atomics on results: nothing depends on
//    timing.
//
// Measured, device time of a layer: one token, 8 of 128 experts of 8 bits, 1408 x 2816: 40 us, 2.7 TB/s (the first kernel
// is 4 to 5 us of latency); 32 tokens, nearly the whole bank: 354 us, 4.2 TB/s; 64 tokens, 6 of 64 experts of 4 bits,
// 2048 x 1024: 116 us, 2.0 TB/s; the 128-expert bank in 2 bits, groups of 64: one token 47 us, 32 tokens 515 us, 0.8 TB/s.  The
// large kernels are bound by the latency of a stage (wait, shared memory, MMA, fold) at the 10 to 12 warps an SM that
// their registers allow: 37 to 43% of the issue slots, 20 to 59% of the DRAM peak.  Down kernels of activations in two parts spill
// (4 bits 150 to 180 bytes of stores a thread, 2 bits 320 to 360), and of one part with 2 bits, groups of 64 (150).
#pragma once

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "moe.h"
#include "warp_mma_kernel.cuh"

namespace aq {
namespace moe {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int ROWS = 32;               // weight rows of a stage
constexpr int RP = ROWS + 1;           // floats per token of a partial tile
constexpr int UP_GROUPS = 64;          // most groups of a row whose scales a warp of the gate/up kernel holds whole
constexpr int DOWN_GROUPS = 256;       // ... and a CTA of the down kernel, twice
constexpr uint64_t WAIT_NS = 2000000000ull;   // budget of a bounded wait

template <int BITS, int G>
struct Geo {
    static constexpr int SC = 512 / BITS;                 // codes of a row per half stage (64 bytes)
    static constexpr int KS = G < 64 ? G : 64;            // codes per sub-block: a lane holds KS / 4 in a row
    static constexpr int SUBS = SC / KS;
    static constexpr int STEPS = KS / 16;
    static constexpr int LB = KS * BITS / 32;             // bytes of a row per lane and sub-block
    static constexpr int FU = G < SC ? G : SC;            // codes per fold: a group, or a half stage's part of it
    static constexpr int SPF = FU / KS;
    static constexpr int GPS = SC / FU;                   // folds per half stage
    // A half stage in shared memory: codes, and where they come stage by stage the rows' scales and biases (the
    // 4 or 8 aligned bytes around its folds).
    static constexpr int SBB = GPS == 4 ? 8 : 4;
    static constexpr int CODES = ROWS * 64;
    static constexpr int half(bool blk) { return CODES + (blk ? 0 : 2 * ROWS * SBB); }
    // Stages of a warp's ring.  The down kernel's is short for a third CTA on an SM next to the tiles of y (32 tokens,
    // 128 experts of 8 bits: 428 us the layer with 3 stages, two CTAs, 393 with 2; where three fit anyway: alike).
    static constexpr int NST = 3, NST_DOWN = 2;
    static constexpr int ring(int stages, bool blk) { return WARPS * stages * 2 * half(blk); }
    static_assert(LB >= 4, "a lane's codes fill whole words");
};

// Where element j of 16 consecutive ones goes in the order of the expanded codes, and the power of two
// that its code carries: 8 bits in order; 4 bits (0,4) (1,5) (2,6) (3,7) of a word, odd ones 16 times;
// 2 bits (j, j + 8) of a word, 4^(j % 4) times.
template <int BITS>
__device__ __forceinline__ int code_pos(int j) {
    if constexpr (BITS == 8) return j;
    else if constexpr (BITS == 4) return (j & 8) | ((j & 3) << 1) | ((j >> 2) & 1);
    else return ((j & 7) << 1) | (j >> 3);
}
template <int BITS>
__device__ __forceinline__ float code_scale(int j) {
    if constexpr (BITS == 8) return 1.0f;
    else if constexpr (BITS == 4) return (j & 1) ? 0.0625f : 1.0f;
    else return __uint_as_float((127u - 2u * (uint32_t)(j & 3)) << 23);
}
// a lane's codes of one row and sub-block as pairs for the k steps
template <int BITS, int STEPS>
__device__ __forceinline__ void expand(const uint32_t* w, uint32_t (*a)[2]) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        if constexpr (BITS == 8) {
            a[s][0] = __byte_perm(w[s], 0, 0x4140);
            a[s][1] = __byte_perm(w[s], 0, 0x4342);
        } else if constexpr (BITS == 4) {
            const uint32_t v = (s & 1) ? w[s >> 1] >> 8 : w[s >> 1];
            a[s][0] = v & 0x000F000Fu;
            a[s][1] = v & 0x00F000F0u;
        } else {
            const uint32_t v = (s & 2) ? w[s >> 2] >> 8 : w[s >> 2];
            a[s][0] = v & ((s & 1) ? 0x00300030u : 0x00030003u);
            a[s][1] = v & ((s & 1) ? 0x00C000C0u : 0x000C000Cu);
        }
    }
}
// the pairs of k step s as they are for codes of one
template <int BITS>
__device__ __forceinline__ void ones(int s, uint32_t& lo, uint32_t& hi) {
    if constexpr (BITS == 8) lo = hi = 0x00010001u;
    else if constexpr (BITS == 4) { lo = 0x00010001u; hi = 0x00100010u; }
    else { lo = (s & 1) ? 0x00100010u : 0x00010001u; hi = (s & 1) ? 0x00400040u : 0x00040004u; }
}
constexpr float CODE = 0x1p24f;        // a code's weight in the sums

__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// ---- routing and x ----

struct Routing {
    uint64_t mask[MAX_EXPERTS];              // tokens of each expert
    uint16_t sel[MAX_TOKENS * MAX_TOPK];     // the chosen expert, 0xffff: none
    uint16_t entry[MAX_ENTRIES];             // work list: expert | token block << 12
    int entries;
};
constexpr int PREP_WARPS = 32;

__device__ __forceinline__ uint32_t ordered(float v) {   // order-preserving; NaN above everything, -inf is 0: never chosen
    if (v != v) return 0xffffffffu;
    if (v == -INFINITY) return 0u;
    v += 0.0f;                                           // -0 and 0 tie
    const uint32_t u = __float_as_uint(v);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int EPL>
__device__ __forceinline__ void route_tokens(const Args& a, Routing& R, int warp, int lane) {
    for (int t = warp; t < a.T; t += PREP_WARPS) {
        float v[EPL];
        uint32_t key[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane + 32 * j;
            v[j] = -INFINITY;
            if (e < a.E) {
                const int64_t off = t * a.l_row + e;
                v[j] = a.ldt == (int)DT::F32 ? __ldcg(reinterpret_cast<const float*>(a.logits) + off)
                       : a.ldt == (int)DT::BF16
                           ? half_bits_to_float(__ldcg(reinterpret_cast<const unsigned short*>(a.logits) + off), bf16_t{})
                           : half_bits_to_float(__ldcg(reinterpret_cast<const unsigned short*>(a.logits) + off), f16_t{});
            }
            key[j] = ordered(v[j]);
        }
        float top = 0.0f, mine = 0.0f;       // lane j of the warp keeps choice j's value
        int chosen = 0xffff;
        for (int k = 0; k < a.topk; ++k) {
            uint32_t best = 0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) best = max(best, key[j]);
            best = __reduce_max_sync(0xffffffffu, best);
            if (best == 0) break;            // only -inf left
            uint32_t at = 0xffffffffu;
            float val = 0.0f;
#pragma unroll
            for (int j = EPL - 1; j >= 0; --j)
                if (key[j] == best) {
                    at = lane + 32 * j;
                    val = v[j];
                }
            const uint32_t e = __reduce_min_sync(0xffffffffu, at);   // of equal values the lowest expert
            val = __shfl_sync(0xffffffffu, val, e & 31);
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (e == (uint32_t)(lane + 32 * j)) key[j] = 0;
            if (k == 0) top = val;
            if (lane == k) {
                mine = val;
                chosen = (int)e;
            }
            if (lane == 0) atomicOr(reinterpret_cast<unsigned long long*>(&R.mask[e]), 1ull << t);
        }
        const float p = chosen != 0xffff ? expf(mine - top) : 0.0f;
        float sum = p;
        if (!a.norm) {
            sum = 0.0f;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (v[j] != -INFINITY) sum += expf(v[j] - top);
        }
        sum = warp_sum(sum);
        if (lane < a.topk) {
            R.sel[t * a.topk + lane] = (uint16_t)chosen;
            a.weight[t * a.topk + lane] = p / sum;
        }
    }
}

// Block 0 routes all tokens; block 1 + t prepares token t.
template <int BITS, typename XT>
__global__ void __launch_bounds__(32 * PREP_WARPS) prep_kernel(const __grid_constant__ Args a) {
    __shared__ Routing R;
    __shared__ float red[2][PREP_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::pdl_wait();                 // x and the logits may come from the kernel before, and the workspace be in use
    ptx::pdl_launch_dependents();
    if (blockIdx.x > 0) {
        const int t = blockIdx.x - 1;
        const uint16_t* x = a.x + t * a.x_row;
        float am = 0.0f, s2 = 0.0f;
        for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
            const float v = half_bits_to_float(__ldcg(x + k), XT{});
            am = fmaxf(am, fabsf(v));
            s2 = fmaf(v, v, s2);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        s2 = warp_sum(s2);
        if (lane == 0) {
            red[0][warp] = am;
            red[1][warp] = s2;
        }
        __syncthreads();
        am = s2 = 0.0f;
#pragma unroll
        for (int w = 0; w < PREP_WARPS; ++w) {
            am = fmaxf(am, red[0][w]);
            s2 += red[1][w];
        }
        // 2^(14 - exponent of the largest value): exact products (an infinity's exponent stays in range)
        const int ex = min(max((int)((__float_as_uint(am) >> 23) & 255) - 127, -100), 127);
        const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
        const int kp = x_pitch(a.K);         // padded with zeros to whole stages
        for (int k = threadIdx.x; k < kp; k += blockDim.x) {
            const int j = k & 15;
            const float v = k < a.K ? half_bits_to_float(__ldcg(x + k), XT{}) * up : 0.0f;
            a.xh[(int64_t)t * kp + (k & ~15) + code_pos<BITS>(j)] = float_to_half_bits(v * code_scale<BITS>(j), f16_t{});
        }
        if (threadIdx.x == 0) {
            const float norm = a.rms_eps > 0.0f ? rsqrtf(s2 / (float)a.K + a.rms_eps) : 1.0f;
            a.xfac[t] = __uint_as_float((uint32_t)(ex - 14 + 127) << 23) * norm;
        }
        return;
    }
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) R.mask[e] = 0;
    for (int i = threadIdx.x; i < a.T * a.topk; i += blockDim.x) a.hmax[i] = 0;
    __syncthreads();
    if (a.E <= 128) route_tokens<4>(a, R, warp, lane);
    else route_tokens<MAX_EXPERTS / 32>(a, R, warp, lane);
    __syncthreads();
    if (warp == 0) {
        int n = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int blocks = e < a.E ? (__popcll(R.mask[e]) + TB - 1) / TB : 0;
            int incl = blocks;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += u;
            }
            for (int b = 0; b < blocks; ++b) R.entry[n + incl - blocks + b] = (uint16_t)(e | (b << 12));
            n += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) R.entries = n;
    }
    __syncthreads();
    if (threadIdx.x == 0) a.entries[0] = R.entries;
    for (int i = warp; i < R.entries; i += PREP_WARPS) {
        const int e = R.entry[i] & 0xfff, first = (R.entry[i] >> 12) * TB;
        const uint64_t m = R.mask[e];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = lane + 32 * half;
            if ((m >> t) & 1) {
                const int rank = __popcll(m & ((1ull << t) - 1)) - first;
                if (rank >= 0 && rank < TB) {
                    int j = 0;
                    while (j + 1 < a.topk && R.sel[t * a.topk + j] != e) ++j;
                    a.pairs[i * TB + rank] = (uint16_t)(t * a.topk + j);
                }
            }
        }
        if (lane == 0) a.entries[1 + i] = e | (min(__popcll(m) - first, TB) << 16);
    }
}

// ---- streams of packed codes ----

__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, int size) {   // size 0: zeros, nothing is read
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ int swz(int row) { return ((row >> 1) & 1) << 1; }   // spreads 32-byte reads over the banks

__device__ __forceinline__ void cp_small(uint32_t dst, const void* src, int bytes) {   // 4 or 8
    if (bytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// One row's scales (or biases) of a stage into the ring: the GPS halves from p + g0.  Where rows keep them
// aligned (vec), one asynchronous copy of the 4 or 8 bytes that hold them (a single one, GPS 1, with its even
// or odd neighbour); else through registers.
template <int GPS, int SBB>
__device__ __forceinline__ void copy_sb(uint32_t dst, const uint16_t* p, int g0, int kg, bool vec) {
    if (vec) {
        cp_small(dst, p + (GPS == 1 ? g0 & ~1 : g0), SBB);
        return;
    }
    uint32_t w[SBB / 4];
#pragma unroll
    for (int i = 0; i < SBB / 4; ++i) {
        // GPS 1: the value in both halves
        const uint32_t lo = __ldg(p + min(g0 + 2 * i, kg - 1)), hi = GPS == 1 ? lo : (uint32_t)__ldg(p + min(g0 + 2 * i + 1, kg - 1));
        w[i] = lo | (hi << 16);
    }
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(w[0]) : "memory");
    if constexpr (SBB == 8) asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + 4), "r"(w[1]) : "memory");
}
// value f of a row's scales in the ring; g0: the stage's first group
template <int GPS, typename XT>
__device__ __forceinline__ float sb_value(const uint32_t* v, int f, int g0) {
    if constexpr (GPS == 1) return half_bits_to_float((uint16_t)((g0 & 1) ? v[0] >> 16 : v[0]), XT{});
    const uint32_t w = v[f >> 1];
    return half_bits_to_float((uint16_t)((f & 1) ? w >> 16 : w), XT{});
}
// GPS values of a row of a block (rows hold a multiple of GPS, or of 2)
template <int GPS>
__device__ __forceinline__ void read_blk(const uint16_t* p, uint32_t (&v)[(GPS + 1) / 2]) {
    if constexpr (GPS == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        v[0] = u.x; v[1] = u.y;
    } else if constexpr (GPS == 2) {
        v[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
        v[0] = *p;
    }
}
template <int GPS, typename XT>
__device__ __forceinline__ float blk_value(const uint32_t* v, int f) {
    const uint32_t w = v[f >> 1];
    return half_bits_to_float((uint16_t)((f & 1) ? w >> 16 : w), XT{});
}
// A wait for a block's copies, bounded: on expiry the error word says so, and the results are void.
__device__ __forceinline__ void wait_block(uint64_t* bar, uint32_t parity, int* err) {
    volatile int never = 0;
    if (!ptx::mbar_wait(bar, parity, &never, WAIT_NS)) atomicOr(err, DEVERR_TIMEOUT);
}
template <int SBB>
__device__ __forceinline__ void read_sb(const uint8_t* p, uint32_t* v) {
    if constexpr (SBB == 8) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        v[0] = u.x; v[1] = u.y;
    } else {
        v[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}
// One k step of a tile: both row blocks' sums and the sum over the tokens' own values; `first` starts them.
template <int BITS, int STEPS>
__device__ __forceinline__ void mma_step(float (&d0)[4], float (&d1)[4], float (&X)[4], const uint32_t (&fr)[4][STEPS][2], int k,
                                     const uint32_t* b, bool first) {
    uint32_t lo, hi;
    ones<BITS>(k, lo, hi);
    if (first) {
        mma0(d0, fr[0][k][0], fr[1][k][0], fr[0][k][1], fr[1][k][1], b[2 * k], b[2 * k + 1]);
        mma0(d1, fr[2][k][0], fr[3][k][0], fr[2][k][1], fr[3][k][1], b[2 * k], b[2 * k + 1]);
        mma0(X, lo, lo, hi, hi, b[2 * k], b[2 * k + 1]);
    } else {
        wm::mma16816<false>(d0, fr[0][k][0], fr[1][k][0], fr[0][k][1], fr[1][k][1], b[2 * k], b[2 * k + 1]);
        wm::mma16816<false>(d1, fr[2][k][0], fr[3][k][0], fr[2][k][1], fr[3][k][1], b[2 * k], b[2 * k + 1]);
        wm::mma16816<false>(X, lo, lo, hi, hi, b[2 * k], b[2 * k + 1]);
    }
}

// f16 numbers that an activation goes to the down product in: one for bf16 outputs, whose rounding is 8 times its
// own; two (22 bits) for f16 outputs, whose rounding it would equal (2 tokens, 16 experts: 3.1e-4 off instead of
// the 2.0e-4 of the output's rounding alone), and for f32 outputs, whatever x is (a bf16 x, 64 tokens, 4-bit experts: 2.1e-4
// off in one part, 2.8e-5 in two, in 150 instead of 108 us).
inline int parts_of(bool bf16, int ydt) { return bf16 && ydt == (int)DT::BF16 ? 1 : 2; }

// The power of two 2^(e - 14) with 2^e above v, in f16's range around v.
__device__ __forceinline__ float scale_for(float v) {
    const int ex = min(max((int)((__float_as_uint(v) >> 23) & 255) - 126, -100), 127);
    return __uint_as_float((uint32_t)(ex - 14 + 127) << 23);
}
__device__ __forceinline__ float pow2_inverse(float v) { return __uint_as_float(0x7F000000u - __float_as_uint(v)); }

// ---- gate/up ----

// SHARED: the CTA's warps share an item, each a quarter of its stages; else a warp has items of its own.
template <int BITS, typename XT, int G, bool SHARED>
__global__ void __launch_bounds__(THREADS, 3) gate_up_kernel(const __grid_constant__ Args a) {
    using Gm = Geo<BITS, G>;
    constexpr int GPS = Gm::GPS, XV = Gm::KS / 32;
    constexpr int NST = Gm::NST, HALF = Gm::half(!SHARED), STAGE = 2 * HALF, SBB = Gm::SBB;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t sb_bar[WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;
    const int kg = a.K / G;
    uint8_t* ring = smem + warp * NST * STAGE;
    const uint32_t ring_s = ptx::smem_u32(ring);
    float* red = reinterpret_cast<float*>(smem + Gm::ring(Gm::NST, false));   // SHARED: [2][WARPS][16][32]
    // not SHARED: this warp's item's scales and biases, [gate s, up s, gate b, up b][16 rows][kg]
    uint16_t* blk = reinterpret_cast<uint16_t*>(smem + Gm::ring(Gm::NST, true)) + warp * 64 * kg;
    if (!SHARED) {
        if (lane == 0) ptx::mbar_init(&sb_bar[warp], 1);
        ptx::fence_mbar_init();
        __syncwarp();
    }

    ptx::pdl_wait();                 // routing and x
    ptx::pdl_launch_dependents();    // after the wait: the down kernel reads the routing before its own

    const int nb_all = a.N / 16;
    const int items = __ldcg(a.entries) * nb_all;
    const int kp = x_pitch(a.K);
    const int nst = (a.K + 2 * Gm::SC - 1) / (2 * Gm::SC);
    const int s0 = SHARED ? warp : 0;
    constexpr int SSTEP = SHARED ? WARPS : 1;
    const int nsw = nst > s0 ? (nst - s0 + SSTEP - 1) / SSTEP : 0;   // stages of this warp per item
    const int row_bytes = a.K * BITS / 8;
    const int first = SHARED ? blockIdx.x : blockIdx.x * WARPS + warp;
    const int step = SHARED ? gridDim.x : gridDim.x * WARPS;

    // load cursor: the item, stage and ring slot of the next load, its rows' addresses, and the expert of
    // the item after it
    int l_item = first, l_s = 0, l_slot = 0, l_next = 0;
    const uint8_t *l_gate = nullptr, *l_up = nullptr;
    const uint16_t *l_sc = nullptr, *l_bi = nullptr;     // of row `lane` of the stage: 16 gate rows, 16 up rows
    if (l_item < items) l_next = __ldcg(a.entries + 1 + l_item / nb_all);
    auto issue = [&]() {
        if (l_item < items && nsw > 0) {
            if (l_s == 0) {
                const int ent = l_item / nb_all, n0 = (l_item - ent * nb_all) * 16;
                const int e = l_next & 0xffff;
                if (l_item + step < items) l_next = __ldcg(a.entries + 1 + (l_item + step) / nb_all);
                l_gate = reinterpret_cast<const uint8_t*>(a.gate.wq + e * a.gate.w_exp + (n0 + r) * a.gate.w_row) + c * 16;
                l_up = reinterpret_cast<const uint8_t*>(a.up.wq + e * a.up.w_exp + (n0 + r) * a.up.w_row) + c * 16;
                if constexpr (SHARED) {
                    const Bank& B = lane < 16 ? a.gate : a.up;
                    const int64_t so = (int64_t)(n0 + (lane & 15)) * kg;
                    l_sc = B.scales + e * B.s_exp + so;
                    l_bi = B.biases + e * B.b_exp + so;
                } else if (lane < 4) {   // on their way to L2, for the bulk copies at the item's turn
                    const Bank& B = (lane & 1) ? a.up : a.gate;
                    ptx::prefetch_l2_bulk((lane < 2 ? B.scales + e * B.s_exp : B.biases + e * B.b_exp) + (int64_t)n0 * kg, 32 * kg);
                }
            }
            const int st = s0 + l_s * SSTEP, off = st * 128;
            const uint32_t slot0 = ring_s + l_slot * STAGE, dst = slot0 + r * 64 + ((c ^ swz(r)) << 4);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int size = off + hf * 64 + c * 16 < row_bytes ? 16 : 0;
                const int o = size ? off + hf * 64 : 0;
                cp16z(dst + hf * HALF, l_gate + o, size);
                cp16z(dst + hf * HALF + 8 * 64, l_gate + o + 32 * a.gate.w_row, size);
                cp16z(dst + hf * HALF + 16 * 64, l_up + o, size);
                cp16z(dst + hf * HALF + 24 * 64, l_up + o + 32 * a.up.w_row, size);
                if (SHARED && off + hf * 64 < row_bytes) {   // a half that K reaches: its folds are all there, or rows are not vec
                    const int g = (2 * st + hf) * Gm::SC / G;
                    copy_sb<GPS, SBB>(slot0 + hf * HALF + Gm::CODES + lane * SBB, l_sc, g, kg, a.gate.svec);
                    copy_sb<GPS, SBB>(slot0 + hf * HALF + Gm::CODES + (ROWS + lane) * SBB, l_bi, g, kg, a.gate.svec);
                }
            }
            if (++l_s == nsw) {
                l_s = 0;
                l_item += step;
            }
            if (++l_slot == NST) l_slot = 0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) issue();

    // the first item's entry and tokens (later ones are fetched an item ahead)
    int next_ent = 0, next_pair = 0;
    auto fetch_item = [&](int item) {
        if (item < items) {
            const int ent = item / nb_all;
            next_ent = __ldcg(a.entries + 1 + ent);
            next_pair = __ldcg(a.pairs + ent * TB + (lane & 15));
        }
    };
    fetch_item(first);
    // one item's scales and biases, whole, into the block (four lanes, one run each)
    auto load_block = [&](int item) {
        if constexpr (!SHARED) {
            if (item < items && lane < 4) {
                const int e = next_ent & 0xffff, n0 = item % nb_all * 16;
                const Bank& B = (lane & 1) ? a.up : a.gate;
                if (lane == 0) ptx::mbar_arrive_expect_tx(&sb_bar[warp], 128 * kg);
                __syncwarp(0xf);
                ptx::bulk_load(blk + lane * 16 * kg, (lane < 2 ? B.scales + e * B.s_exp : B.biases + e * B.b_exp) + (int64_t)n0 * kg,
                               32 * kg, &sb_bar[warp]);
            }
            __syncwarp();
        }
    };
    load_block(first);

    uint32_t turn = 0;
    int slot = 0, buf = 0;
    for (int item = first; item < items; item += step, buf ^= 1) {
        const int nt = next_ent >> 16, pair = next_pair;
        const int nb = item % nb_all, n0 = nb * 16;
        fetch_item(item + step);
        // this lane's x rows (token r of each tile; past the last one: the last one)
        const uint16_t* xr[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
            xr[t] = a.xh + (int64_t)(__shfl_sync(0xffffffffu, pair, min(8 * t + r, nt - 1)) / a.topk) * kp + c * (Gm::KS / 4);
        float acc[2][2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[m][t][q] = 0.0f;

        auto stages = [&](auto tiles) {
            constexpr int NT = decltype(tiles)::value;
            // x: one tile's is fetched half a stage ahead (PRE), two tiles' for the whole half at once or, where
            // registers are short, sub-block by sub-block
            constexpr bool AHEAD = NT * Gm::SUBS * XV <= 4, PRE = NT == 1 && AHEAD;
            uint4 xv[NT][AHEAD ? Gm::SUBS * XV : XV];
            auto load_x = [&](int st, int sb, int at) {
                const int k0 = st * Gm::SC + sb * Gm::KS;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int v = 0; v < XV; ++v)
                        xv[t][at + v] = reinterpret_cast<const uint4*>(xr[t] + k0)[v];
            };
            auto load_half = [&](int st) {
                if constexpr (AHEAD)
#pragma unroll
                    for (int sb = 0; sb < Gm::SUBS; ++sb) load_x(st, sb, sb * XV);
            };
            if (PRE && nsw > 0) load_half(2 * s0);
            if constexpr (!SHARED) wait_block(&sb_bar[warp], turn & 1, a.err);
#pragma unroll 1
            for (int s = 0; s < nsw; ++s) {
              issue();
              asm volatile("cp.async.wait_group %0;" ::"n"(NST - 1) : "memory");
              __syncwarp();
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                const int st = 2 * (s0 + s * SSTEP) + hf;    // in halves
                if (hf == 1 && st * Gm::SC >= a.K) break;    // K ends with the first half
                if (!PRE) load_half(st);
                const uint8_t* stage = ring + slot * STAGE + hf * HALF + r * 64;
                const uint8_t* sbp = ring + slot * STAGE + hf * HALF + Gm::CODES + r * SBB;
                const int g0 = st * Gm::SC / G;
                uint4 xc[NT][AHEAD ? Gm::SUBS * XV : XV];
                if constexpr (AHEAD)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int v = 0; v < Gm::SUBS * XV; ++v) xc[t][v] = xv[t][v];
                // (x is padded to whole stages: the half after this one is there, whether it counts or not)
                if (PRE && (hf == 0 || s + 1 < nsw)) load_half(hf == 0 ? st + 1 : st + 2 * SSTEP - 1);
                [[maybe_unused]] uint32_t bs[4][(GPS + 1) / 2], bb_[4][(GPS + 1) / 2];    // scales and biases of rows r + 8 i
                if constexpr (!SHARED) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        read_blk<GPS>(blk + (i * 8 + r) * kg + g0, bs[i]);
                        read_blk<GPS>(blk + (i * 8 + r + 32) * kg + g0, bb_[i]);
                    }
                }
                float d[2][NT][4], X[NT][4];     // rows of X are alike: elements 0, 1 are those of tokens 2c, 2c + 1
#pragma unroll
                for (int sb = 0; sb < Gm::SUBS; ++sb) {
                    if constexpr (!AHEAD) {
                        load_x(st, sb, 0);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int v = 0; v < XV; ++v) xc[t][v] = xv[t][v];
                    }
                    uint32_t fr[4][Gm::STEPS][2];
                    const int off = sb * 4 * Gm::LB + c * Gm::LB;
                    const uint8_t* wp = stage + (((off >> 4) ^ swz(r)) << 4) + (off & 15);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[Gm::LB / 4];
                        wm::load_lane_words<Gm::LB>(wp + i * 8 * 64, w);
                        expand<BITS, Gm::STEPS>(w, fr[i]);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint32_t* xw = reinterpret_cast<const uint32_t*>(&xc[t][AHEAD ? sb * XV : 0]);
#pragma unroll
                        for (int k = 0; k < Gm::STEPS; ++k) mma_step<BITS>(d[0][t], d[1][t], X[t], fr, k, xw, sb % Gm::SPF == 0 && k == 0);
                    }
                    if (sb % Gm::SPF == Gm::SPF - 1) {
                        const int f = sb / Gm::SPF;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int m = i >> 1, h = i & 1;
                            float ss, bb;
                            if constexpr (SHARED) {
                                uint32_t sv[SBB / 4], bv[SBB / 4];
                                read_sb<SBB>(sbp + i * 8 * SBB, sv);
                                read_sb<SBB>(sbp + ROWS * SBB + i * 8 * SBB, bv);
                                ss = sb_value<GPS, XT>(sv, f, g0);
                                bb = sb_value<GPS, XT>(bv, f, g0);
                            } else {
                                ss = blk_value<GPS, XT>(bs[i], f);
                                bb = blk_value<GPS, XT>(bb_[i], f);
                            }
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int q = 0; q < 2; ++q)
                                    acc[m][t][2 * h + q] = fmaf(ss, d[m][t][2 * h + q], fmaf(bb, X[t][q], acc[m][t][2 * h + q]));
                        }
                    }
                }
              }
              __syncwarp();
              if (++slot == NST) slot = 0;
            }
        };
        if (nt > 8) stages(std::integral_constant<int, 2>{});
        else stages(std::integral_constant<int, 1>{});
        load_block(item + step);     // every lane has read this item's
        ++turn;

        // ---- silu(gate) * up * weight, for columns r and r + 8 and tokens 2c, 2c + 1 of each tile ----
        if constexpr (SHARED) {      // the warps' slices of K together, in slice order, by the first warp's lanes
            float* rw = red + buf * WARPS * 16 * 32;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) rw[(warp * 16 + m * 8 + t * 4 + q) * 32 + lane] = acc[m][t][q];
            __syncthreads();
            if (warp != 0) continue;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int w = 1; w < WARPS; ++w) acc[m][t][q] += rw[(w * 16 + m * 8 + t * 4 + q) * 32 + lane];
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (t == 1 && nt <= 8) break;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int i = 8 * t + 2 * c + q;
                const bool live = i < nt;
                const int p = __shfl_sync(0xffffffffu, pair, live ? i : 0);
                const float fac = __ldcg(a.xfac + p / a.topk), w = __ldcg(a.weight + p);
                const float v0 = wm::silu(acc[0][t][q] * CODE * fac) * (acc[1][t][q] * CODE * fac) * w;
                const float v1 = wm::silu(acc[0][t][2 + q] * CODE * fac) * (acc[1][t][2 + q] * CODE * fac) * w;
                float m = fmaxf(fabsf(v0), fabsf(v1));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                const float sc = scale_for(m), inv = pow2_inverse(sc);
                if (live) {
                    uint16_t* hp = a.h + (int64_t)p * a.N + n0;
                    const float u0 = v0 * inv * code_scale<BITS>(r), u1 = v1 * inv * code_scale<BITS>(r + 8);
                    const uint16_t h0 = float_to_half_bits(u0, f16_t{}), h1 = float_to_half_bits(u1, f16_t{});
                    hp[code_pos<BITS>(r)] = h0;
                    hp[code_pos<BITS>(r + 8)] = h1;
                    if (std::is_same<XT, f16_t>::value || a.parts == 2) {
                        hp += (int64_t)a.T * a.topk * a.N;
                        hp[code_pos<BITS>(r)] = float_to_half_bits(u0 - half_bits_to_float(h0, f16_t{}), f16_t{});
                        hp[code_pos<BITS>(r + 8)] = float_to_half_bits(u1 - half_bits_to_float(h1, f16_t{}), f16_t{});
                    }
                    if (r == 0) {
                        a.hscale[(int64_t)p * nb_all + nb] = sc;
                        atomicMax(a.hmax + p, __float_as_uint(sc));
                    }
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---- down ----

// BLK: an entry's scales and biases come whole into one of two blocks that the CTA's warps share.
// P: parts of an activation.
template <int BITS, typename XT, int G, bool BLK, int P>
__global__ void __launch_bounds__(THREADS, 3) down_kernel(const __grid_constant__ Args a) {
    using Gm = Geo<BITS, G>;
    constexpr int GPS = Gm::GPS, XV = Gm::KS / 32;
    constexpr int NST = Gm::NST_DOWN, HALF = Gm::half(BLK), STAGE = 2 * HALF, SBB = Gm::SBB;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t sb_full[2];
    __shared__ int sb_left[2];       // warps that have left a block's entry
    const int kg = a.N / G;
    uint16_t* blk = reinterpret_cast<uint16_t*>(smem + Gm::ring(NST, BLK));   // BLK: [2][scales, biases][ROWS][kg]
    float* yt = reinterpret_cast<float*>(smem + Gm::ring(NST, BLK) + (BLK ? 2 * 128 * kg : 0));   // [WARPS][T][RP]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;
    const int cs = a.cs;
    const int rank = cs > 1 ? (int)ptx::cluster_ctarank() : 0;
    const int row0 = (int)(blockIdx.x / cs) * ROWS;      // first column of y

    const int entries = __ldcg(a.entries);               // complete: the gate/up kernel waited for it before this one started
    const int nb_all = a.N / 16;
    const int nst = (a.N + 2 * Gm::SC - 1) / (2 * Gm::SC);
    const int row_bytes = a.N * BITS / 8;
    uint8_t* ring = smem + warp * NST * STAGE;
    const uint32_t ring_s = ptx::smem_u32(ring);

    // The CTA's entries are one row of stages, dealt to the warps in turn: with each entry dealt anew, 6 stages an
    // entry left two of the four warps waiting half of the time.
    int l_ent = rank, l_s = warp, l_slot = 0, l_next = 0;
    bool l_new = true;
    auto settle = [&]() {        // the entry that the next stage is in, and its expert
        while (l_s >= nst && l_ent < entries) {
            l_s -= nst;
            l_ent += cs;
            l_new = true;
        }
        if (l_new && l_ent < entries) l_next = __ldcg(a.entries + 1 + l_ent);
    };
    const uint8_t* l_row[4] = {nullptr, nullptr, nullptr, nullptr};
    const uint16_t *l_sc = nullptr, *l_bi = nullptr;     // of row `lane`
    settle();
    auto issue = [&]() {
        if (l_ent < entries) {
            if (l_new) {
                l_new = false;
                const int e = l_next & 0xffff;
                const uint8_t* wp = reinterpret_cast<const uint8_t*>(a.down.wq + e * a.down.w_exp) + c * 16;
#pragma unroll
                for (int i = 0; i < 4; ++i) l_row[i] = wp + min(row0 + r + 8 * i, a.K - 1) * a.down.w_row * 4;
                const int64_t so = (int64_t)min(row0 + lane, a.K - 1) * kg;
                if constexpr (!BLK) {
                    l_sc = a.down.scales + e * a.down.s_exp + so;
                    l_bi = a.down.biases + e * a.down.b_exp + so;
                }
            }
            const int off = l_s * 128;
            const uint32_t slot0 = ring_s + l_slot * STAGE, dst = slot0 + r * 64 + ((c ^ swz(r)) << 4);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int size = off + hf * 64 + c * 16 < row_bytes ? 16 : 0;
                const int o = size ? off + hf * 64 : 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) cp16z(dst + hf * HALF + i * 8 * 64, l_row[i] + o, size);
                if (!BLK && off + hf * 64 < row_bytes) {
                    const int g = (2 * l_s + hf) * Gm::SC / G;
                    copy_sb<GPS, SBB>(slot0 + hf * HALF + Gm::CODES + lane * SBB, l_sc, g, kg, a.down.svec);
                    copy_sb<GPS, SBB>(slot0 + hf * HALF + Gm::CODES + (ROWS + lane) * SBB, l_bi, g, kg, a.down.svec);
                }
            }
            l_s += WARPS;
            settle();
            if (++l_slot == NST) l_slot = 0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) issue();
    if (BLK && threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sb_full[i], 1);
            sb_left[i] = 0;
        }
        ptx::fence_mbar_init();
    }
    // entry number i of this CTA, of expert e, into block i % 2: by one thread, once every warp has left the block
    auto load_block = [&](int i, int e) {
        uint16_t* dst = blk + (i & 1) * 64 * kg;
        ptx::mbar_arrive_expect_tx(&sb_full[i & 1], 128 * kg);
        ptx::bulk_load(dst, a.down.scales + e * a.down.s_exp + (int64_t)row0 * kg, 64 * kg, &sb_full[i & 1]);
        ptx::bulk_load(dst + 32 * kg, a.down.biases + e * a.down.b_exp + (int64_t)row0 * kg, 64 * kg, &sb_full[i & 1]);
    };
    for (int i = threadIdx.x; i < WARPS * a.T * RP; i += THREADS) yt[i] = 0.0f;
    int next_ent = 0, next_pair = 0;
    auto fetch_entry = [&](int ent) {
        if (ent < entries) {
            next_ent = __ldcg(a.entries + 1 + ent);
            next_pair = __ldcg(a.pairs + ent * TB + (lane & 15));
        }
    };
    fetch_entry(rank);
    __syncthreads();             // the y tiles are zero, the barriers ready
    if (BLK && threadIdx.x == 0)
        for (int i = 0; i < 2; ++i)
            if (rank + i * cs < entries) load_block(i, __ldcg(a.entries + 1 + rank + i * cs) & 0xffff);
    __syncwarp();

    ptx::pdl_wait();             // the activations
    ptx::pdl_launch_dependents();

    const int64_t rest = (int64_t)a.T * a.topk * a.N;    // from the activations to their rest
    int slot = 0, turn = 0, s0 = warp;   // s0: this warp's next stage, in the current entry
    float* yw = yt + warp * a.T * RP;
    for (int ent = rank; ent < entries; ent += cs, ++turn) {
        int after = 0;               // the entry that this one's block takes next
        if constexpr (BLK) if (ent + 2 * cs < entries) after = __ldcg(a.entries + 1 + ent + 2 * cs);
        if constexpr (BLK) wait_block(&sb_full[turn & 1], (uint32_t)(turn / 2) & 1, a.err);
        const uint16_t* bk = blk + (turn & 1) * 64 * kg + r * kg;
        const int nt = next_ent >> 16, pair = next_pair;
        fetch_entry(ent + cs);
        // token r of each tile: its activations and their powers of two, against the row's largest; tokens 2c and
        // 2c + 1: that largest
        const uint16_t* hp[2];
        const float* hsp[2];
        float hinv[2], top[2][2];
        int px[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int po = __shfl_sync(0xffffffffu, pair, min(8 * t + r, nt - 1));
            hp[t] = a.h + (int64_t)po * a.N + c * (Gm::KS / 4);
            hsp[t] = a.hscale + (int64_t)po * nb_all + c * (Gm::KS / 4) / 16;
            const float mine = __uint_as_float(__ldcg(a.hmax + po));
            hinv[t] = pow2_inverse(mine);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                px[t][q] = __shfl_sync(0xffffffffu, pair, min(8 * t + 2 * c + q, nt - 1));
                top[t][q] = __shfl_sync(0xffffffffu, mine, 8 * c + 4 * q);
            }
        }
        float acc[2][2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[m][t][q] = 0.0f;

        auto stages = [&](auto tiles) {
            constexpr int NT = decltype(tiles)::value;
            // activations and their powers of two: one tile's are fetched half a stage ahead (PRE), two tiles' for the
            // whole half at once or, where registers are short, sub-block by sub-block
            constexpr bool AHEAD = NT * P * Gm::SUBS * XV <= 4, PRE = NT == 1 && AHEAD;
            uint4 hv[NT][P][AHEAD ? Gm::SUBS * XV : XV];
            float hs[NT][AHEAD ? Gm::SUBS : 1];
            auto load_h = [&](int st, int sb, int at) {
                const int k0 = st * Gm::SC + sb * Gm::KS;
                if (!BLK && k0 >= a.N) return;       // (rows in blocks hold whole halves)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int p = 0; p < P; ++p)
#pragma unroll
                        for (int v = 0; v < XV; ++v)
                            hv[t][p][at * XV + v] = reinterpret_cast<const uint4*>(hp[t] + p * rest + k0)[v];
                    hs[t][at] = hsp[t][k0 / 16];
                }
            };
            auto load_half = [&](int st) {
#pragma unroll
                for (int sb = 0; sb < Gm::SUBS; ++sb) load_h(st, sb, AHEAD ? sb : 0);
            };
            if (PRE) load_half(2 * s0);
#pragma unroll 1
            for (; s0 < nst; s0 += WARPS) {
              issue();
              asm volatile("cp.async.wait_group %0;" ::"n"(NST - 1) : "memory");
              __syncwarp();
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                const int st = 2 * s0 + hf;  // in halves
                if (hf == 1 && st * Gm::SC >= a.N) break;
                const int g0 = st * Gm::SC / G;
                if (AHEAD && !PRE) load_half(st);
                uint4 hc[NT][P][AHEAD ? Gm::SUBS * XV : XV];
                float hsc[NT][AHEAD ? Gm::SUBS : 1];
                if constexpr (AHEAD) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
#pragma unroll
                        for (int p = 0; p < P; ++p)
#pragma unroll
                            for (int v = 0; v < Gm::SUBS * XV; ++v) hc[t][p][v] = hv[t][p][v];
#pragma unroll
                        for (int v = 0; v < Gm::SUBS; ++v) hsc[t][v] = hs[t][v];
                    }
                }
                if (PRE) {
                    const int next = hf == 0 ? st + 1 : st + 2 * WARPS - 1;
                    if (next * Gm::SC < a.N) load_half(next);
                }
                const uint8_t* stage = ring + slot * STAGE + hf * HALF + r * 64;
                const uint8_t* sbp = ring + slot * STAGE + hf * HALF + Gm::CODES + r * SBB;
                [[maybe_unused]] uint32_t bs[4][(GPS + 1) / 2], bb_[4][(GPS + 1) / 2];    // scales and biases of rows r + 8 i
                if constexpr (BLK) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        read_blk<GPS>(bk + i * 8 * kg + g0, bs[i]);
                        read_blk<GPS>(bk + (i * 8 + 32) * kg + g0, bb_[i]);
                    }
                }
                float d[2][NT][4], X[NT][4];
#pragma unroll
                for (int sb = 0; sb < Gm::SUBS; ++sb) {
                    if (!BLK && st * Gm::SC + sb * Gm::KS >= a.N) break;
                    if constexpr (!AHEAD) {
                        load_h(st, sb, 0);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
#pragma unroll
                            for (int p = 0; p < P; ++p)
#pragma unroll
                                for (int v = 0; v < XV; ++v) hc[t][p][v] = hv[t][p][v];
                            hsc[t][0] = hs[t][0];
                        }
                    }
                    uint32_t fr[4][Gm::STEPS][2];
                    const int off = sb * 4 * Gm::LB + c * Gm::LB;
                    const uint8_t* wp = stage + (((off >> 4) ^ swz(r)) << 4) + (off & 15);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[Gm::LB / 4];
                        wm::load_lane_words<Gm::LB>(wp + i * 8 * 64, w);
                        expand<BITS, Gm::STEPS>(w, fr[i]);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const __half2 f = __float2half2_rn(hsc[t][AHEAD ? sb : 0] * hinv[t]);
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            uint32_t* hw = reinterpret_cast<uint32_t*>(&hc[t][p][AHEAD ? sb * XV : 0]);
#pragma unroll
                            for (int k = 0; k < 4 * XV; ++k) {
                                const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&hw[k]), f);
                                hw[k] = *reinterpret_cast<const uint32_t*>(&v);
                            }
#pragma unroll
                            for (int k = 0; k < Gm::STEPS; ++k)
                                mma_step<BITS>(d[0][t], d[1][t], X[t], fr, k, hw, p == 0 && sb % Gm::SPF == 0 && k == 0);
                        }
                    }
                    if (sb % Gm::SPF == Gm::SPF - 1) {
                        const int f = sb / Gm::SPF;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int m = i >> 1, h = i & 1;
                            float ss, bb;
                            if constexpr (BLK) {
                                ss = blk_value<GPS, XT>(bs[i], f);
                                bb = blk_value<GPS, XT>(bb_[i], f);
                            } else {
                                uint32_t sv[SBB / 4], bv[SBB / 4];
                                read_sb<SBB>(sbp + i * 8 * SBB, sv);
                                read_sb<SBB>(sbp + ROWS * SBB + i * 8 * SBB, bv);
                                ss = sb_value<GPS, XT>(sv, f, g0);
                                bb = sb_value<GPS, XT>(bv, f, g0);
                            }
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int q = 0; q < 2; ++q)
                                    acc[m][t][2 * h + q] = fmaf(ss, d[m][t][2 * h + q], fmaf(bb, X[t][q], acc[m][t][2 * h + q]));
                        }
                    }
                }
              }
              __syncwarp();
              if (++slot == NST) slot = 0;
            }
        };
        const bool any = s0 < nst;
        if (any) {
            if (nt > 8) stages(std::integral_constant<int, 2>{});
            else stages(std::integral_constant<int, 1>{});
        }
        s0 -= nst;
        if constexpr (BLK) {         // the last warp to leave has it filled again
            __syncwarp();
            if (lane == 0 && ent + 2 * cs < entries) {
                int left;
                asm volatile("atom.acq_rel.cta.shared.add.s32 %0, [%1], 1;" : "=r"(left) : "r"(ptx::smem_u32(&sb_left[turn & 1])) : "memory");
                if (left == WARPS - 1) {
                    sb_left[turn & 1] = 0;
                    load_block(turn + 2, after & 0xffff);
                }
            }
            __syncwarp();
        }
        // this warp's slice of N into its own tile of y
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (any && 8 * t + 2 * c + q < nt) {
                    float* yp = yw + (px[t][q] / a.topk) * RP;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) yp[16 * m + 8 * h + r] += acc[m][t][2 * h + q] * CODE * top[t][q];
                }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    const int total = a.T * ROWS;
    auto emit = [&](int t, int row, float v) {
        const int n = row0 + row;
        if (n >= a.K) return;
        if (a.r) v += wm::load_out<XT>(a.r, t * a.r_row + n, a.ydt);
        if (a.ydt == (int)DT::F32) reinterpret_cast<float*>(a.y)[t * a.y_row + n] = v;
        else store_out(reinterpret_cast<XT*>(a.y) + t * a.y_row + n, v);
    };
    for (int i = threadIdx.x; i < total; i += THREADS) {
        const int t = i / ROWS, row = i % ROWS;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += yt[(w * a.T + t) * RP + row];
        if (cs == 1) emit(t, row, v);
        else yt[t * RP + row] = v;      // over warp 0's tile: read by this thread alone
    }
    if (cs > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        const uint32_t base = ptx::smem_u32(yt);
        for (int i = rank * THREADS + threadIdx.x; i < total; i += cs * THREADS) {
            const int t = i / ROWS, row = i % ROWS;
            float v = 0.0f;
            for (int q = 0; q < cs; ++q) v += ptx::ld_cluster_f32(ptx::mapa(base + (t * RP + row) * 4, (uint32_t)q));
            emit(t, row, v);
        }
        // no CTA leaves while another may still read its tile
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}

template <int BITS, typename XT, int G>
cudaError_t launch_t(Args a, cudaStream_t st) {
    using Gm = Geo<BITS, G>;
    const int kg = a.K / G, kgd = a.N / G;
    const size_t smem_shared = Gm::ring(Gm::NST, false) + 2 * WARPS * 16 * 32 * sizeof(float);
    const size_t smem_own = Gm::ring(Gm::NST, true) + (size_t)WARPS * 128 * kg;
    const bool blk_down = a.down.blk && kgd <= DOWN_GROUPS;
    const size_t smem_down = Gm::ring(Gm::NST_DOWN, blk_down) + (blk_down ? (size_t)2 * 128 * kgd : 0) + WARPS * a.T * RP * sizeof(float);
    // The down kernel's CTAs all at once on the device, one cluster of up to eight per 32 columns of y, no more
    // CTAs in it than there can be entries (64 tokens, 64 experts of 4 bits: 384 CTAs
    // of 444 that fit 116 us the layer, 512 CTAs 134).
    a.parts = parts_of(std::is_same<XT, bf16_t>::value, a.ydt);
    const int blocks = (a.K + ROWS - 1) / ROWS;
    const int fit = 148 * (int)std::min<size_t>(3, 227 * 1024 / (smem_down + 1024));
    a.cs = std::max(1, std::min({8, fit / blocks, a.T * a.topk, a.E}));
    constexpr int SMEM_MAX = 160 * 1024;
    static std::mutex mu;
    static bool done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev]) {
            constexpr int P1 = std::is_same<XT, bf16_t>::value ? 1 : 2;
            const void* fns[6] = {(const void*)gate_up_kernel<BITS, XT, G, false>, (const void*)gate_up_kernel<BITS, XT, G, true>,
                                  (const void*)down_kernel<BITS, XT, G, false, P1>, (const void*)down_kernel<BITS, XT, G, true, P1>,
                                  (const void*)down_kernel<BITS, XT, G, false, 2>, (const void*)down_kernel<BITS, XT, G, true, 2>};
            for (const void* f : fns) {
                e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
                if (e != cudaSuccess) return e;
            }
            done[dev] = true;
        }
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(1 + a.T));
    cfg.blockDim = dim3(32 * PREP_WARPS);
    e = cudaLaunchKernelEx(&cfg, prep_kernel<BITS, XT>, a);
    if (e != cudaSuccess) return e;
    // As many items as the tokens could choose, at most what fits the device at once (three CTAs an SM; two where a stage's scales
    // take 8 bytes a row, 4 bits in groups of 32 or 2 bits in groups of 64, or a row has 54 groups or more: the last third of
    // the grid then follows the first two).  With no
    // more items than CTAs that fit, four warps share an item: its latency counts, not the throughput (128 items, 16
    // experts of 4 bits: 13.6 against 16.4 us the layer; 512 items, 128 experts of 4 bits: 30.5 against 29.0; 1408 items,
    // of 8 bits: 48 against 41).  The same kernel takes rows whose scales do not fit a warp's block.
    const int64_t pairs = (int64_t)a.T * a.topk;
    const int64_t most = pairs < a.E + pairs / TB ? pairs : a.E + pairs / TB;
    const int64_t items = most * (a.N / 16), all = 148 * 3;
    cfg.blockDim = dim3(THREADS);
    if (items <= all || kg > UP_GROUPS || !a.gate.blk || !a.up.blk) {
        cfg.gridDim = dim3((unsigned)(items < all ? items : all));
        cfg.dynamicSmemBytes = smem_shared;
        e = cudaLaunchKernelEx(&cfg, gate_up_kernel<BITS, XT, G, true>, a);
    } else {
        const int64_t ctas = (items + WARPS - 1) / WARPS;
        cfg.gridDim = dim3((unsigned)(ctas < all ? ctas : all));
        cfg.dynamicSmemBytes = smem_own;
        e = cudaLaunchKernelEx(&cfg, gate_up_kernel<BITS, XT, G, false>, a);
    }
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)((a.K + ROWS - 1) / ROWS * a.cs));
    cfg.dynamicSmemBytes = smem_down;
    cfg.numAttrs = a.cs > 1 ? 2 : 1;
    if constexpr (std::is_same<XT, bf16_t>::value)
        if (a.parts == 1)
            return blk_down ? cudaLaunchKernelEx(&cfg, down_kernel<BITS, XT, G, true, 1>, a)
                            : cudaLaunchKernelEx(&cfg, down_kernel<BITS, XT, G, false, 1>, a);
    return blk_down ? cudaLaunchKernelEx(&cfg, down_kernel<BITS, XT, G, true, 2>, a)
                    : cudaLaunchKernelEx(&cfg, down_kernel<BITS, XT, G, false, 2>, a);
}

template <int BITS, typename XT>
cudaError_t launch_g(const Args& a, int group, cudaStream_t st) {
    switch (group) {
        case 32:
            if constexpr (BITS >= 4) return launch_t<BITS, XT, 32>(a, st);
            break;
        case 64: return launch_t<BITS, XT, 64>(a, st);
        case 128: return launch_t<BITS, XT, 128>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
}  // namespace aq
