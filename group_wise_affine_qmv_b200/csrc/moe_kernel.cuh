// moe_kernel.cuh -- a mixture-of-experts layer for a few tokens in two kernels.
//
//     e_1 .. e_k = the top-k of logits[t], w = their softmax weights
//     h[t, j]    = w_j silu(x[t] . Wg[e_j]^T) * (x[t] . Wu[e_j]^T)      (gate/up kernel)
//     y[t]       = r[t] + sum_j h[t, j] . Wd[e_j]^T                     (down kernel)
//
// Every weight that some token chose is read once; at a few dozen tokens that traffic is all that
// counts, so both kernels are built as streams of packed codes that never pause:
//  - The routing costs no launch: every CTA of both kernels computes the top-k of all tokens itself
//    (a few thousand logits from L2, a warp per token), and keeps per expert a 64-bit mask of its
//    tokens.  An entry of the work list is an expert with up to 16 of its tokens.
//  - A warp streams stages of 64 bytes x 32 weight rows through a ring in shared memory; the ring
//    runs on across items, so the next item's codes are in flight while one is finished.  The
//    warps of a CTA split K by stages (neighbouring warps read neighbouring 64 bytes).
//  - The arithmetic is that of the warp-level dense kernel: codes expanded in registers into
//    mma.sync A fragments (16 weight rows x 16 codes, 8 tokens per column tile), group sums of x
//    from an all-ones tile, s D + b X folded in fp32.  Tokens of an expert are few, so a column
//    tile is rarely full; it costs nothing, since the codes' expansion is what a stage takes.
//  - The activations h keep 16 bits of mantissa between the kernels, as two bf16 (hi + lo), which
//    the down kernel feeds as two MMAs: one 8-bit rounding there would cost as much accuracy as the
//    rounding of y itself.  Their group sums come from the gate/up kernel's epilogue (sums of 16).
//  - The down kernel computes its routing and stages its first weights while the gate/up kernel
//    still runs (it waits only for h).  A CTA owns 32 columns of y for all tokens and walks the
//    entries; a cluster of up to eight CTAs splits the entries and adds its tiles in rank order.
//    No atomics: nothing depends on timing.
#pragma once

#include <mutex>

#include "moe.h"
#include "warp_mma_kernel.cuh"

namespace aq {
namespace moe {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int TB = 16;                 // tokens of an entry: two n8 tiles
constexpr int NST = 5;                 // stages of a warp's ring
constexpr int ROWS = 32;               // weight rows of a stage
constexpr int STAGE = ROWS * 64;       // bytes
constexpr int RP = ROWS + 1;           // floats per token of a partial tile

template <int BITS, int G>
struct Geo {
    static constexpr int SC = 512 / BITS;                 // codes of a row per stage (64 bytes)
    static constexpr int KS = G < 64 ? G : 64;            // codes per sub-block (warp_mma_kernel.cuh)
    static constexpr int SUBS = SC / KS;
    static constexpr int STEPS = KS / 16;
    static constexpr int LB = KS * BITS / 32;             // bytes of a row per lane and sub-block
    static constexpr int FU = G < SC ? G : SC;            // codes per fold: a group, or a stage's part of it
    static constexpr int SPF = FU / KS;
    static constexpr int GPS = SC / FU;                   // folds per stage
    static_assert(LB >= 4, "a lane's codes fill whole words");
};

// ---- routing ----

struct Routing {
    uint64_t mask[MAX_EXPERTS];              // tokens of each expert
    float weight[MAX_TOKENS * MAX_TOPK];     // per (token, choice)
    uint16_t sel[MAX_TOKENS * MAX_TOPK];     // the chosen expert, 0xffff: none
    uint16_t entry[MAX_TOKENS * MAX_TOPK];   // work list: expert | token block << 12
    int entries;
};

__device__ __forceinline__ uint32_t ordered(float v) {   // order-preserving; NaN above everything, -inf is 0: never chosen
    if (v != v) return 0xffffffffu;
    if (v == -INFINITY) return 0u;
    v += 0.0f;                                           // -0 and 0 tie
    const uint32_t u = __float_as_uint(v);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int EPL>
__device__ __forceinline__ void route_tokens(const Args& a, Routing& R, int warp, int lane) {
    for (int t = warp; t < a.T; t += WARPS) {
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
            R.weight[t * a.topk + lane] = p / sum;
        }
    }
}

// Top-k, weights, masks and the work list, by the whole CTA.
__device__ __forceinline__ void route(const Args& a, Routing& R, int warp, int lane) {
    for (int e = threadIdx.x; e < a.E; e += THREADS) R.mask[e] = 0;
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
}

// The tokens of an entry in a warp's own list: pair[i] = token * topk + choice.  Returns how many.
__device__ __forceinline__ int entry_pairs(const Args& a, const Routing& R, int entry, uint16_t* pair, int lane) {
    const int e = entry & 0xfff, first = (entry >> 12) * TB;
    const uint64_t m = R.mask[e];
    __syncwarp();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int t = lane + 32 * half;
        if ((m >> t) & 1) {
            const int rank = __popcll(m & ((1ull << t) - 1)) - first;
            if (rank >= 0 && rank < TB) {
                int j = 0;
                while (j + 1 < a.topk && R.sel[t * a.topk + j] != e) ++j;
                pair[rank] = (uint16_t)(t * a.topk + j);
            }
        }
    }
    __syncwarp();
    const int n = __popcll(m) - first;
    return n < TB ? n : TB;
}

// ---- streams of packed codes ----

__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, bool live) {   // zeros where not live
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ int swz(int row) { return ((row >> 1) & 1) << 1; }   // spreads 32-byte reads over the banks

// one lane's codes of sub-block sb of a stage's row
template <int LB>
__device__ __forceinline__ void lane_words(const uint8_t* stage, int row, int sb, int c, uint32_t* w) {
    const int off = sb * 4 * LB + c * LB;
    wm::load_lane_words<LB>(stage + row * 64 + (((off >> 4) ^ swz(row)) << 4) + (off & 15), w);
}

// A stage's scales or biases of one row: GPS halves from element `off`.
template <int GPS>
__device__ __forceinline__ void load_sb(const uint16_t* p, int g0, int kg, bool vec, uint16_t (&v)[GPS]) {
    if constexpr (GPS == 4) {
        if (vec) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(p + g0));
            v[0] = (uint16_t)u.x; v[1] = (uint16_t)(u.x >> 16); v[2] = (uint16_t)u.y; v[3] = (uint16_t)(u.y >> 16);
            return;
        }
    }
    if constexpr (GPS == 2) {
        if (vec) {
            const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(p + g0));
            v[0] = (uint16_t)u; v[1] = (uint16_t)(u >> 16);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < GPS; ++i) v[i] = __ldg(p + min(g0 + i, kg - 1));
}

// ---- gate/up ----

template <int BITS, typename XT, int G>
__global__ void __launch_bounds__(THREADS, 4) gate_up_kernel(const __grid_constant__ Args a) {
    using Gm = Geo<BITS, G>;
    constexpr bool BF = std::is_same<XT, bf16_t>::value;
    constexpr float OFF = (BF && BITS < 8) ? 128.0f : 0.0f;
    constexpr int GPS = Gm::GPS;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* rings = smem;
    float* red = reinterpret_cast<float*>(smem + WARPS * NST * STAGE);          // [2][WARPS][TB][RP]
    float* sqs = red + 2 * WARPS * TB * RP;                                     // [2][WARPS][TB]
    Routing& R = *reinterpret_cast<Routing*>(sqs + 2 * WARPS * TB);
    __shared__ uint16_t pairs[WARPS][TB];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;

    ptx::pdl_wait();                 // x and the logits may come from the kernel before
    ptx::pdl_launch_dependents();    // after the wait: the down kernel reads the logits before its own
    route(a, R, warp, lane);

    const int nb_all = a.N / 16;
    const int items = R.entries * nb_all;
    const int kg = a.K / G;
    const int nst = (a.K + Gm::SC - 1) / Gm::SC;
    const int nsw = (nst - warp + WARPS - 1) / WARPS;        // stages of this warp per item
    const int row_bytes = a.K * BITS / 8;
    uint8_t* ring = rings + warp * NST * STAGE;
    const uint32_t ring_s = ptx::smem_u32(ring);

    // load cursor: item and stage of the next load
    int l_item = blockIdx.x, l_s = 0, l_slot = 0;
    auto issue = [&]() {
        if (l_item < items && nsw > 0) {
            const int ent = R.entry[l_item / nb_all], e = ent & 0xfff, n0 = (l_item % nb_all) * 16;
            const int off = (warp + l_s * WARPS) * 64;
            const uint8_t* gp = reinterpret_cast<const uint8_t*>(a.gate.wq + e * a.gate.w_exp);
            const uint8_t* up = reinterpret_cast<const uint8_t*>(a.up.wq + e * a.up.w_exp);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (lane >> 2) + 8 * i, ch = lane & 3;
                const int n = n0 + (row & 15);
                const uint8_t* src = (row < 16 ? gp + n * a.gate.w_row * 4 : up + n * a.up.w_row * 4) + off + ch * 16;
                const bool live = off + ch * 16 < row_bytes;
                cp16z(ring_s + l_slot * STAGE + row * 64 + ((ch ^ swz(row)) << 4), live ? src : gp, live);
            }
            if (l_s == 0) {      // the scales and biases of the item's rows on their way to L2
                const int64_t so = (int64_t)(n0 + (lane & 15)) * kg;
                ptx::prefetch_l2(lane < 16 ? a.gate.scales + e * a.gate.s_exp + so : a.up.scales + e * a.up.s_exp + so);
                ptx::prefetch_l2(lane < 16 ? a.gate.biases + e * a.gate.b_exp + so : a.up.biases + e * a.up.b_exp + so);
            }
            if (++l_s == nsw) {
                l_s = 0;
                l_item += gridDim.x;
            }
            if (++l_slot == NST) l_slot = 0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) issue();

    int slot = 0, buf = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x, buf ^= 1) {
        const int ent = R.entry[item / nb_all], e = ent & 0xfff, nb = item % nb_all, n0 = nb * 16;
        const int nt = entry_pairs(a, R, ent, pairs[warp], lane);
        const bool two = nt > 8;
        // this lane's x rows (token r of each tile; past the last one: the last one)
        const uint16_t* xr[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int p = pairs[warp][min(8 * t + r, nt - 1)];
            xr[t] = a.x + (p / a.topk) * a.x_row + c * (Gm::KS / 4);
        }
        // rows r and r + 8 of gate (0, 1) and up (2, 3)
        const uint16_t *sp[4], *bp[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Bank& B = i < 2 ? a.gate : a.up;
            const int64_t ro = (int64_t)(n0 + r + 8 * (i & 1)) * kg;
            sp[i] = B.scales + e * B.s_exp + ro;
            bp[i] = B.biases + e * B.b_exp + ro;
        }
        float acc[2][2][4], sq[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[m][t][q] = 0.0f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) sq[t][q] = 0.0f;
        const uint32_t ONES = BF ? 0x3F803F80u : 0x3C003C00u;

#pragma unroll 1
        for (int s = 0; s < nsw; ++s) {
            const int st = warp + s * WARPS;
            uint16_t sv[4][GPS], bv[4][GPS];
            const int g0 = st * Gm::SC / G;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                load_sb<GPS>(sp[i], g0, kg, a.gate.svec, sv[i]);
                load_sb<GPS>(bp[i], g0, kg, a.gate.svec, bv[i]);
            }
            constexpr int XV = Gm::KS / 32;          // 16-byte pieces of x per lane, tile and sub-block
            uint4 xv[2][Gm::SUBS * XV];
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (t == 0 || two)
#pragma unroll
                    for (int sb = 0; sb < Gm::SUBS; ++sb) {
                        const int k0 = st * Gm::SC + sb * Gm::KS;
#pragma unroll
                        for (int v = 0; v < XV; ++v)
                            xv[t][sb * XV + v] = k0 < a.K ? __ldcg(reinterpret_cast<const uint4*>(xr[t] + k0) + v) : make_uint4(0, 0, 0, 0);
                    }
            issue();
            asm volatile("cp.async.wait_group %0;" ::"n"(NST - 1) : "memory");
            __syncwarp();
            const uint8_t* stage = ring + slot * STAGE;
            float d[2][2][4], xs[2][4];
#pragma unroll
            for (int sb = 0; sb < Gm::SUBS; ++sb) {
                if (sb % Gm::SPF == 0)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int q = 0; q < 4; ++q) d[0][t][q] = d[1][t][q] = xs[t][q] = 0.0f;
                uint32_t fr[4][Gm::STEPS][2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[Gm::LB / 4];
                    lane_words<Gm::LB>(stage, r + 8 * i, sb, c, w);
                    wm::expand_row<BITS, BF, Gm::STEPS>(w, fr[i]);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (t == 0 || two) {
                        const uint32_t* xw = reinterpret_cast<const uint32_t*>(&xv[t][sb * XV]);
#pragma unroll
                        for (int k = 0; k < Gm::STEPS; ++k) {
#pragma unroll
                            for (int m = 0; m < 2; ++m)
                                wm::mma16816<BF>(d[m][t], fr[2 * m][k][0], fr[2 * m + 1][k][0], fr[2 * m][k][1], fr[2 * m + 1][k][1],
                                                 xw[2 * k], xw[2 * k + 1]);
                            wm::mma16816<BF>(xs[t], ONES, ONES, ONES, ONES, xw[2 * k], xw[2 * k + 1]);
                            if (a.rms_eps > 0.0f)
                                wm::mma16816<BF>(sq[t], xw[2 * k], xw[2 * k], xw[2 * k + 1], xw[2 * k + 1], xw[2 * k], xw[2 * k + 1]);
                        }
                    }
                if (sb % Gm::SPF == Gm::SPF - 1) {
                    const int f = sb / Gm::SPF;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = i >> 1, h = i & 1;
                        const float ss = half_bits_to_float(sv[i][f], XT{});
                        float bb = half_bits_to_float(bv[i][f], XT{});
                        if (OFF != 0.0f) bb = fmaf(-OFF, ss, bb);
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                acc[m][t][2 * h + q] = fmaf(ss, d[m][t][2 * h + q], fmaf(bb, xs[t][q], acc[m][t][2 * h + q]));
                    }
                }
            }
            __syncwarp();
            if (++slot == NST) slot = 0;
        }
        // ---- the warps' slices of K together; silu(gate) * up * weight ----
        float* rw = red + (buf * WARPS + warp) * TB * RP;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int tok = 8 * t + 2 * c + q;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) rw[tok * RP + 16 * m + 8 * h + r] = acc[m][t][2 * h + q];
            }
        if (c == (r >> 1))
#pragma unroll
            for (int t = 0; t < 2; ++t) sqs[(buf * WARPS + warp) * TB + 8 * t + r] = (r & 1) ? sq[t][1] : sq[t][0];
        __syncthreads();
        for (int i = threadIdx.x; i < TB * 16; i += THREADS) {
            const int tok = i >> 4, col = i & 15;
            float g = 0.0f, u = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float* q = red + (buf * WARPS + w) * TB * RP + tok * RP;
                g += q[col];
                u += q[16 + col];
                s2 += sqs[(buf * WARPS + w) * TB + tok];
            }
            float hv = 0.0f;
            const bool live = tok < nt;
            const int p = pairs[warp][live ? tok : 0];
            if (a.rms_eps > 0.0f) {
                const float sc = rsqrtf(s2 / (float)a.K + a.rms_eps);
                g *= sc;
                u *= sc;
            }
            const float v = wm::silu(g) * u * R.weight[p];
            const uint16_t hi = float_to_half_bits(v, bf16_t{});
            const float hf = half_bits_to_float(hi, bf16_t{});
            // an infinite activation has no remainder
            const uint16_t lo = isfinite(v) && isfinite(hf) ? float_to_half_bits(v - hf, bf16_t{}) : 0;
            hv = hf + half_bits_to_float(lo, bf16_t{});
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) hv += __shfl_xor_sync(0xffffffffu, hv, o);
            if (live) {
                a.h_hi[(int64_t)p * a.N + n0 + col] = hi;
                a.h_lo[(int64_t)p * a.N + n0 + col] = lo;
                if (col == 0) a.h_sum[(int64_t)p * nb_all + nb] = hv;
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---- down ----

template <int BITS, typename XT, int G>
__global__ void __launch_bounds__(THREADS, 4) down_kernel(const __grid_constant__ Args a) {
    using Gm = Geo<BITS, G>;
    constexpr float OFF = BITS < 8 ? 128.0f : 0.0f;      // h is bf16 whatever x's type
    constexpr int GPS = Gm::GPS;
    extern __shared__ __align__(128) uint8_t smem[];
    float* yt = reinterpret_cast<float*>(smem + WARPS * NST * STAGE);           // [WARPS][T][RP]
    Routing& R = *reinterpret_cast<Routing*>(yt + ((WARPS * a.T * RP + 3) & ~3));
    __shared__ uint16_t pairs[WARPS][TB];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;
    const int cs = a.cs;
    const int rank = cs > 1 ? (int)ptx::cluster_ctarank() : 0;
    const int row0 = (int)(blockIdx.x / cs) * ROWS;      // first column of y

    route(a, R, warp, lane);     // the logits are complete: the gate/up kernel waited for them before this one started
    for (int i = threadIdx.x; i < WARPS * a.T * RP; i += THREADS) yt[i] = 0.0f;

    const int kg = a.N / G;
    const int nst = (a.N + Gm::SC - 1) / Gm::SC;
    const int nsw = (nst - warp + WARPS - 1) / WARPS;
    const int row_bytes = a.N * BITS / 8;
    uint8_t* ring = smem + warp * NST * STAGE;
    const uint32_t ring_s = ptx::smem_u32(ring);

    int l_ent = rank, l_s = 0, l_slot = 0;
    auto issue = [&]() {
        if (l_ent < R.entries && nsw > 0) {
            const int e = R.entry[l_ent] & 0xfff;
            const int off = (warp + l_s * WARPS) * 64;
            const uint8_t* wp = reinterpret_cast<const uint8_t*>(a.down.wq + e * a.down.w_exp);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (lane >> 2) + 8 * i, ch = lane & 3;
                const int n = min(row0 + row, a.K - 1);
                const bool live = off + ch * 16 < row_bytes;
                cp16z(ring_s + l_slot * STAGE + row * 64 + ((ch ^ swz(row)) << 4), live ? wp + n * a.down.w_row * 4 + off + ch * 16 : wp, live);
            }
            if (l_s == 0) {
                const int64_t so = (int64_t)min(row0 + lane, a.K - 1) * kg;
                ptx::prefetch_l2(a.down.scales + e * a.down.s_exp + so);
                ptx::prefetch_l2(a.down.biases + e * a.down.b_exp + so);
            }
            if (++l_s == nsw) {
                l_s = 0;
                l_ent += cs;
            }
            if (++l_slot == NST) l_slot = 0;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) issue();
    __syncthreads();             // the y tiles are zero

    ptx::pdl_wait();             // h
    ptx::pdl_launch_dependents();

    int slot = 0;
    float* yw = yt + warp * a.T * RP;
    for (int ent = rank; ent < R.entries; ent += cs) {
        const int en = R.entry[ent], e = en & 0xfff;
        const int nt = entry_pairs(a, R, en, pairs[warp], lane);
        const bool two = nt > 8;
        const uint16_t *hr[2], *lr[2];
        const float* xsum[2][2];                         // sums of tokens 2c and 2c + 1 of each tile
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int64_t o = (int64_t)pairs[warp][min(8 * t + r, nt - 1)] * a.N + c * (Gm::KS / 4);
            hr[t] = a.h_hi + o;
            lr[t] = a.h_lo + o;
#pragma unroll
            for (int q = 0; q < 2; ++q) xsum[t][q] = a.h_sum + (int64_t)pairs[warp][min(8 * t + 2 * c + q, nt - 1)] * (a.N / 16);
        }
        const uint16_t *sp[4], *bp[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t ro = (int64_t)min(row0 + r + 8 * i, a.K - 1) * kg;
            sp[i] = a.down.scales + e * a.down.s_exp + ro;
            bp[i] = a.down.biases + e * a.down.b_exp + ro;
        }
        float acc[2][2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[m][t][q] = 0.0f;

#pragma unroll 1
        for (int s = 0; s < nsw; ++s) {
            const int st = warp + s * WARPS;
            uint16_t sv[4][GPS], bv[4][GPS];
            const int g0 = st * Gm::SC / G;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                load_sb<GPS>(sp[i], g0, kg, a.down.svec, sv[i]);
                load_sb<GPS>(bp[i], g0, kg, a.down.svec, bv[i]);
            }
            issue();
            asm volatile("cp.async.wait_group %0;" ::"n"(NST - 1) : "memory");
            __syncwarp();
            const uint8_t* stage = ring + slot * STAGE;
            float d[2][2][4];
#pragma unroll
            for (int sb = 0; sb < Gm::SUBS; ++sb) {
                const int k0 = st * Gm::SC + sb * Gm::KS;
                if (k0 >= a.N) break;
                if (sb % Gm::SPF == 0)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int q = 0; q < 4; ++q) d[0][t][q] = d[1][t][q] = 0.0f;
                uint32_t fr[4][Gm::STEPS][2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[Gm::LB / 4];
                    lane_words<Gm::LB>(stage, r + 8 * i, sb, c, w);
                    wm::expand_row<BITS, true, Gm::STEPS>(w, fr[i]);
                }
                constexpr int XV = Gm::KS / 32;
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (t == 0 || two) {
                        uint4 hv[XV], lv[XV];
#pragma unroll
                        for (int v = 0; v < XV; ++v) {
                            hv[v] = __ldcg(reinterpret_cast<const uint4*>(hr[t] + k0) + v);
                            lv[v] = __ldcg(reinterpret_cast<const uint4*>(lr[t] + k0) + v);
                        }
                        const uint32_t *hw = reinterpret_cast<const uint32_t*>(hv), *lw = reinterpret_cast<const uint32_t*>(lv);
#pragma unroll
                        for (int k = 0; k < Gm::STEPS; ++k)
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                wm::mma16816<true>(d[m][t], fr[2 * m][k][0], fr[2 * m + 1][k][0], fr[2 * m][k][1], fr[2 * m + 1][k][1],
                                                   hw[2 * k], hw[2 * k + 1]);
                                wm::mma16816<true>(d[m][t], fr[2 * m][k][0], fr[2 * m + 1][k][0], fr[2 * m][k][1], fr[2 * m + 1][k][1],
                                                   lw[2 * k], lw[2 * k + 1]);
                            }
                    }
                if (sb % Gm::SPF == Gm::SPF - 1) {
                    const int f = sb / Gm::SPF;
                    const int x0 = (st * Gm::SC + f * Gm::FU) / 16;
                    float X[2][2];
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            X[t][q] = 0.0f;
                            if (t == 0 || two)
#pragma unroll
                                for (int i = 0; i < Gm::FU / 16; i += 2) {
                                    X[t][q] += __ldcg(xsum[t][q] + x0 + i);
                                    X[t][q] += __ldcg(xsum[t][q] + x0 + i + 1);
                                }
                        }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = i >> 1, h = i & 1;
                        const float ss = half_bits_to_float(sv[i][f], XT{});
                        float bb = half_bits_to_float(bv[i][f], XT{});
                        if (OFF != 0.0f) bb = fmaf(-OFF, ss, bb);
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                acc[m][t][2 * h + q] = fmaf(ss, d[m][t][2 * h + q], fmaf(bb, X[t][q], acc[m][t][2 * h + q]));
                    }
                }
            }
            __syncwarp();
            if (++slot == NST) slot = 0;
        }
        // this warp's slice of K into its own tile of y
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int i = 8 * t + 2 * c + q;
                if (i < nt) {
                    float* yp = yw + (pairs[warp][i] / a.topk) * RP;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) yp[16 * m + 8 * h + r] += acc[m][t][2 * h + q];
                }
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
cudaError_t launch_t(const Args& a, cudaStream_t st) {
    const size_t ring = (size_t)WARPS * NST * STAGE;
    const size_t smem1 = ring + (2 * WARPS * TB * RP + 2 * WARPS * TB) * sizeof(float) + sizeof(Routing);
    const size_t smem2 = ring + ((WARPS * a.T * RP + 3) & ~3) * sizeof(float) + sizeof(Routing);
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
            e = cudaFuncSetAttribute(gate_up_kernel<BITS, XT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
            if (e != cudaSuccess) return e;
            e = cudaFuncSetAttribute(down_kernel<BITS, XT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
            if (e != cudaSuccess) return e;
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
    // as many items as the tokens could choose, at most what fits the device at once
    const int64_t pairs = (int64_t)a.T * a.topk;
    const int64_t most = pairs < a.E + pairs / TB ? pairs : a.E + pairs / TB;
    const int64_t items = most * (a.N / 16);
    cfg.gridDim = dim3((unsigned)(items < 148 * 4 ? items : 148 * 4));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem1;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gate_up_kernel<BITS, XT, G>, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)((a.K + ROWS - 1) / ROWS * a.cs));
    cfg.dynamicSmemBytes = smem2;
    cfg.numAttrs = a.cs > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, down_kernel<BITS, XT, G>, a);
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
