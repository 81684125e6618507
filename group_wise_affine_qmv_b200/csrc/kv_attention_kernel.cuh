// kv_attention_kernel.cuh -- attention of a few query tokens over a paged cache of 4-bit keys and
// values (instantiated per head size in kernels_kv_attention_d{64,128,256}.cu).
//
//     out[i, h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q . k_j - max)
//     k_j[d] = s q4 + b  =>  q . k_j = sum_g  s[j,g] D[j,g] + b[j,g] X[g],
//                            D = sum_{d in g} q_d code_d,  X = sum_{d in g} q_d
//     v_j likewise       =>  sum_j p_j v_j[d] = sum_j (p_j s[j,g]) code_jd + sum_j p_j b[j,g]
//
// so the codes go to the tensor cores as exact small integers and scales and biases stay fp32.
//
// What bounds it: a cached token costs D/2 + 4 D/G bytes per head and side, and every code has to
// be widened once; at the full HBM rate that leaves about three instructions per code and lane, so
// the kernel is built around few instructions per code:
//  - Everything is transposed (S^T = K q^T, O^T = V^T P^T): the 16 rows of mma.sync.m16n8k16 hold
//    tokens (then V's dims), its 8 columns the query rows of one key/value head.  A tile of 16
//    tokens x 16 dims is one MMA whatever the number of query heads, up to 8.
//  - f16 operands whatever q's type: a code widens with one AND-OR into the mantissa of 1024 (low
//    nibble of a half) or 64 (high nibble), two codes at a time, without shifting each nibble into
//    place.  For the keys the offsets stay in and leave with the group's fold (O = 1024 sum of even
//    q + 64 sum of odd q; the fp32 cancellation costs 2^-24 * 1024 / 15 of |s q|, far below the
//    rounding of p).  For the values they are subtracted (exact): those sums run over the whole
//    context.  q is scaled by a power of two per row (its largest value near 2^12), so bf16 queries
//    lose nothing as f16.
//  - The order of dims inside an MMA is free as long as both operands agree; lanes read whole
//    words, and q is stored permuted (0,4,1,5,2,6,3,7 within a word).
//  - V^T needs pairs of tokens in one register: one PRMT per pair of words and half.
//  - Running maximum: a warp keeps a reference per query row and rescales only when a score exceeds
//    it by more than 8 (in log2), decided by one vote per 16 tokens: p <= 2^8 instead of 1, and no
//    shuffles on the usual path.  Sums and the bias term stay per lane until the end.
//  - p s is rounded to f16 (11 bits, against the output's 8 or 11); s varies over tokens and may
//    lie anywhere in its 16-bit type's range, so p s is scaled by a power of two per group that
//    follows the largest |s| seen (the same vote), which keeps p s below 2^15 and exact to 11 bits
//    down to 2^-29 of that.
//
// Work split.  A unit is 64 consecutive tokens of one (sequence, key/value head, row tile), 16 per
// warp; warps keep their own softmax state and meet only at the end of an item.  All units of all
// items form one line, and every CTA takes an equal stretch of it, so ragged batches and single
// long sequences load the SMs alike.  A stretch that ends inside an item leaves a partial result
// (at most two per CTA), which the combine kernel adds in CTA order; nothing depends on timing.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>

#include "device_common.cuh"
#include "kv_cache.h"
#include "sm100_ptx.cuh"

namespace aq {
namespace kv {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int TILE = 16;              // tokens per warp and unit
constexpr int UNIT = TILE * WARPS;

// f16 pairs from the nibbles of a word's halves
__device__ __forceinline__ uint32_t nib_lo(uint32_t w) { return (w & 0x000F000Fu) | 0x64006400u; }   // 1024 + n
__device__ __forceinline__ uint32_t nib_hi(uint32_t w) { return (w & 0x00F000F0u) | 0x54005400u; }   // 64 + n
__device__ __forceinline__ uint32_t hsub2u(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t code_lo(uint32_t w) { return hsub2u(nib_lo(w), 0x64006400u); }
__device__ __forceinline__ uint32_t code_hi(uint32_t w) { return hsub2u(nib_hi(w), 0x54005400u); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {   // an 8 x 8 block of 16-bit values across the warp
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ float2 half_pair(uint32_t v, bf16_t) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 half_pair(uint32_t v, f16_t) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// ---- the line of units ----

// The cached tokens [first, end) that some query of a sequence sees; first on a tile boundary.
struct Span {
    int64_t len, first;
    int64_t units;
};
__device__ __forceinline__ Span seq_span(const AttnArgs& a, int b) {
    Span s;
    int64_t n = __ldcg(a.lengths + b);
    const int64_t most = a.max_pages * a.S;
    if (n < 0 || n > most) {
        atomicOr(a.err, DEVERR_INDEX);
        n = n < 0 ? 0 : most;
    }
    s.len = n;
    int64_t f = 0;
    if (a.window > 0) {
        f = n - a.Tq - a.window + 1;
        f = f < 0 ? 0 : f & ~(int64_t)(TILE - 1);
    }
    s.first = f;
    s.units = (n - f + UNIT - 1) / UNIT;
    return s;
}

__device__ __forceinline__ int64_t warp_incl_scan(int64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Units of all sequences, and (second pass) the sequence that holds unit `at` with the units before
// that sequence.  One warp.  Units count a sequence's items (heads x row tiles) too.
__device__ __forceinline__ int64_t total_units(const AttnArgs& a, int lane) {
    int64_t n = 0;
    for (int b = lane; b < a.B; b += 32) n += seq_span(a, b).units;
    n *= (int64_t)a.Hkv * a.rtiles;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n;
}
__device__ __forceinline__ void find_seq(const AttnArgs& a, int lane, int64_t at, int* seq, int64_t* before) {
    const int64_t items = (int64_t)a.Hkv * a.rtiles;
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        const int64_t u = b < a.B ? seq_span(a, b).units * items : 0;
        const int64_t incl = warp_incl_scan(u, lane) + base;
        const unsigned hit = __ballot_sync(0xffffffffu, incl > at);
        if (hit) {
            const int l = __ffs(hit) - 1;
            *seq = b0 + l;
            *before = __shfl_sync(0xffffffffu, incl - u, l);
            return;
        }
        base = __shfl_sync(0xffffffffu, incl, 31);
    }
    *seq = a.B;
    *before = base;
}
// CTA i of n takes units [i W / n, (i + 1) W / n)
__device__ __forceinline__ int64_t cut(int64_t W, int64_t n, int64_t i) { return W / n * i + W % n * i / n; }
// CTAs that share W units: no more than units
__device__ __forceinline__ int64_t sharing(int64_t W, int64_t grid) { return W < grid ? (W < 1 ? 1 : W) : grid; }

template <int D, int G, int NT>
struct Geo {
    static constexpr int KG = D / G;                       // groups per row
    static constexpr int ROWB = D / 2;                     // bytes of a row of codes
    static constexpr int CH = ROWB / 16;                   // its 16-byte pieces
    static constexpr int CODES = TILE * ROWB;              // a tile of one side
    static constexpr int SB = TILE * KG * 2;               // its scales, or its biases
    static constexpr int STAGE = 2 * CODES + 4 * SB;
    static constexpr int NST = D == 256 ? 3 : 4;           // stages of a warp's ring
    static constexpr int ROWS = 8 * NT;
    static constexpr int QP = D * 2 + 16;                  // bytes of a q row in shared memory
    static constexpr int RING = WARPS * NST * STAGE;
    static constexpr int MERGE = WARPS * ROWS * (D + 4) * 4;   // partial outputs of the warps (over the ring)
    static constexpr int BODY = RING > MERGE ? RING : MERGE;
    static constexpr int SMEM = BODY + ROWS * QP + KG * ROWS * 8 + ROWS * 4 + 64;
    // positions of a side's rows in a tile: 16-byte pieces are swizzled by position so that the eight
    // lanes of a shared-memory phase meet different banks
    static __device__ __forceinline__ int swz(int pos) {
        return D == 256 ? (pos & 3) << 1 : D == 128 ? ((pos >> 1) & 1) << 1 : 0;
    }
    // token t of a value tile: even tokens of an octet first, then odd ones
    static __device__ __forceinline__ int vpos(int t) { return (t & 8) | ((t & 1) << 2) | ((t >> 1) & 3); }
};

template <int D, int G, int NT, typename XT>
__global__ void __launch_bounds__(THREADS, (D == 256 || NT == 4) ? 2 : NT == 2 ? 3 : 4)
attention_kernel(const __grid_constant__ AttnArgs a) {
    using Gm = Geo<D, G, NT>;
    constexpr int KG = Gm::KG, ROWS = Gm::ROWS, NST = Gm::NST;
    constexpr int KS = G < 64 ? G : 64;        // dims per sub-block
    constexpr int SUBS = D / KS;
    constexpr int MT = D / 16;                 // m tiles of the output
    constexpr bool QREG = NT == 1 && D <= 128; // q fragments in registers

    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* qs = smem + Gm::BODY;                                        // [ROWS][QP] f16, permuted
    float2* xo = reinterpret_cast<float2*>(qs + ROWS * Gm::QP);           // [KG][ROWS] (X, O)
    float* csc = reinterpret_cast<float*>(xo + KG * ROWS);                // [ROWS] score scale
    volatile int64_t* sched = reinterpret_cast<volatile int64_t*>(reinterpret_cast<uint8_t*>(csc) + ROWS * 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;

    ptx::pdl_launch_dependents();
    ptx::pdl_wait();   // q and the cache may come from the kernels before

    if (warp == 0) {
        int64_t lo = 0, hi = 0, before = 0;
        int seq = 0;
        if (a.split) {
            const int64_t W = total_units(a, lane);
            const int64_t n = sharing(W, gridDim.x);
            if ((int64_t)blockIdx.x < n) {
                lo = cut(W, n, blockIdx.x);
                hi = cut(W, n, (int64_t)blockIdx.x + 1);
            }
            if (lo < hi) find_seq(a, lane, lo, &seq, &before);
        } else {   // one item per CTA
            const int items = a.Hkv * a.rtiles;
            seq = blockIdx.x / items;
            const int64_t units = seq_span(a, seq).units;
            lo = (blockIdx.x - seq * items) * units;
            hi = lo + units;
        }
        if (lane == 0) {
            sched[0] = lo;
            sched[1] = hi;
            sched[2] = seq;
            sched[3] = before;
        }
    }
    // sequences without a visible token: their rows are zeros
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)
        if (seq_span(a, b).units == 0) {
            const int64_t n = (int64_t)a.Tq * a.Hq * D;
            for (int64_t i = threadIdx.x; i < n; i += THREADS) {
                const int64_t th = i / D, t = th / a.Hq;
                a.out[b * a.o_b + t * a.o_t + (th - t * a.Hq) * a.o_h + (i - th * D)] = 0;
            }
        }
    __syncthreads();
    int64_t at = sched[0];
    const int64_t at_end = sched[1];
    int seq = (int)sched[2];
    int64_t before = sched[3];
    bool first_seg = true;

    uint8_t* ring = smem + warp * NST * Gm::STAGE;
    const uint32_t ring_s = ptx::smem_u32(ring);

    while (at < at_end) {
        // ---- the segment: units [u0, u1) of item (seq, head, row tile) ----
        Span sp = seq_span(a, seq);
        const int64_t items = (int64_t)a.Hkv * a.rtiles;
        while (at >= before + sp.units * items) {
            before += sp.units * items;
            sp = seq_span(a, ++seq);
        }
        const int64_t it = (at - before) / sp.units;
        const int64_t u0 = at - before - it * sp.units;
        const int64_t u1 = u0 + (at_end - at) < sp.units ? u0 + (at_end - at) : sp.units;
        const int head = (int)(it / a.rtiles), rt = (int)(it - (int64_t)head * a.rtiles);
        const int row0 = rt * ROWS;
        at += u1 - u0;
        const int64_t* pages = a.pages + seq * a.pages_row;

        // ---- loads of a tile (16 tokens from t0) into ring slot st ----
        auto load_tile = [&](int64_t t0, int st) {
            const uint32_t dst = ring_s + st * Gm::STAGE;
            if (a.fast) {
                const int64_t pg = t0 / a.S;
                const int64_t sl = t0 - pg * a.S;
                const int64_t pid = __ldcg(pages + pg);
                if (pid < 0 || pid >= a.P) {   // no such page: its tokens take no part (zero scales)
                    if (lane == 0) atomicOr(a.err, DEVERR_INDEX);
                    return false;
                }
                const uint8_t* kp = reinterpret_cast<const uint8_t*>(a.k.wq + pid * a.k.w_page + head * a.k.w_head + sl * a.k.w_slot);
                const uint8_t* vp = reinterpret_cast<const uint8_t*>(a.v.wq + pid * a.v.w_page + head * a.v.w_head + sl * a.v.w_slot);
#pragma unroll
                for (int i = 0; i < TILE * Gm::CH / 32; ++i) {
                    const int x = lane + 32 * i, row = x / Gm::CH, ch = x % Gm::CH;
                    cp16(dst + row * Gm::ROWB + ((ch ^ Gm::swz(row)) << 4), kp + row * a.k.w_slot * 4 + ch * 16);
                    const int vp_ = Gm::vpos(row);
                    cp16(dst + Gm::CODES + vp_ * Gm::ROWB + ((ch ^ Gm::swz(vp_)) << 4), vp + row * a.v.w_slot * 4 + ch * 16);
                }
                // scales and biases: 16 tokens are one run of 2 KG pieces per array
#pragma unroll
                for (int i = 0; i < (8 * KG + 31) / 32; ++i) {
                    const int x = lane + 32 * i;
                    if (x < 8 * KG) {
                        const int arr = x / (2 * KG), ch = x % (2 * KG);
                        const Side& sd = arr < 2 ? a.k : a.v;
                        const uint16_t* p = (arr & 1) ? sd.biases + pid * sd.b_page + head * sd.b_head + sl * sd.b_slot
                                                      : sd.scales + pid * sd.s_page + head * sd.s_head + sl * sd.s_slot;
                        cp16(dst + 2 * Gm::CODES + arr * Gm::SB + ch * 16, p + ch * 8);
                    }
                }
                return true;
            }
            // any page size and strides: rows one by one, scales through registers
            bool ok = true;
            for (int x = lane; x < TILE * Gm::CH; x += 32) {
                const int row = x / Gm::CH, ch = x % Gm::CH;
                const int64_t t = t0 + row;
                if (t >= sp.len) continue;
                const int64_t pg = t / a.S, sl = t - pg * a.S;
                const int64_t pid = __ldcg(pages + pg);
                if (pid < 0 || pid >= a.P) {
                    atomicOr(a.err, DEVERR_INDEX);
                    ok = false;
                    continue;
                }
                const uint8_t* kp = reinterpret_cast<const uint8_t*>(a.k.wq + pid * a.k.w_page + head * a.k.w_head + sl * a.k.w_slot);
                const uint8_t* vp = reinterpret_cast<const uint8_t*>(a.v.wq + pid * a.v.w_page + head * a.v.w_head + sl * a.v.w_slot);
                cp16(dst + row * Gm::ROWB + ((ch ^ Gm::swz(row)) << 4), kp + ch * 16);
                const int vp_ = Gm::vpos(row);
                cp16(dst + Gm::CODES + vp_ * Gm::ROWB + ((ch ^ Gm::swz(vp_)) << 4), vp + ch * 16);
            }
            uint16_t* sc = reinterpret_cast<uint16_t*>(ring + st * Gm::STAGE + 2 * Gm::CODES);
            for (int x = lane; x < TILE * KG; x += 32) {
                const int row = x / KG, g = x % KG;
                const int64_t t = t0 + row;
                uint16_t v4[4] = {0, 0, 0, 0};
                if (t < sp.len) {
                    const int64_t pg = t / a.S, sl = t - pg * a.S;
                    const int64_t pid = __ldcg(pages + pg);
                    if (pid >= 0 && pid < a.P) {
                        v4[0] = __ldcg(a.k.scales + pid * a.k.s_page + head * a.k.s_head + sl * a.k.s_slot + g);
                        v4[1] = __ldcg(a.k.biases + pid * a.k.b_page + head * a.k.b_head + sl * a.k.b_slot + g);
                        v4[2] = __ldcg(a.v.scales + pid * a.v.s_page + head * a.v.s_head + sl * a.v.s_slot + g);
                        v4[3] = __ldcg(a.v.biases + pid * a.v.b_page + head * a.v.b_head + sl * a.v.b_slot + g);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[k * TILE * KG + x] = v4[k];
            }
            return (bool)__all_sync(0xffffffffu, ok);
        };
        const int nu = (int)(u1 - u0);
        const int64_t tw = sp.first + u0 * UNIT + warp * TILE;     // this warp's tile of unit u0
        // tiles of this warp with a token below len
        int nt = 0;
        if (tw < sp.len) {
            const int64_t left = (sp.len - tw + UNIT - 1) / UNIT;
            nt = left < nu ? (int)left : nu;
        }
        unsigned bad = 0;   // ring slots whose page does not exist (uniform in the warp)
        auto issue = [&](int i) {
            const int st = i % NST;
            if (i < nt) {
                if (load_tile(tw + (int64_t)i * UNIT, st)) bad &= ~(1u << st);
                else bad |= 1u << st;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < NST - 1; ++i) issue(i);

        // ---- q rows of the item: scaled to f16, permuted, with their group sums ----
        for (int row = warp; row < ROWS; row += WARPS) {
            constexpr int EPL = D / 32;           // elements per lane
            const int rr = row0 + row;
            float f[EPL];
#pragma unroll
            for (int e = 0; e < EPL; ++e) f[e] = 0.0f;
            if (rr < a.rows) {
                const int i = rr / a.rep;
                const uint16_t* qp = a.q + seq * a.q_b + i * a.q_t + (head * a.rep + rr - i * a.rep) * (int64_t)a.q_h + lane * EPL;
#pragma unroll
                for (int e = 0; e < EPL; ++e) f[e] = half_bits_to_float(__ldcg(qp + e), XT{});
            }
            float am = 0.0f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) am = fmaxf(am, fabsf(f[e]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
            // 2^(12 - exponent of the largest value): exact products (an exponent of infinity stays in range)
            const int ex = min(max((int)((__float_as_uint(am) >> 23) & 255) - 127, -100), 127);
            const float up = __uint_as_float((uint32_t)(12 - ex + 127) << 23);
            float X = 0.0f, O = 0.0f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                const __half hf = __float2half_rn(f[e] * up);
                const float v = __half2float(hf);
                const int d = lane * EPL + e, n = d & 7;
                X += v;
                O += (n & 1) ? 64.0f * v : 1024.0f * v;
                // order within a word: 0 4 1 5 2 6 3 7
                const int pos = (d & ~7) + 2 * (n & 3) + (n >> 2);
                *reinterpret_cast<__half*>(qs + row * Gm::QP + pos * 2) = hf;
            }
            constexpr int GL = G / EPL;           // lanes per group
#pragma unroll
            for (int o = GL / 2; o > 0; o >>= 1) {
                X += __shfl_xor_sync(0xffffffffu, X, o);
                O += __shfl_xor_sync(0xffffffffu, O, o);
            }
            if (lane % GL == 0) xo[(lane / GL) * ROWS + row] = make_float2(X, O);
            if (lane == 0) csc[row] = a.scale_log2 * __uint_as_float((uint32_t)(ex - 12 + 127) << 23);
        }
        __syncthreads();

        uint32_t qf[QREG ? D / 8 : 1];            // [word of this lane][4]
        if constexpr (QREG) {
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const int word = KS == 64 ? (w >> 1) * 8 + 2 * c + (w & 1) : w * 4 + c;
                const uint4 v = *reinterpret_cast<const uint4*>(qs + r * Gm::QP + word * 16);
                qf[4 * w] = v.x; qf[4 * w + 1] = v.y; qf[4 * w + 2] = v.z; qf[4 * w + 3] = v.w;
            }
        }
        float cs[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            cs[n][0] = csc[8 * n + 2 * c];
            cs[n][1] = csc[8 * n + 2 * c + 1];
        }

        // ---- softmax state of this warp ----
        float mu[NT][2], thr[NT][2], l[NT][2], ab[KG][NT][2], vmul[KG], vthr[KG];
        float acc[MT][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mu[n][e] = 0.0f;
                thr[n][e] = -INFINITY;
                l[n][e] = 0.0f;
#pragma unroll
                for (int g = 0; g < KG; ++g) ab[g][n][e] = 0.0f;
            }
#pragma unroll
        for (int g = 0; g < KG; ++g) {
            vmul[g] = 1.0f;
            vthr[g] = -1.0f;
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][n][e] = 0.0f;

        const int64_t pos0 = sp.len - a.Tq;       // position of query token 0
        const int last_i = a.Tq - 1;

#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
            issue(i + NST - 1);
            cp_wait<NST - 1>();
            __syncwarp();
            const int st = i % NST;
            const uint8_t* kt = ring + st * Gm::STAGE;
            const uint8_t* vt = kt + Gm::CODES;
            const uint16_t* ssb = reinterpret_cast<const uint16_t*>(kt + 2 * Gm::CODES);
            const int64_t t0 = tw + (int64_t)i * UNIT;
            const bool slot_bad = (bad >> st) & 1u;
            // every token of the tile visible to every row?
            const bool full = !slot_bad && pos0 >= 0 && t0 + TILE - 1 <= pos0 &&
                              (a.window == 0 || t0 > pos0 + last_i - a.window);

            // ---- scores of tokens r and r + 8 for query rows 2c, 2c + 1 of each n tile ----
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
            float d[NT][4];
#pragma unroll
            for (int sb = 0; sb < SUBS; ++sb) {
                constexpr int SPG = G / KS;
                const int g = sb / SPG;
                if (sb % SPG == 0)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) d[n][e] = 0.0f;
                uint32_t w0[2], w1[2];            // rows r and r + 8
                if constexpr (KS == 64) {
                    const int ch = sb * 2 + (c >> 1), o = (c & 1) * 8;
                    const uint2 x = *reinterpret_cast<const uint2*>(kt + r * Gm::ROWB + ((ch ^ Gm::swz(r)) << 4) + o);
                    const uint2 y = *reinterpret_cast<const uint2*>(kt + (r + 8) * Gm::ROWB + ((ch ^ Gm::swz(r + 8)) << 4) + o);
                    w0[0] = x.x; w0[1] = x.y;
                    w1[0] = y.x; w1[1] = y.y;
                } else {
                    w0[0] = *reinterpret_cast<const uint32_t*>(kt + r * Gm::ROWB + ((sb ^ Gm::swz(r)) << 4) + c * 4);
                    w1[0] = *reinterpret_cast<const uint32_t*>(kt + (r + 8) * Gm::ROWB + ((sb ^ Gm::swz(r + 8)) << 4) + c * 4);
                }
#pragma unroll
                for (int j = 0; j < KS / 32; ++j) {
                    const int word = KS == 64 ? sb * 8 + 2 * c + j : sb * 4 + c;
                    const uint32_t u = w0[j], v = w1[j], us = u >> 8, vs = v >> 8;
                    const uint32_t e0 = nib_lo(u), e1 = nib_lo(v), e2 = nib_hi(u), e3 = nib_hi(v);
                    const uint32_t f0 = nib_lo(us), f1 = nib_lo(vs), f2 = nib_hi(us), f3 = nib_hi(vs);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint32_t b[4];
                        if constexpr (QREG) {
                            const int w = sb * (KS / 32) + j;
#pragma unroll
                            for (int k = 0; k < 4; ++k) b[k] = qf[4 * w + k];
                        } else {
                            const uint4 x = *reinterpret_cast<const uint4*>(qs + (8 * n + r) * Gm::QP + word * 16);
                            b[0] = x.x; b[1] = x.y; b[2] = x.z; b[3] = x.w;
                        }
                        mma_f16(d[n], e0, e1, e2, e3, b[0], b[1]);
                        mma_f16(d[n], f0, f1, f2, f3, b[2], b[3]);
                    }
                }
                if (sb % SPG == SPG - 1) {        // the group's fold: s (D - O) + b X
                    const float s0 = half_bits_to_float(ssb[r * KG + g], XT{});
                    const float s1 = half_bits_to_float(ssb[(r + 8) * KG + g], XT{});
                    const float b0 = half_bits_to_float(ssb[TILE * KG + r * KG + g], XT{});
                    const float b1 = half_bits_to_float(ssb[TILE * KG + (r + 8) * KG + g], XT{});
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float4 x = *reinterpret_cast<const float4*>(xo + g * ROWS + 8 * n + 2 * c);
                        s[n][0] += fmaf(s0, d[n][0] - x.y, b0 * x.x);
                        s[n][1] += fmaf(s0, d[n][1] - x.w, b0 * x.z);
                        s[n][2] += fmaf(s1, d[n][2] - x.y, b1 * x.x);
                        s[n][3] += fmaf(s1, d[n][3] - x.w, b1 * x.z);
                    }
                }
            }
            float sv[KG][2], bv[KG][2];           // value scales and biases of tokens r and r + 8
#pragma unroll
            for (int g = 0; g < KG; ++g) {
                sv[g][0] = half_bits_to_float(ssb[2 * TILE * KG + r * KG + g], XT{});
                sv[g][1] = half_bits_to_float(ssb[2 * TILE * KG + (r + 8) * KG + g], XT{});
                bv[g][0] = half_bits_to_float(ssb[3 * TILE * KG + r * KG + g], XT{});
                bv[g][1] = half_bits_to_float(ssb[3 * TILE * KG + (r + 8) * KG + g], XT{});
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] *= cs[n][e & 1];
            if (!full) {
                // rows see tokens up to their position, and from their window's start; a token that no
                // row sees (stale, another sequence's, of a missing page) may hold any scale: it is zeroed
                const int64_t ta = t0 + r, tb = ta + 8;
                const bool in[2] = {!slot_bad && ta < sp.len && ta >= 0, !slot_bad && tb < sp.len};
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = row0 + 8 * n + 2 * c + (e & 1);
                        int qi = row / a.rep;
                        if (qi > last_i) qi = last_i;
                        const int64_t pos = pos0 + qi, t = e < 2 ? ta : tb;
                        if (!(in[e >> 1] && t <= pos && (a.window == 0 || t > pos - a.window))) s[n][e] = -INFINITY;
                    }
                const int64_t seen_lo = a.window == 0 ? 0 : pos0 - a.window + 1;
#pragma unroll
                for (int g = 0; g < KG; ++g) {
                    if (!in[0] || ta < seen_lo) sv[g][0] = bv[g][0] = 0.0f;
                    if (!in[1] || tb < seen_lo) sv[g][1] = bv[g][1] = 0.0f;
                }
            }
            // ---- one vote: does a score or a value scale leave the range of the references? ----
            bool out_of = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) out_of |= s[n][e] > thr[n][e & 1];
#pragma unroll
            for (int g = 0; g < KG; ++g) out_of |= fmaxf(fabsf(sv[g][0]), fabsf(sv[g][1])) > vthr[g];
            if (__any_sync(0xffffffffu, out_of)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(s[n][e], s[n][e + 2]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        if (m > mu[n][e] || thr[n][e] == -INFINITY) {
                            if (m > -INFINITY) {
                                const float f = thr[n][e] == -INFINITY ? 0.0f : ex2(mu[n][e] - m);
                                mu[n][e] = m;
                                thr[n][e] = m + 8.0f;
                                l[n][e] *= f;
#pragma unroll
                                for (int g = 0; g < KG; ++g) ab[g][n][e] *= f;
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt) {
                                    acc[mt][n][e] *= f;
                                    acc[mt][n][e + 2] *= f;
                                }
                            }
                        }
                    }
#pragma unroll
                for (int g = 0; g < KG; ++g) {
                    // an infinite scale is no reference: it would flush the rows that do not see its token
                    float m = fmaxf(isinf(sv[g][0]) ? 0.0f : fabsf(sv[g][0]), isinf(sv[g][1]) ? 0.0f : fabsf(sv[g][1]));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    if (m > vthr[g]) {            // 2^E >= m: p s 2^(6 - E) <= 2^15 until the next change
                        const int E = min(max((int)((__float_as_uint(m) >> 23) & 255) - 126, -100), 127);
                        const float mul = __uint_as_float((uint32_t)(6 - E + 127) << 23);
                        const float f = vthr[g] < 0.0f ? 0.0f : mul / vmul[g];
                        vmul[g] = mul;
                        vthr[g] = E == 127 ? INFINITY : __uint_as_float((uint32_t)(E + 1 + 127) << 23);
#pragma unroll
                        for (int mt = 0; mt < MT / KG; ++mt)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[g * (MT / KG) + mt][n][e] *= f;
                    }
                }
            }
            // ---- p, its sums, and p s as f16 with tokens along k ----
            uint32_t pb[KG][NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = ex2(s[n][e] - mu[n][e & 1]);
                l[n][0] += p[0] + p[2];
                l[n][1] += p[1] + p[3];
#pragma unroll
                for (int g = 0; g < KG; ++g) {
                    float t[4] = {p[0] * (sv[g][0] * vmul[g]), p[1] * (sv[g][0] * vmul[g]),
                                  p[2] * (sv[g][1] * vmul[g]), p[3] * (sv[g][1] * vmul[g])};
                    if (full) {
                        ab[g][n][0] = fmaf(p[0], bv[g][0], fmaf(p[2], bv[g][1], ab[g][n][0]));
                        ab[g][n][1] = fmaf(p[1], bv[g][0], fmaf(p[3], bv[g][1], ab[g][n][1]));
                    } else {                      // a token that this row does not see may be infinite or NaN
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (s[n][e] == -INFINITY) t[e] = 0.0f;
                            else ab[g][n][e & 1] = fmaf(p[e], bv[g][e >> 1], ab[g][n][e & 1]);
                        }
                    }
                    const __half2 x = __floats2half2_rn(t[0], t[1]);
                    const __half2 y = __floats2half2_rn(t[2], t[3]);
                    pb[g][n][0] = transpose8(*reinterpret_cast<const uint32_t*>(&x));
                    pb[g][n][1] = transpose8(*reinterpret_cast<const uint32_t*>(&y));
                }
            }
            // ---- O^T += V^T (p s)^T ----
#pragma unroll
            for (int sb = 0; sb < SUBS; ++sb) {
                const int g = sb * KS / G;
                const int word = KS == 64 ? sb * 8 + r : sb * 4 + (r >> 1);
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {     // tokens 2c, 2c + 1, 2c + 8, 2c + 9
                    const int pos = (k >> 1) * 8 + (k & 1) * 4 + c;
                    w[k] = *reinterpret_cast<const uint32_t*>(vt + pos * Gm::ROWB + (((word >> 2) ^ Gm::swz(pos)) << 4) + (word & 3) * 4);
                }
                if constexpr (KS == 64) {
                    uint32_t xl = __byte_perm(w[0], w[1], 0x5410), xh = __byte_perm(w[0], w[1], 0x7632);
                    uint32_t yl = __byte_perm(w[2], w[3], 0x5410), yh = __byte_perm(w[2], w[3], 0x7632);
#pragma unroll
                    for (int j = 0; j < 2; ++j) { // nibbles 2j, 2j + 1 (rows r) and 2j + 4, 2j + 5 (rows r + 8)
                        const uint32_t a0 = code_lo(xl), a1 = code_lo(xh), a2 = code_lo(yl), a3 = code_lo(yh);
                        const uint32_t c0 = code_hi(xl), c1 = code_hi(xh), c2 = code_hi(yl), c3 = code_hi(yh);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_f16(acc[sb * 4 + 2 * j][n], a0, a1, a2, a3, pb[g][n][0], pb[g][n][1]);
                            mma_f16(acc[sb * 4 + 2 * j + 1][n], c0, c1, c2, c3, pb[g][n][0], pb[g][n][1]);
                        }
                        xl >>= 8; xh >>= 8; yl >>= 8; yh >>= 8;
                    }
                } else {
                    const uint32_t sel = (r & 1) ? 0x7632 : 0x5410;
                    uint32_t x = __byte_perm(w[0], w[1], sel), y = __byte_perm(w[2], w[3], sel);
#pragma unroll
                    for (int j = 0; j < 2; ++j) { // nibble 2j (rows r) and 2j + 1 (rows r + 8) of this lane's half word
                        const uint32_t a0 = code_lo(x), a1 = code_hi(x), a2 = code_lo(y), a3 = code_hi(y);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_f16(acc[sb * 2 + j][n], a0, a1, a2, a3, pb[g][n][0], pb[g][n][1]);
                        x >>= 8; y >>= 8;
                    }
                }
            }
            __syncwarp();   // every lane has read the slot before it is refilled
        }
        cp_wait<0>();
        __syncthreads();    // the ring becomes the merge buffer

        // ---- the warp's result: unnormalised outputs, reference and sum per query row ----
        float* mo = reinterpret_cast<float*>(smem) + warp * ROWS * (D + 4);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
#pragma unroll
                    for (int g = 0; g < KG; ++g) ab[g][n][e] += __shfl_xor_sync(0xffffffffu, ab[g][n][e], o);
                }
                const int row = 8 * n + 2 * c + e;
                if (r == 0) {
                    // nothing seen (a NaN sum is not nothing)
                    mo[row * (D + 4) + D] = thr[n][e] == -INFINITY && l[n][e] == 0.0f ? -INFINITY : mu[n][e];
                    mo[row * (D + 4) + D + 1] = l[n][e];
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int g = mt * 16 / G;
                    const float inv = 1.0f / vmul[g];   // a power of two: exact
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int dim = KS == 64 ? (mt >> 2) * 64 + 8 * r + (mt & 3) + 4 * h : (mt >> 1) * 32 + 4 * r + 2 * (mt & 1) + h;
                        mo[row * (D + 4) + dim] = fmaf(acc[mt][n][e + 2 * h], inv, ab[g][n][e]);
                    }
                }
            }
        __syncthreads();

        // ---- the warps' results together; a whole item is finished here, a part goes to the workspace ----
        const bool whole = u0 == 0 && u1 == sp.units;
        const int64_t pslot = 2 * (int64_t)blockIdx.x + (first_seg ? 0 : 1);
        for (int x = threadIdx.x; x < ROWS * (D / 4); x += THREADS) {
            const int row = x / (D / 4), d4 = (x % (D / 4)) * 4;
            const int rr = row0 + row;
            const float* base = reinterpret_cast<const float*>(smem) + row * (D + 4);
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) m = fmaxf(m, base[w * ROWS * (D + 4) + D]);
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float ls = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float* bw = base + w * ROWS * (D + 4);
                const float f = bw[D] == -INFINITY ? 0.0f : ex2(bw[D] - m);
                const float4 v = *reinterpret_cast<const float4*>(bw + d4);
                if (bw[D] != -INFINITY) {
                    o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y);
                    o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
                    ls = fmaf(f, bw[D + 1], ls);
                }
            }
            if (whole) {
                if (rr < a.rows) {
                    const int i = rr / a.rep;
                    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
                    uint16_t* op = a.out + seq * a.o_b + i * a.o_t + (head * a.rep + rr - i * a.rep) * (int64_t)a.o_h + d4;
                    const uint16_t h0 = float_to_half_bits(o.x * inv, XT{}), h1 = float_to_half_bits(o.y * inv, XT{});
                    const uint16_t h2 = float_to_half_bits(o.z * inv, XT{}), h3 = float_to_half_bits(o.w * inv, XT{});
                    if (a.ovec) {
                        *reinterpret_cast<uint2*>(op) = make_uint2(h0 | ((uint32_t)h1 << 16), h2 | ((uint32_t)h3 << 16));
                    } else {
                        op[0] = h0; op[1] = h1; op[2] = h2; op[3] = h3;
                    }
                }
            } else {
                *reinterpret_cast<float4*>(a.part_o + (pslot * ROWS + row) * D + d4) = o;
                if (d4 == 0) *reinterpret_cast<float2*>(a.part_ml + (pslot * ROWS + row) * 2) = make_float2(m, ls);
            }
        }
        __syncthreads();    // the merge buffer becomes the ring again, q is rewritten
        first_seg = false;
    }
}

// Joins the partial results of an item whose units several CTAs shared: the last segment of the CTA
// it starts in and the first segments of the CTAs after it, added in that order.  Block (x, row): the
// item x when there are fewer items than CTAs, else the item that starts in CTA x's stretch and
// reaches past it, if there is one.
template <int D, typename XT>
__global__ void __launch_bounds__(THREADS) combine_kernel(const __grid_constant__ AttnArgs a, int grid, int ROWS, int by_item) {
    __shared__ int64_t sched[6];
    __shared__ float red[WARPS][D + 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.y;
    ptx::pdl_launch_dependents();
    ptx::pdl_wait();
    if (warp == 0) {
        const int64_t W = total_units(a, lane);
        const int64_t n = sharing(W, grid);
        const int64_t items = (int64_t)a.Hkv * a.rtiles;
        int64_t first = -1, last = -1, slot = 0, it = 0, before = 0, units = 0, j = blockIdx.x;
        int seq = 0;
        if (by_item) {
            seq = (int)(blockIdx.x / items);
            it = blockIdx.x - seq * items;
            units = seq_span(a, seq).units;
            for (int b = lane; b < seq; b += 32) before += seq_span(a, b).units * items;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
            if (units > 0) {          // the CTA whose stretch holds the item's first unit
                const int64_t s0 = before + it * units;
                j = s0 * n / W;
                while (j > 0 && cut(W, n, j) > s0) --j;
                while (cut(W, n, j + 1) <= s0) ++j;
            }
        } else if (j < n - 1) {       // the item of CTA j's last unit
            const int64_t hi = cut(W, n, j + 1);
            find_seq(a, lane, hi - 1, &seq, &before);
            units = seq_span(a, seq).units;
            it = (hi - 1 - before) / units;
        }
        if (units > 0) {
            const int64_t lo = cut(W, n, j), hi = cut(W, n, j + 1);
            const int64_t s0 = before + it * units, s1 = s0 + units;
            if (s1 > hi && s0 >= lo) {
                first = j;
                slot = s0 > lo ? 1 : 0;               // not CTA j's first segment, unless the item starts its stretch
                last = j + 1;
                while (last + 1 < n && cut(W, n, last + 1) < s1) ++last;
            }
        }
        if (lane == 0) {
            sched[0] = first; sched[1] = last; sched[2] = slot; sched[3] = seq;
            sched[4] = it / a.rtiles;
            sched[5] = it % a.rtiles * ROWS + row;
        }
    }
    __syncthreads();
    const int64_t first = sched[0], last = sched[1];
    const int64_t rr = sched[5];
    if (first < 0 || rr >= a.rows) return;
    auto part = [&](int64_t k) { return (2 * (first + k) + (k == 0 ? sched[2] : 0)) * ROWS + row; };
    const int np = (int)(last - first + 1);
    float m = -INFINITY;
    for (int k = lane; k < np; k += 32) m = fmaxf(m, __ldcg(a.part_ml + part(k) * 2));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    constexpr int V = D / 32;
    float o[V], ls = 0.0f;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.0f;
#pragma unroll 4
    for (int k = warp; k < np; k += WARPS) {
        const int64_t p = part(k);
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + p * 2));
        float v[V];
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 u = __ldcg(reinterpret_cast<const float2*>(a.part_o + p * D + lane * V + e));
            v[e] = u.x;
            v[e + 1] = u.y;
        }
        if (ml.x != -INFINITY) {
            const float f = ex2(ml.x - m);
            ls = fmaf(f, ml.y, ls);
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = fmaf(f, v[e], o[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) red[warp][lane * V + e] = o[e];
    if (lane == 0) red[warp][D] = ls;
    __syncthreads();
    float lt = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) lt += red[w][D];
    const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
    const int i = (int)(rr / a.rep);
    uint16_t* op = a.out + sched[3] * a.o_b + i * a.o_t + (sched[4] * a.rep + rr - (int64_t)i * a.rep) * a.o_h;
    for (int d = threadIdx.x; d < D; d += THREADS) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) t += red[w][d];
        op[d] = float_to_half_bits(t * inv, XT{});
    }
}

template <int D, int G, int NT, typename XT>
cudaError_t launch_t(const AttnArgs& a, const AttnShape& s, cudaStream_t st) {
    using Gm = Geo<D, G, NT>;
    static std::mutex mu;
    static bool done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev]) {
            e = cudaFuncSetAttribute(attention_kernel<D, G, NT, XT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Gm::SMEM);
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)s.grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Gm::SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attention_kernel<D, G, NT, XT>, a);
    if (e != cudaSuccess || !s.split) return e;
    const int64_t items = (int64_t)a.B * a.Hkv * a.rtiles;
    const int by_item = items <= s.grid ? 1 : 0;
    cfg.gridDim = dim3((unsigned)(by_item ? items : s.grid), (unsigned)(a.rows < Gm::ROWS ? a.rows : Gm::ROWS));
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, combine_kernel<D, XT>, a, s.grid, (int)Gm::ROWS, by_item);
}

template <int D, int G, typename XT>
cudaError_t launch_n(const AttnArgs& a, const AttnShape& s, cudaStream_t st) {
    switch (s.nt) {
        case 1: return launch_t<D, G, 1, XT>(a, s, st);
        case 2: return launch_t<D, G, 2, XT>(a, s, st);
        case 4:
            if constexpr (D <= 128) return launch_t<D, G, 4, XT>(a, s, st);
            break;
    }
    return cudaErrorInvalidValue;
}

template <int D, typename XT>
cudaError_t launch_g(const AttnArgs& a, const AttnShape& s, int group, cudaStream_t st) {
    switch (group) {
        case 32: return launch_n<D, 32, XT>(a, s, st);
        case 64: return launch_n<D, 64, XT>(a, s, st);
        case 128:
            if constexpr (D >= 128) return launch_n<D, 128, XT>(a, s, st);
            break;
    }
    return cudaErrorInvalidValue;
}

// instantiated in kernels_kv_attention_d<D>_<type>.cu
template <int D, bool BF>
cudaError_t launch_d(const AttnArgs& a, const AttnShape& s, int group, cudaStream_t st);

}  // namespace kv
}  // namespace aq
