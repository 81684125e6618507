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
//  - f16 operands whatever q's type: the low byte of a half masked to one nibble is, as it stands, the
//    f16 subnormal n 2^-24 (low nibble) or n 2^-20 (high nibble), which the tensor cores take exactly.  So
//    a pair of codes widens with one AND, and half the nibbles need no shift either.  The powers of two
//    leave with q (keys: its odd dims are scaled by 1/16) and with the final outputs (values).  q itself is
//    scaled by a power of two per row (its largest value near 2^14): elements down to 2^-24 of that largest (bf16 2^-27) are
//    exact as f16, smaller ones off by at most 2^-35 of it.
//  - The order of dims inside an MMA is free as long as both operands agree; lanes read whole
//    words, and q is stored permuted (0,4,1,5,2,6,3,7 within a word).
//  - V^T needs pairs of tokens in one register: one PRMT per pair of words and half.
//  - Running maximum: a warp keeps a reference per query row and rescales only when a score exceeds
//    it by more than 8 (in log2), decided by one vote per tile: p <= 2^8 instead of 1, and no
//    shuffles on the usual path.  Sums and the bias term stay per lane until the end.
//  - p s is rounded to f16 (11 bits, against the output's 8 or 11); s varies over tokens and may
//    lie anywhere in its 16-bit type's range, so p s is scaled by a power of two per group that
//    follows the largest |s| seen (the same vote), which keeps p s below 2^15 and exact to 11 bits
//    down to 2^-29 of that.
//  - Values: the sum over a context cancels.  Codes are positive, sum (p s) code and sum p b all but 1/1000 of each
//    other after 10^5 tokens, and the tensor cores cut an accumulator toward zero at every step, always the same
//    way: one running through a context of 131072 tokens left 5e-2 of the result's size (bf16 rounds 1.7e-3).  So
//      a tile's MMAs start from minus the middle of the codes (7.5, as 8 and 7 for half of the tokens each; one more MMA a
//      group, codes all -8 or -7: a sign bit makes the subnormal negative) and their result is added to an fp32 sum,
//      rounded to nearest; the bias term takes p (b + 7.5 s);
//      every second piece goes in as its mirror image, 15 - code with negative weights, whose cut goes the other
//      way (w ^ mask costs nothing in front of an AND).
//    Centred codes in one long accumulator do for channels around zero, but where some channels of a group lie far
//    off, the others' codes are all small: f16, one channel of 32 at 20 deviations: the others 2.6e-3 off after 8192 tokens
//    and 9.2e-2 after 131072; as it is 2.2e-4 and 4.6e-4 (rounding: 2.1e-4).  Without the mirror 3.0e-4 and 8.6e-4.  Cost: bf16
//    3 to 5% (32 sequences of 9001 to 32768: 250 against 243 us; 9% of a chunk of 512 queries over 4096 tokens), f16 0 to 4%.
//  - f16 outputs carry p s as two f16 numbers (PARTS): one rounding of 11 bits for every term would equal the output's
//    own.  131071 tokens, 32 heads on 8 of 128, group 128: 2.06e-4 off, the output's rounding 2.05e-4; bf16 in one part
//    1.70e-3, its rounding 1.69e-3.
//
//  - A warp's tile is 32 tokens where registers allow it (up to 8 query rows, head size up to 128),
//    two pieces of 16 whose votes, waits and loop control are shared; else 16.
//
// Work split.  A unit is one tile per warp, consecutive tokens of one (sequence, key/value head, row tile);
// warps keep their own softmax state and meet only at the end of an item.  All units of all
// items form one line, and every CTA takes an equal stretch of it, so ragged batches and single
// long sequences load the SMs alike.  A stretch that ends inside an item leaves a partial result
// (at most two per CTA), which the combine kernel adds in CTA order; nothing depends on timing.
//
// Measured, device time of a call: 32 sequences of 500 to 4096 tokens, 16 heads on 8 of 128, bf16: 43 us, 2.0 TB/s; of 9001
// to 32768, 32 heads on 8: 250 us, 3.1 TB/s (47% of a copy); one of 131071, f16: 56 us, 2.5 TB/s.  Bound by latency at the 11 warps
// an SM that registers allow: about 750 instructions a warp and tile of 32 tokens x 128, issue slots 46 to 56% busy, stalls on
// fixed latencies and shared memory.  Instantiations for 16 and 32 query rows with groups of 32 spill, f16 most (D 128, 32
// rows: 838 bytes of stores a thread; D 256, 16 rows: 750).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>
#include <type_traits>

#include "device_common.cuh"
#include "kv_cache.h"
#include "sm100_ptx.cuh"

namespace aq {
namespace kv {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int TILE = 16;              // tokens of a piece: the rows of an MMA

// f16 pairs from the nibbles of a word's halves: n 2^-24 and n 2^-20
__device__ __forceinline__ uint32_t nib_lo(uint32_t w) { return w & 0x000F000Fu; }
__device__ __forceinline__ uint32_t nib_hi(uint32_t w) { return w & 0x00F000F0u; }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = a b + c
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
// The pieces of a tile, odd ones (odd tiles where a tile is one piece) with complemented codes and negative weights: mask p.
template <int PCS>
struct Flip {
    uint32_t odd;                     // PCS 1: all ones in odd tiles
    __device__ __forceinline__ uint32_t mask(int p) const { return PCS == 1 ? odd : p & 1 ? ~0u : 0u; }
};
// -sum of a tile's weights times 8 (tokens 0 to 7 of a piece) or 7 (8 to 15), as the sums of low nibbles (mid[0], mid[1]) and of
// high ones
template <int PCS, int N>
__device__ __forceinline__ void middle(float (&mid)[4], const uint32_t (&b)[PCS][N], Flip<PCS> f) {
#pragma unroll
    for (int i = 0; i < PCS * N; i += 2) {
        const int p = i / N;
        const uint32_t lo = f.mask(p) & 0x000F000Fu, hi = f.mask(p) & 0x00F000F0u;
        if (i == 0) mma_from(mid, 0x80088008u ^ lo, 0x80808080u ^ hi, 0x80078007u ^ lo, 0x80708070u ^ hi, b[p][i % N], b[p][i % N + 1], 0.0f, 0.0f, 0.0f, 0.0f);
        else mma_f16(mid, 0x80088008u ^ lo, 0x80808080u ^ hi, 0x80078007u ^ lo, 0x80708070u ^ hi, b[p][i % N], b[p][i % N + 1]);
    }
}
// sum += (codes - middle) weights.  HI_R, HI_R8: rows r, r + 8 are low nibbles (weight 2^-24) or high ones (2^-20).
template <bool HI_R, bool HI_R8, int PCS, int N>
__device__ __forceinline__ void weigh(float (&sum)[4], const uint32_t (&a)[PCS][4], const uint32_t (&b)[PCS][N], const float (&mid)[4], Flip<PCS> f) {
    float d[4];
#pragma unroll
    for (int i = 0; i < PCS * N; i += 2) {
        const int p = i / N;
        const auto nib = [&](int k, bool hi) { return hi ? nib_hi(a[p][k] ^ f.mask(p)) : nib_lo(a[p][k] ^ f.mask(p)); };
        if (i == 0)
            mma_from(d, nib(0, HI_R), nib(1, HI_R8), nib(2, HI_R), nib(3, HI_R8), b[p][i % N], b[p][i % N + 1],
                     mid[HI_R ? 2 : 0], mid[HI_R ? 3 : 1], mid[HI_R8 ? 2 : 0], mid[HI_R8 ? 3 : 1]);
        else
            mma_f16(d, nib(0, HI_R), nib(1, HI_R8), nib(2, HI_R), nib(3, HI_R8), b[p][i % N], b[p][i % N + 1]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += d[e];
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
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int size) {   // size 0: zeros, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_small(uint32_t dst, const void* src, bool on) {   // 4, 8 or 16 bytes, or as many zeros
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N < 4 ? 4 : N), "r"(on ? N : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ float2 half_pair(uint32_t v, bf16_t) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 half_pair(uint32_t v, f16_t) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// N 16-bit values of a row as one load from shared memory
template <int N, typename XT>
struct Halves {
    static constexpr int W = N < 2 ? 1 : N / 2;
    uint32_t w[W];
    __device__ __forceinline__ void load(const uint16_t* p) {
        if constexpr (N == 1) w[0] = *p;
        else if constexpr (N == 2) w[0] = *reinterpret_cast<const uint32_t*>(p);
        else if constexpr (N == 4) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
        else *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ float f(int i) const {
        if constexpr (N == 1) return half_bits_to_float((uint16_t)w[0], XT{});
        const float2 v = half_pair(w[i >> 1], XT{});
        return (i & 1) ? v.y : v.x;
    }
};

// ---- the line of units ----

// The cached tokens [first, len) that some query of a sequence sees; first on a tile boundary.
struct Span {
    int len, first, units;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int64_t n, int unit) {
    Span s;
    const int most = (int)(a.max_pages * a.S);
    if (n < 0 || n > most) {
        atomicOr(a.err, DEVERR_INDEX);
        n = n < 0 ? 0 : most;
    }
    s.len = (int)n;
    s.first = 0;
    if (a.window > 0) {
        const int64_t f = n - a.Tq - a.window + 1;
        s.first = f < 0 ? 0 : (int)f & ~(TILE - 1);
    }
    s.units = (s.len - s.first + unit - 1) / unit;
    return s;
}

// The lengths as one warp sees them: 32 sequences at a time, lane b the b-th of the current ones.
// Every warp of every CTA walks them alike, so nothing has to be shared.
struct Lengths {
    const AttnArgs& a;
    const int lane, unit;
    int base;              // first sequence held
    Span mine;
    __device__ __forceinline__ Lengths(const AttnArgs& args, int ln, int un) : a(args), lane(ln), unit(un), base(-1) { hold(0); }
    __device__ __forceinline__ void hold(int b0) {
        if (b0 == base) return;
        base = b0;
        mine = span_of(a, b0 + lane < a.B ? __ldcg(a.lengths + b0 + lane) : 0, unit);
        if (b0 + lane >= a.B) mine.units = 0;
    }
    __device__ __forceinline__ Span of(int seq) {
        hold(seq & ~31);
        Span s;
        s.len = __shfl_sync(0xffffffffu, mine.len, seq & 31);
        s.first = __shfl_sync(0xffffffffu, mine.first, seq & 31);
        s.units = __shfl_sync(0xffffffffu, mine.units, seq & 31);
        return s;
    }
    // units of all sequences, times their items (the host keeps them below 2^31)
    __device__ __forceinline__ int total() {
        int n = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            hold(b0);
            n += mine.units;
        }
        return __reduce_add_sync(0xffffffffu, n) * a.Hkv * a.rtiles;
    }
    // the sequence that holds unit `at`, and the units before that sequence
    __device__ __forceinline__ void find(int at, int* seq, int* before) {
        int run = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            hold(b0);
            const int u = mine.units * a.Hkv * a.rtiles;
            int incl = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            incl += run;
            const unsigned hit = __ballot_sync(0xffffffffu, incl > at);
            if (hit) {
                const int l = __ffs(hit) - 1;
                *seq = b0 + l;
                *before = __shfl_sync(0xffffffffu, incl - u, l);
                return;
            }
            run = __shfl_sync(0xffffffffu, incl, 31);
        }
        *seq = a.B;
        *before = run;
    }
    // the units before a sequence
    __device__ __forceinline__ int before(int seq) {
        int n = 0;
        for (int b0 = 0; b0 < seq; b0 += 32) {
            hold(b0);
            if (b0 + lane < seq) n += mine.units;
        }
        return __reduce_add_sync(0xffffffffu, n) * a.Hkv * a.rtiles;
    }
};
// How CTAs share the line: no more CTAs than units, the first `more` of them one unit more than the others.
struct Shares {
    int n, each, more;
    __device__ __forceinline__ Shares(int W, int grid) {
        n = W < grid ? (W < 1 ? 1 : W) : grid;
        each = W / n;
        more = W - each * n;
    }
    __device__ __forceinline__ int start(int cta) const { return cta * each + (cta < more ? cta : more); }
    __device__ __forceinline__ int owner(int unit) const {
        const int big = more * (each + 1);
        return unit < big ? unit / (each + 1) : more + (unit - big) / each;
    }
};

template <int D, int G, int NT>
struct Geo {
    static constexpr int KG = D / G;                       // groups per row
    static constexpr int CH = D / 32;                      // 16-byte chunks of a row of codes
    static constexpr int PCS = pieces_of(D, NT);           // pieces of a tile
    // a piece of one side: chunk by chunk, the 16 tokens of a chunk together.  64 bytes of padding between
    // chunks put the two chunks that a shared-memory phase touches on different banks, and every lane reads
    // at one address plus constants
    static constexpr int CP = TILE * 16 + 64;
    static constexpr int CODES = CH * CP;
    static constexpr int SB = TILE * KG * 2;               // its scales, or its biases
    static constexpr int PIECE = 2 * CODES + 4 * SB;       // keys, values, their scales and biases
    static constexpr int STAGE = PCS * PIECE;
    static constexpr int NST = D == 64 ? 4 : 3;                       // stages of a warp's ring
    static constexpr int ROWS = 8 * NT;
    static constexpr int QP = D * 2 + 16;                  // bytes of a q row in shared memory
    static constexpr int RING = WARPS * NST * STAGE;
    static constexpr int MERGE = WARPS * ROWS * (D + 4) * 4;   // partial outputs of the warps (over the ring)
    static constexpr int BODY = RING > MERGE ? RING : MERGE;
    static constexpr int SMEM = BODY + ROWS * QP + KG * ROWS * 4 + ROWS * 4;
    // value token t of a piece: even tokens of an octet first, then odd ones
    static __device__ __forceinline__ int vpos(int t) { return (t & 8) | ((t & 1) << 2) | ((t >> 1) & 3); }
    static __device__ __forceinline__ int vtok(int pos) { return (pos & 8) | ((pos & 3) << 1) | ((pos >> 2) & 1); }
};

template <int D, int G, int NT, typename XT, bool FAST>
__global__ void __launch_bounds__(THREADS, ctas_per_sm(D, NT))
attention_kernel(const __grid_constant__ AttnArgs a) {
    using Gm = Geo<D, G, NT>;
    constexpr int KG = Gm::KG, ROWS = Gm::ROWS, NST = Gm::NST, PCS = Gm::PCS;
    constexpr int UNIT = unit_tokens(D, NT);
    static_assert(UNIT == WARPS * PCS * TILE, "a tile per warp");
    constexpr int KS = G < 64 ? G : 64;        // dims per sub-block
    constexpr int SUBS = D / KS;
    constexpr int MT = D / 16;                 // m tiles of the output
    constexpr int PARTS = std::is_same<XT, f16_t>::value ? 2 : 1;   // f16 numbers that carry a p s
    constexpr bool QREG = NT == 1 && D <= 128; // q fragments in registers

    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* qs = smem + Gm::BODY;                                        // [ROWS][QP] f16, permuted
    float* xs = reinterpret_cast<float*>(qs + ROWS * Gm::QP);             // [KG][ROWS] sums of q
    float* csc = xs + KG * ROWS;                                          // [ROWS] score scale
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;

    ptx::pdl_wait();                 // q, the cache and the lengths may come from the kernels before
    ptx::pdl_launch_dependents();    // after the wait: the combine kernel reads the lengths before its own
    Lengths L(a, lane, UNIT);
    int at = 0, at_end = 0, before = 0, seq = 0;
    if (a.split) {
        const Shares sh(L.total(), gridDim.x);
        if ((int)blockIdx.x < sh.n) {
            at = sh.start(blockIdx.x);
            at_end = sh.start(blockIdx.x + 1);
        }
        if (at < at_end) L.find(at, &seq, &before);
    } else {   // one item per CTA
        const int items = a.Hkv * a.rtiles;
        seq = blockIdx.x / items;
        const int units = L.of(seq).units;
        at = ((int)blockIdx.x - seq * items) * units;
        at_end = at + units;
    }
    bool first_seg = true;

    uint8_t* ring = smem + warp * NST * Gm::STAGE;
    // this lane's words of a tile: of token r (keys), of token 2c (values)
    const int k_lane = KS == 64 ? (c >> 1) * Gm::CP + r * 16 + (c & 1) * 8 : r * 16 + c * 4;
    const int v_lane = KS == 64 ? (r >> 2) * Gm::CP + c * 16 + (r & 3) * 4 : c * 16 + (r >> 1) * 4;
    const uint32_t ring_s = ptx::smem_u32(ring);

    while (at < at_end) {
        // ---- the segment: units [u0, u1) of item (seq, head, row tile) ----
        Span sp = L.of(seq);
        const int items = a.Hkv * a.rtiles;
        while (at >= before + sp.units * items) {
            before += sp.units * items;
            sp = L.of(++seq);
        }
        const int in_seq = at - before;
        const int it = in_seq / sp.units;
        const int u0 = in_seq - it * sp.units;
        const int u1 = at_end - at < sp.units - u0 ? u0 + at_end - at : sp.units;
        const int head = it / a.rtiles, rt = it - head * a.rtiles;
        const int row0 = rt * ROWS;
        at += u1 - u0;
        const int64_t* pages = a.pages + seq * a.pages_row;

        // ---- this warp's tiles: 16 PCS tokens from tw, every UNIT ----
        const int nu = u1 - u0;
        const int tw = sp.first + u0 * UNIT + warp * (PCS * TILE);
        int nt = 0;                  // those with a token below len
        if (tw < sp.len) {
            const int left = (sp.len - tw + UNIT - 1) / UNIT;
            nt = left < nu ? left : nu;
        }
        bool missing = false;        // a page id outside the cache: its tokens count as zeros

        // Fast layout: a piece lies in one page, and a lane copies the same chunks of every piece.  The
        // slot in the page moves on by whole units.  Page ids are fetched 32 tiles at a time, a lane per
        // tile, one batch ahead, so that no copy waits for one.  All strides fit 32 bits (in bytes).
        int l_slot = 0;
        uint32_t pid_now[PCS];       // this lane's tile of the current batch; ~0: no such page
        int64_t pid_next[PCS];       // ... of the next one, as loaded: a look at one would wait for it
        const uint8_t *kh = nullptr, *vh = nullptr, *sh = nullptr;
        uint32_t s_page = 0;
        // this lane's chunk and tokens: eight lanes write one stretch of banks, a warp reads whole rows
        const int l_ch = (lane & 1) | (Gm::CH >= 4 ? ((lane >> 3) & (Gm::CH / 2 - 1)) << 1 : 0);
        const int l_row = ((lane >> 1) & 3) | (Gm::CH == 2 ? (lane >> 3) << 2 : Gm::CH == 4 ? (lane >> 4) << 2 : 0);
        constexpr int RPI = 32 / Gm::CH;             // tokens per copy instruction
        auto fetch_pids = [&](int i0) {              // the pages of tiles i0 .. i0 + 31
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc) {
                pid_next[pc] = -1;
                if (i0 + lane < nt) {
                    const int t = tw + (i0 + lane) * UNIT + pc * TILE;
                    if (t < sp.len) pid_next[pc] = __ldcg(pages + t / a.S);
                }
            }
        };
        auto next_pids = [&](int i0) {               // the fetched batch becomes the current one, tiles i0 .. on
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc) pid_now[pc] = (uint64_t)pid_next[pc] < (uint64_t)a.P ? (uint32_t)pid_next[pc] : 0xffffffffu;
            fetch_pids(i0 + 32);
        };
        if constexpr (FAST) {
            l_slot = tw % a.S;
            fetch_pids(0);
            kh = reinterpret_cast<const uint8_t*>(a.k.wq + head * a.k.w_head + l_row * a.k.w_slot) + l_ch * 16;
            vh = reinterpret_cast<const uint8_t*>(a.v.wq + head * a.v.w_head + Gm::vtok(l_row) * a.v.w_slot) + l_ch * 16;
            // scales and biases: a piece is one run of 2 KG chunks in each of the four arrays; with KG 8
            // this lane copies chunk lane % 16 of two arrays (keys' and values', lane / 16 choosing)
            const int arr = (lane / (2 * KG)) & 3, pc = lane % (2 * KG);
            const Side& sd = arr < 2 ? a.k : a.v;
            const bool bias = arr & 1;
            sh = reinterpret_cast<const uint8_t*>((bias ? sd.biases + head * sd.b_head : sd.scales + head * sd.s_head) + pc * 8);
            s_page = (uint32_t)((bias ? sd.b_page : sd.s_page) * 2);
        }
        auto load_fast = [&](int i, uint32_t dst) {
            const int t0 = tw + i * UNIT;
            if ((i & 31) == 0) next_pids(i);
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc)
                if (t0 + pc * TILE < sp.len) {
                    const uint32_t id = __shfl_sync(0xffffffffu, pid_now[pc], i & 31);
                    const bool ok = id != 0xffffffffu;
                    const uint32_t pid = ok ? id : 0u;
                    const int size = ok ? 16 : 0;    // zeros for a missing page
                    uint32_t slot = l_slot + pc * TILE;
                    if (slot >= (uint32_t)a.S) slot = 0;
                    missing |= !ok;
                    const uint32_t d0 = dst + pc * Gm::PIECE;
                    const uint8_t* kp = kh + (uint64_t)pid * a.k_page + (uint64_t)slot * a.k_slot;
                    const uint8_t* vp = vh + (uint64_t)pid * a.v_page + (uint64_t)slot * a.v_slot;
#pragma unroll
                    for (int i = 0; i < TILE / RPI; ++i) {
                        // D 256 copies four tokens at a time: values in the order of their positions
                        const int vt = Gm::CH == 8 ? (i & 1) + 8 * (i >> 1) : RPI * i;
                        cp16(d0 + l_ch * Gm::CP + (l_row + RPI * i) * 16, kp + (uint64_t)(RPI * i) * a.k_slot, size);
                        cp16(d0 + Gm::CODES + l_ch * Gm::CP + (l_row + RPI * i) * 16, vp + (uint64_t)vt * a.v_slot, size);
                    }
                    const uint8_t* sp_ = sh + (uint64_t)pid * s_page + slot * (KG * 2);
                    if (KG >= 4 || lane < 8 * KG) cp16(d0 + 2 * Gm::CODES + lane * 16, sp_, size);
                    if constexpr (KG == 8) {         // the values' two arrays
                        const bool bias = lane >= 16;
                        const uint8_t* vs = reinterpret_cast<const uint8_t*>(
                            bias ? a.v.biases + pid * a.v.b_page + head * a.v.b_head : a.v.scales + pid * a.v.s_page + head * a.v.s_head);
                        cp16(d0 + 2 * Gm::CODES + 512 + lane * 16, vs + slot * (KG * 2) + (lane & 15) * 16, size);
                    }
                }
            l_slot += a.unit_slots;
            if (l_slot >= a.S) l_slot -= a.S;
        };
        // Any page size and strides: every token has a page and a slot of its own, looked up by the lanes r of
        // its piece (lane % 16) a tile ahead.  Scales and biases copy row by row where rows of them allow it
        // (scp); else they go through registers, which are stored with the next tile's issue.  (32 sequences of 500 to
        // 4096 tokens, 16 heads on 8 of 128, pages of 8: 47 us against 41 in pages of 64; each lookup and scale waited
        // for in its own tile took 108.  Pages of 1 and one group a head: 62 us.)
        // Tokens before the first query's window share a tile with it, but not a page: theirs may be gone.
        const int64_t w0 = (int64_t)sp.len - a.Tq - a.window + 1;
        const int seen0 = a.window > 0 && w0 > 0 ? (int)w0 : 0;
        int64_t id_ahead[PCS];
        int sl_ahead[PCS], late_st = -1;
        uint16_t late[PCS][2][KG];
        auto fetch_rows = [&](int i) {
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc) {
                const int t = tw + i * UNIT + pc * TILE + (lane & 15);
                id_ahead[pc] = -1;
                sl_ahead[pc] = 0;
                if (i < nt && t < sp.len && t >= seen0) {
                    const int pg = t / a.S;
                    sl_ahead[pc] = t - pg * a.S;
                    id_ahead[pc] = __ldcg(pages + pg);
                }
            }
        };
        auto store_late = [&]() {
            if (late_st < 0) return;
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int g = 0; g < KG; ++g)
                        reinterpret_cast<uint16_t*>(ring + late_st * Gm::STAGE + pc * Gm::PIECE + 2 * Gm::CODES)
                            [(2 * x + (lane >> 4)) * TILE * KG + (lane & 15) * KG + g] = late[pc][x][g];
            late_st = -1;
        };
        auto load_any = [&](int i, int st) {
            uint32_t id[PCS];            // ~0: no token, or no such page
            int sl[PCS];
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc) {
                id[pc] = (uint64_t)id_ahead[pc] < (uint64_t)a.P ? (uint32_t)id_ahead[pc] : 0xffffffffu;
                sl[pc] = sl_ahead[pc];
                const int t = tw + i * UNIT + pc * TILE + (lane & 15);
                missing |= id[pc] == 0xffffffffu && t < sp.len && t >= seen0;
            }
            fetch_rows(i + 1);
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc) {
                const uint32_t dst = ring_s + st * Gm::STAGE + pc * Gm::PIECE;
#pragma unroll
                for (int x = 0; x < TILE * Gm::CH / 32; ++x) {
                    const int row = (lane + 32 * x) / Gm::CH, ch = lane % Gm::CH;
                    uint32_t pid = __shfl_sync(0xffffffffu, id[pc], row);
                    const int slot = __shfl_sync(0xffffffffu, sl[pc], row);
                    const int size = pid != 0xffffffffu ? 16 : 0;
                    if (!size) pid = 0;
                    cp16(dst + ch * Gm::CP + row * 16,
                         reinterpret_cast<const uint8_t*>(a.k.wq + pid * a.k.w_page + head * a.k.w_head + slot * a.k.w_slot) + ch * 16, size);
                    cp16(dst + Gm::CODES + ch * Gm::CP + Gm::vpos(row) * 16,
                         reinterpret_cast<const uint8_t*>(a.v.wq + pid * a.v.w_page + head * a.v.w_head + slot * a.v.w_slot) + ch * 16, size);
                }
                const bool ok = id[pc] != 0xffffffffu;
                const int64_t pid = ok ? id[pc] : 0;
#pragma unroll
                for (int x = 0; x < 2; ++x) {        // keys, values; scales by lanes 0 to 15, biases by the others
                    const Side& sd = x ? a.v : a.k;
                    const uint16_t* src = lane < 16 ? sd.scales + pid * sd.s_page + head * sd.s_head + sl[pc] * sd.s_slot
                                                    : sd.biases + pid * sd.b_page + head * sd.b_head + sl[pc] * sd.b_slot;
                    if (KG > 1 && a.scp) {
                        cp_small<KG * 2>(dst + 2 * Gm::CODES + (2 * x + (lane >> 4)) * Gm::SB + (lane & 15) * KG * 2, src, ok);
                    } else {
#pragma unroll
                        for (int g = 0; g < KG; ++g) late[pc][x][g] = ok ? __ldcg(src + g) : (uint16_t)0;
                    }
                }
            }
            if (KG == 1 || !a.scp) late_st = st;
        };
        if constexpr (!FAST) fetch_rows(0);
        auto issue = [&](int i, int st) {
            if constexpr (!FAST) store_late();
            if (i < nt) {
                if constexpr (FAST) load_fast(i, ring_s + st * Gm::STAGE);
                else load_any(i, st);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < NST - 1; ++i) issue(i, i);

        // ---- q rows of the item: scaled to f16, permuted, with their group sums.  The softmax scale's sign
        // goes with q, so that a row's score scale is positive (a zero scale: q = 0, scale 1) ----
        const float sgn = a.scale_log2 > 0.0f ? 1.0f : a.scale_log2 < 0.0f ? -1.0f : 0.0f;
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
                for (int e = 0; e < EPL; ++e) f[e] = half_bits_to_float(__ldcg(qp + e), XT{}) * sgn;
            }
            float am = 0.0f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) am = fmaxf(am, fabsf(f[e]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
            // 2^(14 - exponent of the largest value): exact products (an exponent of infinity stays in range)
            const int ex = min(max((int)((__float_as_uint(am) >> 23) & 255) - 127, -100), 127);
            const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
            float X = 0.0f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                const int d = lane * EPL + e, n = d & 7;
                X += f[e] * up;
                // odd dims meet codes of 16 times the weight
                const __half hf = __float2half_rn((n & 1) ? f[e] * up * 0.0625f : f[e] * up);
                // order within a word: 0 4 1 5 2 6 3 7
                const int pos = (d & ~7) + 2 * (n & 3) + (n >> 2);
                *reinterpret_cast<__half*>(qs + row * Gm::QP + pos * 2) = hf;
            }
            constexpr int GL = G / EPL;           // lanes per group
#pragma unroll
            for (int o = GL / 2; o > 0; o >>= 1) X += __shfl_xor_sync(0xffffffffu, X, o);
            // scores are kept in units of 2^-24: the codes' weight
            if (lane % GL == 0) xs[(lane / GL) * ROWS + row] = X * 0x1p-24f;
            if (lane == 0)
                csc[row] = (a.scale_log2 == 0.0f ? 1.0f : fabsf(a.scale_log2)) * __uint_as_float((uint32_t)(ex - 14 + 127) << 23) * 0x1p24f;
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
        float nm[NT][2], thr[NT][2], l[NT][2], ab[KG][NT][2], vmul[KG], vthr[KG];
        float acc[MT][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                nm[n][e] = 0.0f;                  // minus the reference, in log2
                thr[n][e] = -INFINITY;            // the score above which it has to move
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

        const int pos0 = sp.len - a.Tq;           // position of query token 0
        const int last_i = a.Tq - 1;
        int st = 0;                               // ring slot of tile i

#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
            issue(i + NST - 1, st == 0 ? NST - 1 : st - 1);
            cp_wait<NST - 1>();
            __syncwarp();
            const uint8_t* kt = ring + st * Gm::STAGE;
            const int t0 = tw + i * UNIT;
            // every token of the tile visible to every row?
            const bool full = pos0 >= 0 && t0 + PCS * TILE - 1 <= pos0 &&
                              (a.window == 0 || t0 > (int64_t)pos0 + last_i - a.window);

            // ---- scores of tokens r and r + 8 of each piece for query rows 2c, 2c + 1 of each n tile ----
            float s[PCS][NT][4];
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc) {
                const uint8_t* kp = kt + pc * Gm::PIECE;
                const uint16_t* ssb = reinterpret_cast<const uint16_t*>(kp + 2 * Gm::CODES);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[pc][n][e] = 0.0f;
                float d[NT][4];
                Halves<KG, XT> ks[2], kb[2];      // key scales and biases of tokens r and r + 8
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ks[h].load(ssb + (r + 8 * h) * KG);
                    kb[h].load(ssb + TILE * KG + (r + 8 * h) * KG);
                }
#pragma unroll
                for (int sb = 0; sb < SUBS; ++sb) {
                    constexpr int SPG = G / KS;
                    const int g = sb / SPG;
                    if (sb % SPG == 0)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) d[n][e] = 0.0f;
                    uint32_t w0[2], w1[2];        // rows r and r + 8
                    if constexpr (KS == 64) {
                        const uint2 x = *reinterpret_cast<const uint2*>(kp + k_lane + sb * 2 * Gm::CP);
                        const uint2 y = *reinterpret_cast<const uint2*>(kp + k_lane + sb * 2 * Gm::CP + 8 * 16);
                        w0[0] = x.x; w0[1] = x.y;
                        w1[0] = y.x; w1[1] = y.y;
                    } else {
                        w0[0] = *reinterpret_cast<const uint32_t*>(kp + k_lane + sb * Gm::CP);
                        w1[0] = *reinterpret_cast<const uint32_t*>(kp + k_lane + sb * Gm::CP + 8 * 16);
                    }
#pragma unroll
                    for (int j = 0; j < KS / 32; ++j) {
                        const int word = KS == 64 ? sb * 8 + 2 * c + j : sb * 4 + c;
                        const uint32_t u = w0[j], v = w1[j], us = u >> 8, vs = v >> 8;
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
                            mma_f16(d[n], nib_lo(u), nib_lo(v), nib_hi(u), nib_hi(v), b[0], b[1]);
                            mma_f16(d[n], nib_lo(us), nib_lo(vs), nib_hi(us), nib_hi(vs), b[2], b[3]);
                        }
                    }
                    if (sb % SPG == SPG - 1) {    // the group's fold: s D + b X
                        const float s0 = ks[0].f(g), s1 = ks[1].f(g), b0 = kb[0].f(g), b1 = kb[1].f(g);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const float2 x = *reinterpret_cast<const float2*>(xs + g * ROWS + 8 * n + 2 * c);
                            s[pc][n][0] = fmaf(s0, d[n][0], fmaf(b0, x.x, s[pc][n][0]));
                            s[pc][n][1] = fmaf(s0, d[n][1], fmaf(b0, x.y, s[pc][n][1]));
                            s[pc][n][2] = fmaf(s1, d[n][2], fmaf(b1, x.x, s[pc][n][2]));
                            s[pc][n][3] = fmaf(s1, d[n][3], fmaf(b1, x.y, s[pc][n][3]));
                        }
                    }
                }
            }
            float sv[PCS][KG][2], bv[PCS][KG][2]; // value scales and biases of tokens r and r + 8
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc) {
                const uint16_t* ssb = reinterpret_cast<const uint16_t*>(kt + pc * Gm::PIECE + 2 * Gm::CODES);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    Halves<KG, XT> x, y;
                    x.load(ssb + 2 * TILE * KG + (r + 8 * h) * KG);
                    y.load(ssb + 3 * TILE * KG + (r + 8 * h) * KG);
#pragma unroll
                    for (int g = 0; g < KG; ++g) {
                        sv[pc][g][h] = x.f(g);
                        bv[pc][g][h] = fmaf(h == 0 ? 8.0f : 7.0f, sv[pc][g][h], y.f(g));
                    }
                }
            }
            if (!full) {
                // rows see tokens up to their position, and from their window's start; a token that no
                // row sees (stale, another sequence's) may hold any scale: it is zeroed
                const int64_t seen_lo = a.window == 0 ? 0 : (int64_t)pos0 - a.window + 1;
#pragma unroll
                for (int pc = 0; pc < PCS; ++pc)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = t0 + pc * TILE + r + 8 * h;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int row = row0 + 8 * n + 2 * c + e;
                                int qi = row / a.rep;
                                if (qi > last_i) qi = last_i;
                                const int pos = pos0 + qi;
                                if (!(t <= pos && (a.window == 0 || t > (int64_t)pos - a.window))) s[pc][n][2 * h + e] = -INFINITY;
                            }
                        if (t >= sp.len || t < seen_lo)
#pragma unroll
                            for (int g = 0; g < KG; ++g) sv[pc][g][h] = bv[pc][g][h] = 0.0f;
                    }
            }
            // ---- one vote: does a score or a value scale leave the range of the references? ----
            bool out_of = false;
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) out_of |= fmaxf(s[pc][n][e], s[pc][n][e + 2]) > thr[n][e];
            }
#pragma unroll
            for (int g = 0; g < KG; ++g) {
                float m = fmaxf(fabsf(sv[0][g][0]), fabsf(sv[0][g][1]));
#pragma unroll
                for (int pc = 1; pc < PCS; ++pc) m = fmaxf(m, fmaxf(fabsf(sv[pc][g][0]), fabsf(sv[pc][g][1])));
                out_of |= m > vthr[g];
            }
            if (__any_sync(0xffffffffu, out_of)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = -INFINITY;
#pragma unroll
                        for (int pc = 0; pc < PCS; ++pc) m = fmaxf(m, fmaxf(s[pc][n][e], s[pc][n][e + 2]));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        const bool none = thr[n][e] == -INFINITY;
                        if (m > -INFINITY && (none || fmaf(m, cs[n][e], nm[n][e]) > 0.0f)) {
                            const float f = none ? 0.0f : ex2(-fmaf(m, cs[n][e], nm[n][e]));
                            nm[n][e] = -m * cs[n][e];
                            thr[n][e] = m + 8.0f / cs[n][e];
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
#pragma unroll
                for (int g = 0; g < KG; ++g) {
                    // an infinite scale is no reference: it would flush the rows that do not see its token
                    float m = 0.0f;
#pragma unroll
                    for (int pc = 0; pc < PCS; ++pc)
#pragma unroll
                        for (int h = 0; h < 2; ++h) m = fmaxf(m, isinf(sv[pc][g][h]) ? 0.0f : fabsf(sv[pc][g][h]));
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
            uint32_t pb[KG][NT][PCS][2 * PARTS];   // elements 2, 3: what the rounding left over
            const Flip<PCS> flip{(i & 1) ? ~0u : 0u};
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc) {
                // ---- p, its sums, and p s as f16 with tokens along k ----
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = ex2(fmaf(s[pc][n][e], cs[n][e & 1], nm[n][e & 1]));
                    l[n][0] += p[0] + p[2];
                    l[n][1] += p[1] + p[3];
#pragma unroll
                    for (int g = 0; g < KG; ++g) {
                        const float vm = flip.mask(pc) ? -vmul[g] : vmul[g];
                        const float m0 = sv[pc][g][0] * vm, m1 = sv[pc][g][1] * vm;
                        float t[4] = {p[0] * m0, p[1] * m0, p[2] * m1, p[3] * m1};
                        if (full) {
                            ab[g][n][0] = fmaf(p[0], bv[pc][g][0], fmaf(p[2], bv[pc][g][1], ab[g][n][0]));
                            ab[g][n][1] = fmaf(p[1], bv[pc][g][0], fmaf(p[3], bv[pc][g][1], ab[g][n][1]));
                        } else {                  // a token that this row does not see may be infinite or NaN
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (s[pc][n][e] == -INFINITY) t[e] = 0.0f;
                                else ab[g][n][e & 1] = fmaf(p[e], bv[pc][g][e >> 1], ab[g][n][e & 1]);
                            }
                        }
                        const __half2 x = __floats2half2_rn(t[0], t[1]);
                        const __half2 y = __floats2half2_rn(t[2], t[3]);
                        pb[g][n][pc][0] = transpose8(*reinterpret_cast<const uint32_t*>(&x));
                        pb[g][n][pc][1] = transpose8(*reinterpret_cast<const uint32_t*>(&y));
                        if constexpr (PARTS == 2) {
                            const float2 fx = __half22float2(x), fy = __half22float2(y);
                            const __half2 u = __floats2half2_rn(t[0] - fx.x, t[1] - fx.y);
                            const __half2 v = __floats2half2_rn(t[2] - fy.x, t[3] - fy.y);
                            pb[g][n][pc][2] = transpose8(*reinterpret_cast<const uint32_t*>(&u));
                            pb[g][n][pc][3] = transpose8(*reinterpret_cast<const uint32_t*>(&v));
                        }
                    }
                }
            }
            // ---- O^T += V^T (p s)^T ----
            const uint8_t* vp = kt + Gm::CODES + v_lane;
            float mid[NT][4];
#pragma unroll
            for (int sb = 0; sb < SUBS; ++sb) {
                const int g = sb * KS / G;
                if (sb * KS % G == 0)
#pragma unroll
                    for (int n = 0; n < NT; ++n) middle(mid[n], pb[g][n], flip);
                uint32_t a[PCS][4];
#pragma unroll
                for (int pc = 0; pc < PCS; ++pc) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)   // tokens 2c, 2c + 1, 2c + 8, 2c + 9
                        w[k] = *reinterpret_cast<const uint32_t*>(vp + pc * Gm::PIECE + sb * (KS / 32) * Gm::CP + k * 64);
                    if constexpr (KS == 64) {
                        a[pc][0] = __byte_perm(w[0], w[1], 0x5410); a[pc][1] = __byte_perm(w[0], w[1], 0x7632);
                        a[pc][2] = __byte_perm(w[2], w[3], 0x5410); a[pc][3] = __byte_perm(w[2], w[3], 0x7632);
                    } else {
                        const uint32_t sel = (r & 1) ? 0x7632 : 0x5410;
                        a[pc][0] = a[pc][1] = __byte_perm(w[0], w[1], sel);
                        a[pc][2] = a[pc][3] = __byte_perm(w[2], w[3], sel);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if constexpr (KS == 64) {   // nibbles 2j, 2j + 1 (rows r) and 2j + 4, 2j + 5 (rows r + 8)
                            weigh<false, false>(acc[sb * 4 + 2 * j][n], a, pb[g][n], mid[n], flip);
                            weigh<true, true>(acc[sb * 4 + 2 * j + 1][n], a, pb[g][n], mid[n], flip);
                        } else {                    // nibble 2j (rows r) and 2j + 1 (rows r + 8) of this lane's half word
                            weigh<false, true>(acc[sb * 2 + j][n], a, pb[g][n], mid[n], flip);
                        }
                    }
#pragma unroll
                    for (int pc = 0; pc < PCS; ++pc)
#pragma unroll
                        for (int k = 0; k < 4; ++k) a[pc][k] >>= 8;
                }
            }
            __syncwarp();   // every lane has read the slot before it is refilled
            st = st + 1 == NST ? 0 : st + 1;
        }
        if (missing) atomicOr(a.err, DEVERR_INDEX);
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
                    mo[row * (D + 4) + D] = thr[n][e] == -INFINITY && l[n][e] == 0.0f ? -INFINITY : -nm[n][e];
                    mo[row * (D + 4) + D + 1] = l[n][e];
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int g = mt * 16 / G;
                    const float inv = 1.0f / vmul[g];   // a power of two: exact
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int dim = KS == 64 ? (mt >> 2) * 64 + 8 * r + (mt & 3) + 4 * h : (mt >> 1) * 32 + 4 * r + 2 * (mt & 1) + h;
                        // the codes' weight, by the nibble that they came from
                        const float w = (KS == 64 ? mt & 1 : h) ? 0x1p20f : 0x1p24f;
                        mo[row * (D + 4) + dim] = fmaf(acc[mt][n][e + 2 * h] * w, inv, ab[g][n][e]);
                    }
                }
            }
        __syncthreads();

        // ---- the warps' results together; a whole item is finished here, a part goes to the workspace ----
        const bool whole = u0 == 0 && u1 == sp.units;
        const int64_t pslot = 2 * blockIdx.x + (first_seg ? 0 : 1);
        for (int x = threadIdx.x; x < ROWS * (D / 4); x += THREADS) {
            const int row = x / (D / 4), d4 = (x % (D / 4)) * 4;
            const int rr = row0 + row;
            if (rr >= a.rows) break;      // rows in order: nothing behind it
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
                {
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
    // sequences without a visible token: their rows are zeros
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)
        if (L.of(b).units == 0) {
            const int64_t n = (int64_t)a.Tq * a.Hq * D;
            for (int64_t i = threadIdx.x; i < n; i += THREADS) {
                const int64_t th = i / D, t = th / a.Hq;
                a.out[b * a.o_b + t * a.o_t + (th - t * a.Hq) * a.o_h + (i - th * D)] = 0;
            }
        }
}

// Joins the partial results of an item whose units several CTAs shared: the last segment of the CTA
// it starts in and the first segments of the CTAs after it, added in that order.  Block (x, row): the
// item x when there are fewer items than CTAs, else the item that starts in CTA x's stretch and
// reaches past it, if there is one.  WP warps: 16 for items of many parts, which then are all in flight at once (one
// sequence of 8191 tokens, 8 items of 55 parts: 14.6 us the call against 16.2 with 4 warps), 4 for few.
template <int D, typename XT, int WP>
__global__ void __launch_bounds__(32 * WP) combine_kernel(const __grid_constant__ AttnArgs a, int grid, int ROWS, int by_item, int unit) {
    __shared__ float red[WP][D + 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.y;
    // the lengths are complete: the attention kernel waited for them before this one started
    Lengths L(a, lane, unit);
    const Shares sh(L.total(), grid);
    const int items = a.Hkv * a.rtiles;
    int before = 0, j = blockIdx.x, first = -1, last = -1;
    int seq = 0, it = 0, units = 0, slot0 = 0;
    if (by_item) {
        seq = blockIdx.x / items;
        it = blockIdx.x - seq * items;
        before = L.before(seq);
        units = L.of(seq).units;
        if (units > 0) j = sh.owner(before + it * units);   // the CTA whose stretch holds the item's first unit
    } else if (j < sh.n - 1) {        // the item of CTA j's last unit
        const int hi = sh.start(j + 1);
        L.find(hi - 1, &seq, &before);
        units = L.of(seq).units;
        it = (hi - 1 - before) / units;
    }
    if (units > 0) {
        const int lo = sh.start(j), hi = sh.start(j + 1);
        const int s0 = before + it * units, s1 = s0 + units;
        if (s1 > hi && s0 >= lo) {
            first = j;
            slot0 = s0 > lo ? 1 : 0;  // not CTA j's first segment, unless the item starts its stretch
            last = sh.owner(s1 - 1);  // the CTA that holds its last unit
        }
    }
    const int head = it / a.rtiles;
    const int rr = (it - head * a.rtiles) * ROWS + row;
    ptx::pdl_wait();                  // the partial results
    ptx::pdl_launch_dependents();
    if (first < 0 || rr >= a.rows) return;
    auto part = [&](int k) { return (int64_t)(2 * (first + k) + (k == 0 ? slot0 : 0)) * ROWS + row; };
    const int np = last - first + 1;
    // a running reference per warp (parts k = warp, warp + WP, ...), four parts in flight
    constexpr int V = D / 32;
    float o[V], ls = 0.0f, m = -INFINITY;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.0f;
    for (int k0 = warp; k0 < np; k0 += 4 * WP) {
        float2 ml[4];
        float v[4][V];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = k0 + u * WP;
            ml[u] = make_float2(-INFINITY, 0.0f);
            if (k < np) {
                const int64_t p = part(k);
                ml[u] = __ldcg(reinterpret_cast<const float2*>(a.part_ml + p * 2));
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const float2 x = __ldcg(reinterpret_cast<const float2*>(a.part_o + p * D + lane * V + e));
                    v[u][e] = x.x;
                    v[u][e + 1] = x.y;
                }
            }
        }
        const float mn = fmaxf(fmaxf(m, fmaxf(ml[0].x, ml[1].x)), fmaxf(ml[2].x, ml[3].x));
        if (mn == -INFINITY) continue;                    // (a NaN reference is never -inf)
        const float f = m == -INFINITY ? 0.0f : ex2(m - mn);
        ls *= f;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] *= f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (ml[u].x != -INFINITY) {
                const float g = ex2(ml[u].x - mn);
                ls = fmaf(g, ml[u].y, ls);
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = fmaf(g, v[u][e], o[e]);
            }
        m = mn;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) red[warp][lane * V + e] = o[e];
    if (lane == 0) {
        red[warp][D] = ls;
        red[warp][D + 1] = m;
    }
    __syncthreads();
    float mt = -INFINITY;
#pragma unroll
    for (int w = 0; w < WP; ++w) mt = fmaxf(mt, red[w][D + 1]);
    const int i = rr / a.rep;
    uint16_t* op = a.out + seq * a.o_b + i * a.o_t + (head * a.rep + rr - i * a.rep) * (int64_t)a.o_h;
    for (int d = threadIdx.x; d < D; d += 32 * WP) {
        float t = 0.0f, lt = 0.0f;
#pragma unroll
        for (int w = 0; w < WP; ++w) {
            const float f = red[w][D + 1] == -INFINITY ? 0.0f : ex2(red[w][D + 1] - mt);
            lt = fmaf(f, red[w][D], lt);
            t = fmaf(f, red[w][d], t);
        }
        op[d] = float_to_half_bits(t * (lt == 0.0f ? 0.0f : 1.0f / lt), XT{});
    }
}

template <int D, int G, int NT, typename XT, bool FAST>
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
            e = cudaFuncSetAttribute(attention_kernel<D, G, NT, XT, FAST>, cudaFuncAttributeMaxDynamicSharedMemorySize, Gm::SMEM);
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
    e = cudaLaunchKernelEx(&cfg, attention_kernel<D, G, NT, XT, FAST>, a);
    if (e != cudaSuccess || !s.split) return e;
    const int64_t items = (int64_t)a.B * a.Hkv * a.rtiles;
    const int by_item = items <= s.grid ? 1 : 0;
    cfg.gridDim = dim3((unsigned)(by_item ? items : s.grid), (unsigned)(a.rows < Gm::ROWS ? a.rows : Gm::ROWS));
    cfg.dynamicSmemBytes = 0;
    constexpr int MANY = 16;          // parts of an item, or nearly
    if (s.grid >= MANY * items) {
        cfg.blockDim = dim3(32 * 16);
        return cudaLaunchKernelEx(&cfg, combine_kernel<D, XT, 16>, a, s.grid, (int)Gm::ROWS, by_item, unit_tokens(D, NT));
    }
    return cudaLaunchKernelEx(&cfg, combine_kernel<D, XT, WARPS>, a, s.grid, (int)Gm::ROWS, by_item, unit_tokens(D, NT));
}

template <int D, int G, typename XT>
cudaError_t launch_n(const AttnArgs& a, const AttnShape& s, cudaStream_t st) {
    switch (s.nt) {
        case 1: return a.fast ? launch_t<D, G, 1, XT, true>(a, s, st) : launch_t<D, G, 1, XT, false>(a, s, st);
        case 2: return a.fast ? launch_t<D, G, 2, XT, true>(a, s, st) : launch_t<D, G, 2, XT, false>(a, s, st);
        case 4:
            if constexpr (D <= 128) return a.fast ? launch_t<D, G, 4, XT, true>(a, s, st) : launch_t<D, G, 4, XT, false>(a, s, st);
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
