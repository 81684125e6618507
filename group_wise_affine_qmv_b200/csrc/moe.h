// moe.h -- arguments of the mixture-of-experts layer (kernels_moe*.cu, moe_kernel.cuh).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "aq_internal.h"

namespace aq {
namespace moe {

constexpr int MAX_TOKENS = 64;
constexpr int MAX_EXPERTS = 512;
constexpr int MAX_TOPK = 16;

struct Bank {
    const uint32_t* wq;         // [E, rows, K * bits / 32]
    const uint16_t* scales;     // [E, rows, K / G], rows dense
    const uint16_t* biases;
    int64_t w_row, w_exp;       // words
    int64_t s_exp, b_exp;       // elements
    int svec;                   // 1: a stage's scales (and biases) of a row are one aligned copy
    int blk;                    // 1: those of 16 rows together are a 16-byte aligned run
};

struct Args {
    const uint16_t* x;          // [T, K]
    int64_t x_row;
    const void* logits;         // [T, E]
    int64_t l_row;
    int ldt;                    // DT of logits
    int T, E, topk, norm;
    int K, N;                   // model size, expert size
    Bank gate, up, down;
    // workspace (Layout), written by the routing kernel ...
    int* entries;               // [1 + MAX_ENTRIES]: how many, then expert | tokens << 16 of each
    uint16_t* pairs;            // [MAX_ENTRIES][TB]: token * topk + choice of an entry's tokens
    float* weight;              // [T * topk]
    uint16_t* xh;               // [T, x_pitch(K)] f16: x scaled by a power of two per token, permuted like the codes
    float* xfac;                // [T]: what takes the sums back (and the RMS norm)
    // ... and by the gate/up kernel
    uint16_t* h;                // [T * topk, N] f16: weighted activations, a power of two per 16 columns, permuted;
                                // in two parts, what their rounding left over in T * topk rows more
    int parts;                  // of an activation: 1, or 2 where y is finer than bf16
    float* hscale;              // [T * topk, N / 16]: those powers of two
    unsigned* hmax;             // [T * topk]: the largest of each row's, as the bits of a float (zeroed by the first kernel)
    void* y;
    int64_t y_row;
    int ydt;                    // DT of y
    const void* r;              // optional residual, y's dtype
    int64_t r_row;
    float rms_eps;              // > 0: x normalised per token
    int cs;                     // CTAs of a cluster that share the experts of a block of y columns
    int* err;
};

constexpr int TB = 16;          // tokens of an entry
constexpr int MAX_ENTRIES = MAX_TOKENS * MAX_TOPK;

// columns of prepared x, in whole stages of any width (2-bit stages hold 512 codes)
__host__ __device__ constexpr int x_pitch(int K) { return (K + 511) / 512 * 512; }

// Offsets of the workspace's parts, each on a 16-byte boundary, and its size.
struct Layout {
    size_t pairs, weight, hmax, xh, xfac, h, hscale, bytes;
    Layout(int64_t T, int64_t topk, int64_t K, int64_t N) {
        auto up = [](size_t v) { return (v + 15) / 16 * 16; };
        const size_t p = (size_t)T * topk;
        pairs = up((1 + MAX_ENTRIES) * sizeof(int));
        weight = pairs + up(p * TB * 2);
        hmax = weight + up(p * 4);
        xh = hmax + up(p * 4);
        xfac = xh + up((size_t)T * x_pitch((int)K) * 2);
        h = xfac + up((size_t)T * 4);
        hscale = h + up(2 * p * N * 2);
        bytes = hscale + up(p * (N / 16) * 4);
    }
};

// instantiated in kernels_moe_b<BITS>_<type>.cu
template <int BITS, bool BF>
cudaError_t launch_b(const Args& a, int group, cudaStream_t s);
cudaError_t launch(const Args& a, int bits, int group, bool bf16, cudaStream_t s);

}  // namespace moe
}  // namespace aq
