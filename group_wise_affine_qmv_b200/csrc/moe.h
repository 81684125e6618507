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
    int svec;                   // 1: a stage's scales (and biases) of a row are one aligned vector load
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
    uint16_t* h_hi;             // workspace: [T * topk, N] bf16, the activations' leading 8 bits
    uint16_t* h_lo;             //   ... and the next 8
    float* h_sum;               // workspace: [T * topk, N / 16], sums of 16 activations
    void* y;
    int64_t y_row;
    int ydt;                    // DT of y
    const void* r;              // optional residual, y's dtype
    int64_t r_row;
    float rms_eps;              // > 0: x normalised per token
    int cs;                     // CTAs of a cluster that share the experts of a block of y columns
};

// workspace bytes; every part starts on a 16-byte boundary
inline size_t h_bytes(int64_t T, int64_t topk, int64_t N) { return ((size_t)T * topk * N * 2 + 15) / 16 * 16; }
inline size_t workspace_bytes(int64_t T, int64_t topk, int64_t N) { return 2 * h_bytes(T, topk, N) + (size_t)T * topk * (N / 16) * 4; }

// instantiated in kernels_moe_b<BITS>_<type>.cu
template <int BITS, bool BF>
cudaError_t launch_b(const Args& a, int group, cudaStream_t s);
cudaError_t launch(Args& a, int bits, int group, bool bf16, cudaStream_t s);

}  // namespace moe
}  // namespace aq
