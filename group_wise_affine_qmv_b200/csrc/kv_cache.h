// kv_cache.h -- arguments of the 4-bit key/value cache kernels (kernels_kv_append.cu,
// kernels_kv_attention*.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "aq_internal.h"

namespace aq {
namespace kv {

// One side (keys or values) of a paged cache: element [page, head, slot, d] as packed codes, with
// its group scales and biases.  Strides of pages, heads and slots; the innermost stride is 1.
struct Side {
    uint32_t* wq;       // [P, H, S, D/8]
    uint16_t* scales;   // [P, H, S, D/G]
    uint16_t* biases;
    int64_t w_page, w_head, w_slot;   // words
    int64_t s_page, s_head, s_slot;   // elements
    int64_t b_page, b_head, b_slot;
};

struct AppendArgs {
    const uint16_t* x[2];       // k, v: [T, H, D]
    int64_t x_tok[2], x_head[2];
    uint16_t* out[2];           // optional: the values the cache then stands for, [T, H, D]
    int64_t o_tok[2], o_head[2];
    int xvec[2], ovec[2];       // 1: every 8-element piece is 16-byte aligned
    Side side[2];
    const int64_t* slots;       // device, T: page * S + slot; negative: not stored
    int64_t T, nslots;          // nslots = P * S
    int H, D, S;
    int log2g;
    int* err;
};
cudaError_t launch_append(const AppendArgs& a, bool bf16, cudaStream_t s);

struct AttnArgs {
    const uint16_t* q;          // [B, Tq, Hq, D]
    int64_t q_b, q_t, q_h;
    uint16_t* out;
    int64_t o_b, o_t, o_h;
    int ovec;                   // 1: every 4-element piece of out is 8-byte aligned
    Side k, v;
    const int64_t* pages;       // device, [B, max_pages]
    int64_t pages_row, max_pages, P;
    const int64_t* lengths;     // device, [B]
    int B, Tq, Hq, Hkv, S;
    int rep;                    // Hq / Hkv
    int rows;                   // rep * Tq: query rows per key/value head
    int rtiles;                 // row tiles of 8 * NT rows
    int window;                 // 0: none
    float scale_log2;           // softmax scale * log2(e)
    int fast;                   // 1: 16-token tiles lie inside a page and copy as whole 16-byte pieces
    int scp;                    // not fast: a row's scales (and biases) are one aligned copy of 4, 8 or 16 bytes
    uint32_t k_page, k_slot, v_page, v_slot;   // fast: strides of the codes in bytes
    int unit_slots;             // fast: a unit's tokens past whole pages
    int split;                  // 1: a combine launch follows (an item's units may be shared by CTAs)
    float* part_o;              // [2 * grid][8 * NT][D]
    float* part_ml;             // [2 * grid][8 * NT][2]
    int* err;
};

// How the kernel's tiles go by head size and n tiles: 16-token pieces of a warp's tile (two where the
// registers of up to 8 query rows allow it), tokens of a work unit (a tile per warp, four warps), and
// CTAs that fit an SM.
constexpr int pieces_of(int D, int nt) { return nt == 1 && D <= 128 ? 2 : 1; }
constexpr int unit_tokens(int D, int nt) { return 64 * pieces_of(D, nt); }
constexpr int ctas_per_sm(int D, int nt) { return (D == 256 || nt == 4) ? 2 : 3; }

// A launch's shape, by sizes only: NT (n tiles of 8 query rows), CTAs, workspace bytes.
struct AttnShape {
    int nt;
    int rtiles;
    int grid;
    int split;
    size_t o_floats, ml_floats;
};
AttnShape attn_shape(int64_t B, int64_t rows, int64_t Hkv, int D, int64_t max_tokens);
cudaError_t launch_attention(const AttnArgs& a, const AttnShape& s, int D, int group, bool bf16, cudaStream_t st);

}  // namespace kv
}  // namespace aq
