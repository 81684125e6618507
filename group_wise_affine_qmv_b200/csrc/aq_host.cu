// aq_host.cu -- the C ABI of libaq: argument validation, view resolution,
// batch folding, kernel selection.  No device code lives here.
//
// Batch folding follows the candle "Metal batched matmul" pitfall page
// (section "how to check"): a batch dim folds into rows only when
// stride[i] == stride[i+1] * dims[i+1] holds for it (size-1 dims exempt);
// every other batch dim stays a real batch dim whose offset is computed from
// its own stride -- never from stride[-3] alone, and never by treating a 3D
// input as 2D [shape[-2], K] (transformers issue #47331, root cause).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "aq_internal.h"
#include "kv_cache.h"
#include "moe.h"

#define AQ_API extern "C" __attribute__((visibility("default")))

namespace {

thread_local char g_msg[512] = "";

aq_status fail(aq_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof g_msg, fmt, ap);
    va_end(ap);
    return st;
}

int elem_size(int dt) {
    switch (dt) {
        case AQ_F32: return 4;
        case AQ_BF16: return 2;
        case AQ_F16: return 2;
        case AQ_U32: return 4;
        default: return 0;
    }
}

bool is_half(int dt) { return dt == AQ_BF16 || dt == AQ_F16; }

aq_status check_view(const aq_view* v, const char* name, int min_rank, int max_rank) {
    if (!v) return fail(AQ_ERR_NULL, "%s: view is NULL", name);
    if (v->rank < min_rank || v->rank > max_rank)
        return fail(AQ_ERR_RANK, "%s: rank %d outside [%d, %d]", name, v->rank, min_rank, max_rank);
    if (elem_size(v->dtype) == 0) return fail(AQ_ERR_DTYPE, "%s: unknown dtype %d", name, v->dtype);
    bool empty = false;
    for (int i = 0; i < v->rank; ++i) {
        if (v->shape[i] < 0) return fail(AQ_ERR_SHAPE, "%s: negative extent", name);
        if (v->stride[i] < 0) return fail(AQ_ERR_STRIDE, "%s: negative stride", name);
        if (v->shape[i] == 0) empty = true;
    }
    if (!empty && v->shape[v->rank - 1] > 1 && v->stride[v->rank - 1] != 1)
        return fail(AQ_ERR_STRIDE, "%s: innermost stride must be 1", name);
    if (!empty && !v->data) return fail(AQ_ERR_NULL, "%s: data is NULL", name);
    return AQ_OK;
}

int64_t numel(const aq_view* v) {
    int64_t n = 1;
    for (int i = 0; i < v->rank; ++i) n *= v->shape[i];
    return n;
}

// byte span [lo, hi) touched by a view (0,0 if empty)
void span(const aq_view* v, uintptr_t* lo, uintptr_t* hi) {
    if (numel(v) == 0) { *lo = *hi = 0; return; }
    int64_t last = 0;
    for (int i = 0; i < v->rank; ++i) last += (v->shape[i] - 1) * v->stride[i];
    *lo = (uintptr_t)v->data;
    *hi = *lo + (uintptr_t)((last + 1) * elem_size(v->dtype));
}

bool overlaps(const aq_view* a, const aq_view* b) {
    uintptr_t alo, ahi, blo, bhi;
    span(a, &alo, &ahi);
    span(b, &blo, &bhi);
    if (alo == ahi || blo == bhi) return false;
    return alo < bhi && blo < ahi;
}

// Whether two different indices of an output view reach the same element (a zero stride on a
// dimension of extent > 1, as an expand()ed tensor has, or strides too small for the extents
// inside them): several threads would then race on one element.  Dimensions are visited from the
// smallest stride up; each stride must exceed the largest offset the dimensions below it reach.
bool self_overlapping(const aq_view* v) {
    int idx[4];
    int n = 0;
    for (int i = 0; i < v->rank && i < 4; ++i)   // (ranks above 4 are rejected before)
        if (v->shape[i] > 1) idx[n++] = i;
    for (int j = 1; j < n; ++j)                   // by stride, ascending (at most 4 entries)
        for (int k = j; k > 0 && v->stride[idx[k]] < v->stride[idx[k - 1]]; --k) std::swap(idx[k], idx[k - 1]);
    int64_t reach = 0;
    for (int j = 0; j < n; ++j) {
        const int i = idx[j];
        if (v->stride[i] <= reach) return true;
        reach += (v->shape[i] - 1) * v->stride[i];
    }
    return false;
}

aq_status check_output(const aq_view* v, const char* name) {
    if (numel(v) > 0 && self_overlapping(v))
        return fail(AQ_ERR_OVERLAP, "%s: elements overlap (zero or too small stride)", name);
    return AQ_OK;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

aq_status check_bits_group(int bits, int group) {
    if (!(bits == 2 || bits == 3 || bits == 4 || bits == 5 || bits == 6 || bits == 8))
        return fail(AQ_ERR_BITS, "bits=%d not in {2,3,4,5,6,8}", bits);
    if (!(group == 32 || group == 64 || group == 128))
        return fail(AQ_ERR_GROUP, "group=%d not in {32,64,128}", group);
    return AQ_OK;
}

int log2i(int v) { int r = 0; while ((1 << r) < v) ++r; return r; }

aq_status cuda_fail(cudaError_t e, const char* what) {
    return fail(AQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The kernels are built for sm_100a only.
aq_status check_device() {
    static std::mutex mu;
    static int checked[64] = {0};  // 0 unknown, 1 ok, 2 bad
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= 64) return fail(AQ_ERR_DEVICE, "device ordinal %d", dev);
    std::lock_guard<std::mutex> lk(mu);
    if (checked[dev] == 0) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return fail(AQ_ERR_CUDA, "cannot query device %d", dev);
        checked[dev] = (major == 10 && minor == 0) ? 1 : 2;
    }
    if (checked[dev] != 1) return fail(AQ_ERR_DEVICE, "device %d is not sm_100", dev);
    return AQ_OK;
}

// ---------------------------------------------------------------------------
// view resolution for the linear entry points
// ---------------------------------------------------------------------------

struct Resolved {
    aq_plan plan;
    int64_t w_row, s_row, b_row;
    int xvec;
    bool mma_ok;
    const char* mma_why;
    aq::MmaProblem mp;
};

void fill_mma_problem(const aq_view* x, const aq_view* wq, const aq_view* sc, const aq_view* bi, int group,
                      int bits, const aq_view* y, Resolved* R);

aq_status resolve_linear(const aq_view* x, const aq_view* wq, const aq_view* sc, const aq_view* bi,
                         int group, int bits, const aq_view* y, int force_qmv, Resolved* R) {
    aq_status st;
    if ((st = check_view(x, "x", 1, 4)) != AQ_OK) return st;
    if ((st = check_view(wq, "wq", 2, 4)) != AQ_OK) return st;
    if ((st = check_view(sc, "scales", 2, 4)) != AQ_OK) return st;
    if ((st = check_view(bi, "biases", 2, 4)) != AQ_OK) return st;
    if ((st = check_view(y, "y", 1, 4)) != AQ_OK) return st;
    if ((st = check_output(y, "y")) != AQ_OK) return st;
    if ((st = check_bits_group(bits, group)) != AQ_OK) return st;
    if (!is_half(x->dtype)) return fail(AQ_ERR_DTYPE, "x must be bf16 or f16");
    if (wq->dtype != AQ_U32) return fail(AQ_ERR_DTYPE, "wq must be u32");
    if (sc->dtype != x->dtype || bi->dtype != x->dtype)
        return fail(AQ_ERR_DTYPE, "scales/biases must have x's dtype");
    if (y->dtype != x->dtype && y->dtype != AQ_F32)
        return fail(AQ_ERR_DTYPE, "y must have x's dtype or f32");

    const int rx = x->rank, rw = wq->rank;
    const int64_t K = x->shape[rx - 1];
    const int64_t N = wq->shape[rw - 2];
    if (K % group != 0) return fail(AQ_ERR_GROUP, "K=%lld not a multiple of group=%d", (long long)K, group);
    if (wq->shape[rw - 1] != K * bits / 32)
        return fail(AQ_ERR_SHAPE, "wq last dim %lld != K*bits/32 = %lld", (long long)wq->shape[rw - 1],
                    (long long)(K * bits / 32));
    if (sc->rank != rw || bi->rank != rw) return fail(AQ_ERR_RANK, "scales/biases rank must equal wq rank");
    for (int i = 0; i < rw - 1; ++i)
        if (sc->shape[i] != wq->shape[i] || bi->shape[i] != wq->shape[i])
            return fail(AQ_ERR_SHAPE, "scales/biases leading dims must equal wq's");
    if (sc->shape[rw - 1] != K / group || bi->shape[rw - 1] != K / group)
        return fail(AQ_ERR_SHAPE, "scales/biases last dim must be K/group = %lld", (long long)(K / group));
    if (y->rank != rx) return fail(AQ_ERR_RANK, "y rank must equal x rank");
    for (int i = 0; i < rx - 1; ++i)
        if (y->shape[i] != x->shape[i]) return fail(AQ_ERR_SHAPE, "y.shape[:-1] must equal x.shape[:-1]");
    if (y->shape[rx - 1] != N) return fail(AQ_ERR_SHAPE, "y last dim must be N=%lld", (long long)N);

    const int nxb = rx >= 2 ? rx - 2 : 0;
    const int nwb = rw - 2;
    if (nwb > nxb && numel(wq) > 0) {
        for (int i = 0; i < nwb - nxb; ++i)
            if (wq->shape[i] != 1) return fail(AQ_ERR_SHAPE, "wq has more batch dims than x");
    }

    // alignment of weights (vector loads in every kernel)
    if (numel(wq) > 0) {
        if (!aligned16(wq->data)) return fail(AQ_ERR_ALIGN, "wq data must be 16-byte aligned");
        const int64_t need = (bits == 4 || bits == 8) ? 4 : (bits == 2 || bits == 6) ? 2 : 1;  // words
        if (N > 1 && wq->stride[rw - 2] % need != 0)
            return fail(AQ_ERR_ALIGN, "wq row stride must keep rows %lld-byte aligned", (long long)(need * 4));
    }

    if (numel(x) > 0 || numel(y) > 0) {
        if (overlaps(y, x) || overlaps(y, wq) || overlaps(y, sc) || overlaps(y, bi))
            return fail(AQ_ERR_OVERLAP, "y overlaps an input");
    }

    // ---- batch dims, outer to inner ----
    struct Dim { int64_t size, xs, ys, ws, ss, bs; bool wb; };
    Dim dims[2];
    int nd = 0;
    bool w_batched = false;
    for (int i = 0; i < nxb; ++i) {
        Dim d{};
        d.size = x->shape[i];
        d.xs = x->stride[i];
        d.ys = y->stride[i];
        int j = i - (nxb - nwb);
        if (j >= 0 && wq->shape[j] != 1) {
            if (wq->shape[j] != x->shape[i])
                return fail(AQ_ERR_SHAPE, "wq batch dim %d (%lld) does not match x (%lld)", j,
                            (long long)wq->shape[j], (long long)x->shape[i]);
            d.wb = true;
            d.ws = wq->stride[j];
            d.ss = sc->stride[j];
            d.bs = bi->stride[j];
            if (d.ws % 4 != 0 && bits != 3 && bits != 5)
                return fail(AQ_ERR_ALIGN, "wq batch stride must keep rows 16-byte aligned");
        }
        if (d.size == 1) continue;  // size-1 dims carry no offset
        if (d.wb) w_batched = true;
        dims[nd++] = d;
    }
    int64_t M = rx >= 2 ? x->shape[rx - 2] : 1;
    int64_t xrow = rx >= 2 ? x->stride[rx - 2] : K;
    int64_t yrow = y->rank >= 2 ? y->stride[rx - 2] : N;
    // fold from the innermost batch dim outwards
    int keep = nd;
    for (int i = nd - 1; i >= 0; --i) {
        const Dim& d = dims[i];
        if (d.wb) break;
        if (M == 1) {  // a single row has no row stride of its own: adopt this dim's
            M = d.size;
            xrow = d.xs;
            yrow = d.ys;
            keep = i;
            continue;
        }
        if (d.xs == xrow * M && d.ys == yrow * M) {
            M *= d.size;
            keep = i;
            continue;
        }
        break;
    }
    nd = keep;

    aq_plan& P = R->plan;
    memset(&P, 0, sizeof P);
    P.w_batched = w_batched ? 1 : 0;
    P.M = M;
    P.N = N;
    P.K = K;
    P.nbatch_dims = nd;
    P.batch_shape[0] = P.batch_shape[1] = 1;
    // right-align the remaining batch dims into slots [0,1]
    for (int i = 0; i < nd; ++i) {
        int s = 2 - nd + i;
        P.batch_shape[s] = dims[i].size;
        P.x_batch_stride[s] = dims[i].xs;
        P.y_batch_stride[s] = dims[i].ys;
        P.w_batch_stride[s] = dims[i].ws;
        P.s_batch_stride[s] = dims[i].ss;
        P.b_batch_stride[s] = dims[i].bs;
    }
    P.x_row_stride = xrow;
    P.y_row_stride = yrow;
    P.total_rows = P.batch_shape[0] * P.batch_shape[1] * M;

    R->w_row = wq->stride[rw - 2];
    R->s_row = sc->stride[rw - 2];
    R->b_row = bi->stride[rw - 2];
    // x rows usable with 16-byte vector loads?
    bool xv = aligned16(x->data) && (M <= 1 || xrow % 8 == 0);
    for (int s = 0; s < 2; ++s)
        if (P.batch_shape[s] > 1 && P.x_batch_stride[s] % 8 != 0) xv = false;
    R->xvec = xv ? 1 : 0;

    // ---- regime ----
    R->mma_ok = false;
    R->mma_why = "forced GEMV";
    if (!force_qmv) {
        if (w_batched) R->mma_why = "batched weights take the GEMV kernel";
        else if (M <= 4) R->mma_why = "few rows per launch: GEMV";
        else if (K == 0 || N == 0) R->mma_why = "empty contraction";
        else {
            fill_mma_problem(x, wq, sc, bi, group, bits, y, R);
            aq::MmaProblem& mp = R->mp;
            // scales/biases rows must be contiguous for the tile loads
            if (R->s_row != K / group || R->b_row != K / group) R->mma_why = "scales/biases rows not contiguous";
            else R->mma_ok = aq::mma_supported(mp, &R->mma_why);
        }
    }
    P.regime = R->mma_ok ? AQ_REGIME_MMA : AQ_REGIME_QMV;
    P.kernel = R->mma_ok ? (int32_t)aq::mma_kernel_for(R->mp) : AQ_KERNEL_GEMV;
    P.y_tiles = R->mma_ok && aq::mma_y_tiles(R->mp) ? 1 : 0;
    return AQ_OK;
}

// The tensor-core problem of a resolved call (its plan already filled in).
void fill_mma_problem(const aq_view* x, const aq_view* wq, const aq_view* sc, const aq_view* bi, int group,
                      int bits, const aq_view* y, Resolved* R) {
    const aq_plan& P = R->plan;
    aq::MmaProblem& mp = R->mp;
    memset(&mp, 0, sizeof mp);
    mp.x = x->data;
    mp.y = y->data;
    mp.wq = (const uint32_t*)wq->data;
    mp.scales = sc->data;
    mp.biases = bi->data;
    mp.M = P.M;
    mp.N = P.N;
    mp.K = P.K;
    mp.x_row = P.x_row_stride;
    mp.y_row = P.y_row_stride;
    mp.nb[0] = P.batch_shape[0];
    mp.nb[1] = P.batch_shape[1];
    for (int s = 0; s < 2; ++s) { mp.xb[s] = P.x_batch_stride[s]; mp.yb[s] = P.y_batch_stride[s]; }
    mp.w_row = R->w_row;
    mp.group = group;
    mp.bits = bits;
    mp.xdt = (aq::DT)x->dtype;
    mp.ydt = (aq::DT)y->dtype;
    mp.offsets = nullptr;
}

aq_status run_linear(const aq_view* x, const aq_view* wq, const aq_view* sc, const aq_view* bi, int group,
                     int bits, const aq_view* y, void* stream, int force_qmv) {
    Resolved R;
    aq_status st = resolve_linear(x, wq, sc, bi, group, bits, y, force_qmv, &R);
    if (st != AQ_OK) return st;
    const aq_plan& P = R.plan;
    if (P.total_rows == 0 || P.N == 0) return AQ_OK;  // nothing to write
    if ((st = check_device()) != AQ_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (P.regime == AQ_REGIME_MMA) {
        e = aq::launch_mma(R.mp, s);
        if (e != cudaSuccess) return cuda_fail(e, "tensor-core kernel launch");
        return AQ_OK;
    }
    aq::QmvArgs a;
    memset(&a, 0, sizeof a);
    a.x = x->data;
    a.wq = (const uint32_t*)wq->data;
    a.scales = sc->data;
    a.biases = bi->data;
    a.y = y->data;
    a.x_row = P.x_row_stride;
    a.y_row = P.y_row_stride;
    a.w_row = R.w_row;
    a.s_row = R.s_row;
    a.b_row = R.b_row;
    a.M = P.M;
    a.N = P.N;
    a.K = P.K;
    a.log2g = log2i(group);
    a.xvec = R.xvec;
    a.bshape1 = P.batch_shape[1];
    for (int i = 0; i < 2; ++i) {
        a.xb[i] = P.x_batch_stride[i];
        a.yb[i] = P.y_batch_stride[i];
        a.wb[i] = P.w_batch_stride[i];
        a.sb[i] = P.s_batch_stride[i];
        a.bb[i] = P.b_batch_stride[i];
    }
    const int64_t nbatch = P.batch_shape[0] * P.batch_shape[1];
    if (nbatch > 65535) return fail(AQ_ERR_UNSUPPORTED, "more than 65535 launch batches");
    e = aq::launch_qmv(a, bits, (aq::DT)x->dtype, (aq::DT)y->dtype, nbatch, s);
    if (e != cudaSuccess) return cuda_fail(e, "GEMV kernel launch");
    return AQ_OK;
}

// ---------------------------------------------------------------------------
// fused calls on the warp-level kernel: several W sharing x, gate/up with silu, a residual
// ---------------------------------------------------------------------------

// Resolves matrix j of a fused call as a plain call and checks that it folds to one 2D problem
// (no launch batch dims, unbatched W) the warp-level kernel can take.
aq_status resolve_fused_part(const aq_view* x, const aq_view* wq, const aq_view* sc, const aq_view* bi, int group,
                             int bits, const aq_view* y, const char* what, Resolved* R, bool* warp_ok) {
    aq_status st = resolve_linear(x, wq, sc, bi, group, bits, y, 0, R);
    if (st != AQ_OK) return st;
    if (R->plan.nbatch_dims != 0 || R->plan.w_batched)
        return fail(AQ_ERR_UNSUPPORTED, "%s: x and y must fold into one 2D problem, with an unbatched W", what);
    fill_mma_problem(x, wq, sc, bi, group, bits, y, R);
    const char* why = nullptr;
    *warp_ok = R->plan.total_rows > 0 && R->plan.N > 0 && R->s_row == R->plan.K / group &&
               R->b_row == R->plan.K / group && aq::mma_supported(R->mp, &why) && aq::warp_mma_supported(R->mp);
    return AQ_OK;
}

aq_status launch_fused(aq::MmaProblem& mp, void* stream) {
    aq_status st = check_device();
    if (st != AQ_OK) return st;
    cudaError_t e = aq::launch_warp_mma(mp, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "fused warp-level kernel launch");
    return AQ_OK;
}

aq_status check_quant_views(const aq_view* w, int group, int bits, const aq_view* wq, const aq_view* sc,
                            const aq_view* bi, bool w_is_output) {
    aq_status st;
    if ((st = check_view(w, w_is_output ? "w_out" : "w", 2, 2)) != AQ_OK) return st;
    if ((st = check_view(wq, "wq", 2, 2)) != AQ_OK) return st;
    if ((st = check_view(sc, "scales", 2, 2)) != AQ_OK) return st;
    if ((st = check_view(bi, "biases", 2, 2)) != AQ_OK) return st;
    if ((st = check_bits_group(bits, group)) != AQ_OK) return st;
    if (!(w->dtype == AQ_F32 || is_half(w->dtype))) return fail(AQ_ERR_DTYPE, "w must be f32, bf16 or f16");
    if (wq->dtype != AQ_U32) return fail(AQ_ERR_DTYPE, "wq must be u32");
    if (!is_half(sc->dtype) || bi->dtype != sc->dtype)
        return fail(AQ_ERR_DTYPE, "scales/biases must be bf16 or f16 (same dtype)");
    const int64_t N = w->shape[0], K = w->shape[1];
    if (K % group != 0) return fail(AQ_ERR_GROUP, "K=%lld not a multiple of group=%d", (long long)K, group);
    if (wq->shape[0] != N || wq->shape[1] != K * bits / 32) return fail(AQ_ERR_SHAPE, "wq must be [N, K*bits/32]");
    if (sc->shape[0] != N || sc->shape[1] != K / group || bi->shape[0] != N || bi->shape[1] != K / group)
        return fail(AQ_ERR_SHAPE, "scales/biases must be [N, K/group]");
    if (numel(wq) > 0 && !aligned16(wq->data)) return fail(AQ_ERR_ALIGN, "wq data must be 16-byte aligned");
    const aq_view* out = w_is_output ? w : wq;
    const aq_view* ins[3] = {w_is_output ? wq : w, sc, bi};
    if (w_is_output) {
        if ((st = check_output(w, "w_out")) != AQ_OK) return st;
    } else {
        if ((st = check_output(wq, "wq")) != AQ_OK) return st;
        if ((st = check_output(sc, "scales")) != AQ_OK) return st;
        if ((st = check_output(bi, "biases")) != AQ_OK) return st;
    }
    if (w_is_output) {
        for (const aq_view* v : ins)
            if (overlaps(out, v)) return fail(AQ_ERR_OVERLAP, "w_out overlaps an input");
    } else {
        if (overlaps(wq, w) || overlaps(sc, w) || overlaps(bi, w) || overlaps(wq, sc) || overlaps(wq, bi) ||
            overlaps(sc, bi))
            return fail(AQ_ERR_OVERLAP, "quantize outputs overlap each other or the input");
    }
    return AQ_OK;
}

// ---------------------------------------------------------------------------
// the 4-bit key/value cache
// ---------------------------------------------------------------------------

// Whether two views of the same shape and strides interleave without meeting (the key and value
// halves of one buffer): together they are one more dimension of extent 2, whose stride is their
// distance.
bool interleave(const aq_view* a, const aq_view* b) {
    if (a->rank != b->rank || a->dtype != b->dtype) return false;
    int64_t st[5], n[5];
    int k = 0;
    for (int i = 0; i < a->rank; ++i) {
        if (a->shape[i] != b->shape[i]) return false;
        if (a->shape[i] <= 1) continue;
        if (a->stride[i] != b->stride[i]) return false;
        st[k] = a->stride[i];
        n[k++] = a->shape[i];
    }
    const uintptr_t pa = (uintptr_t)a->data, pb = (uintptr_t)b->data;
    const uintptr_t dist = pa < pb ? pb - pa : pa - pb;
    if (dist % elem_size(a->dtype) != 0) return false;
    st[k] = (int64_t)(dist / elem_size(a->dtype));
    n[k++] = 2;
    for (int i = 1; i < k; ++i)
        for (int j = i; j > 0 && st[j] < st[j - 1]; --j) {
            std::swap(st[j], st[j - 1]);
            std::swap(n[j], n[j - 1]);
        }
    int64_t reach = 0;
    for (int i = 0; i < k; ++i) {
        if (st[i] <= reach) return false;
        reach += (n[i] - 1) * st[i];
    }
    return true;
}

// One side of a cache: [P, H, S, D/8] words with scales and biases [P, H, S, D/G] of dtype dt.
aq_status check_cache_side(const aq_view* wq, const aq_view* sc, const aq_view* bi, const char* name, int dt, int64_t D,
                           int group, aq::kv::Side* out) {
    aq_status st;
    if ((st = check_view(wq, name, 4, 4)) != AQ_OK) return st;
    if ((st = check_view(sc, name, 4, 4)) != AQ_OK) return st;
    if ((st = check_view(bi, name, 4, 4)) != AQ_OK) return st;
    if (wq->dtype != AQ_U32) return fail(AQ_ERR_DTYPE, "%s: codes must be u32", name);
    if (sc->dtype != dt || bi->dtype != dt) return fail(AQ_ERR_DTYPE, "%s: scales/biases must have the activations' dtype", name);
    if (wq->shape[3] != D / 8) return fail(AQ_ERR_SHAPE, "%s: codes must be [pages, heads, slots, D/8 = %lld]", name, (long long)(D / 8));
    for (int i = 0; i < 3; ++i)
        if (sc->shape[i] != wq->shape[i] || bi->shape[i] != wq->shape[i])
            return fail(AQ_ERR_SHAPE, "%s: scales/biases leading dims must equal the codes'", name);
    if (sc->shape[3] != D / group || bi->shape[3] != D / group)
        return fail(AQ_ERR_SHAPE, "%s: scales/biases last dim must be D/group = %lld", name, (long long)(D / group));
    if (numel(wq) > 0) {
        if (!aligned16(wq->data)) return fail(AQ_ERR_ALIGN, "%s: codes must be 16-byte aligned", name);
        for (int i = 0; i < 3; ++i)
            if (wq->shape[i] > 1 && wq->stride[i] % 4 != 0)
                return fail(AQ_ERR_ALIGN, "%s: strides of the codes must keep rows 16-byte aligned", name);
    }
    auto stride = [](const aq_view* v, int i) { return v->shape[i] > 1 ? v->stride[i] : 0; };
    out->wq = (uint32_t*)wq->data;
    out->scales = (uint16_t*)sc->data;
    out->biases = (uint16_t*)bi->data;
    out->w_page = stride(wq, 0); out->w_head = stride(wq, 1); out->w_slot = stride(wq, 2);
    out->s_page = stride(sc, 0); out->s_head = stride(sc, 1); out->s_slot = stride(sc, 2);
    out->b_page = stride(bi, 0); out->b_head = stride(bi, 1); out->b_slot = stride(bi, 2);
    return AQ_OK;
}

aq_status check_cache_bits(int bits, int group) {
    aq_status st = check_bits_group(bits, group);
    if (st != AQ_OK) return st;
    if (bits != 4) return fail(AQ_ERR_UNSUPPORTED, "key/value caches hold 4-bit codes (bits=%d)", bits);
    return AQ_OK;
}

// what the attention call and its workspace query share: shapes of q and the cache
aq_status check_attention_q(const aq_view* q, const aq_view* k_wq, int64_t max_pages) {
    aq_status st;
    if ((st = check_view(q, "q", 4, 4)) != AQ_OK) return st;
    if ((st = check_view(k_wq, "k cache", 4, 4)) != AQ_OK) return st;
    if (!is_half(q->dtype)) return fail(AQ_ERR_DTYPE, "q must be bf16 or f16");
    const int64_t B = q->shape[0], Tq = q->shape[1], Hq = q->shape[2], D = q->shape[3];
    const int64_t H = k_wq->shape[1], S = k_wq->shape[2];
    if (D != 64 && D != 128 && D != 256) return fail(AQ_ERR_UNSUPPORTED, "head size %lld (64, 128 and 256 are supported)", (long long)D);
    if (H < 1 || Hq % H != 0) return fail(AQ_ERR_SHAPE, "%lld query heads are not a multiple of %lld key/value heads", (long long)Hq, (long long)H);
    if (max_pages < 0) return fail(AQ_ERR_SHAPE, "max_pages < 0");
    if (k_wq->shape[0] > 0x7fffffff) return fail(AQ_ERR_UNSUPPORTED, "more than 2^31 pages");
    if (max_pages > (1 << 30) || S > (1 << 30) || max_pages * S > (1 << 30))
        return fail(AQ_ERR_UNSUPPORTED, "more than 2^30 tokens per sequence");
    // work units of 64 tokens, heads and 8 query rows, counted in 32 bits by the kernel
    if (B <= 65535 && H <= 65535 && Hq / H <= (1 << 20) && Tq <= (1 << 20) &&
        (double)B * H * (double)(Hq / H * Tq / 8 + 1) * (double)(max_pages * S / 64 + 2) > 2e9)
        return fail(AQ_ERR_UNSUPPORTED, "more than 2e9 units of 64 tokens and 8 query rows");
    if (B > 65535 || H > 65535 || Hq / H > (1 << 20) || Tq > (1 << 20) || Hq / H * Tq > (1 << 20))
        return fail(AQ_ERR_UNSUPPORTED, "more than 65535 sequences or heads, or 2^20 query rows per key/value head");
    return AQ_OK;
}

aq::kv::AttnShape attention_shape(const aq_view* q, const aq_view* k_wq, int64_t max_pages) {
    const int64_t H = k_wq->shape[1];
    return aq::kv::attn_shape(q->shape[0], q->shape[2] / H * q->shape[1], H, (int)q->shape[3], max_pages * k_wq->shape[2]);
}

// ---------------------------------------------------------------------------
// the mixture-of-experts layer
// ---------------------------------------------------------------------------

bool same_view(const aq_view* a, const aq_view* b) {
    return a->data == b->data && a->dtype == b->dtype && a->rank == b->rank &&
           memcmp(a->shape, b->shape, sizeof(int64_t) * a->rank) == 0 &&
           memcmp(a->stride, b->stride, sizeof(int64_t) * a->rank) == 0;
}

// One expert bank: [E, rows, K*bits/32] words with dense scale/bias rows [E, rows, K/group] of dtype dt.
aq_status check_bank(const aq_view* wq, const aq_view* sc, const aq_view* bi, const char* name, int dt, int64_t E, int64_t rows,
                     int64_t K, int group, int bits, aq::moe::Bank* out) {
    aq_status st;
    if ((st = check_view(wq, name, 3, 3)) != AQ_OK) return st;
    if ((st = check_view(sc, name, 3, 3)) != AQ_OK) return st;
    if ((st = check_view(bi, name, 3, 3)) != AQ_OK) return st;
    if (wq->dtype != AQ_U32) return fail(AQ_ERR_DTYPE, "%s: codes must be u32", name);
    if (sc->dtype != dt || bi->dtype != dt) return fail(AQ_ERR_DTYPE, "%s: scales/biases must have x's dtype", name);
    if (K % group != 0) return fail(AQ_ERR_GROUP, "%s: %lld columns not a multiple of group=%d", name, (long long)K, group);
    const int64_t kg = K / group;
    if (wq->shape[0] != E || wq->shape[1] != rows || wq->shape[2] != K * bits / 32)
        return fail(AQ_ERR_SHAPE, "%s: codes must be [%lld, %lld, %lld]", name, (long long)E, (long long)rows, (long long)(K * bits / 32));
    for (const aq_view* v : {sc, bi}) {
        if (v->shape[0] != E || v->shape[1] != rows || v->shape[2] != kg)
            return fail(AQ_ERR_SHAPE, "%s: scales/biases must be [%lld, %lld, %lld]", name, (long long)E, (long long)rows, (long long)kg);
        if (rows > 1 && v->stride[1] != kg) return fail(AQ_ERR_UNSUPPORTED, "%s: scale/bias rows must be contiguous", name);
    }
    if (numel(wq) > 0 && (!aligned16(wq->data) || (E > 1 && wq->stride[0] % 4 != 0) || (rows > 1 && wq->stride[1] % 4 != 0)))
        return fail(AQ_ERR_ALIGN, "%s: rows of codes must be 16-byte aligned", name);
    out->wq = (const uint32_t*)wq->data;
    out->scales = (const uint16_t*)sc->data;
    out->biases = (const uint16_t*)bi->data;
    out->w_row = rows > 1 ? wq->stride[1] : 0;
    out->w_exp = E > 1 ? wq->stride[0] : 0;
    out->s_exp = E > 1 ? sc->stride[0] : 0;
    out->b_exp = E > 1 ? bi->stride[0] : 0;
    // scales of 64 bytes (512 / bits codes) of a row as one aligned copy; a single one comes with a
    // neighbour, so rows have to hold an even number
    int64_t per = 512 / bits / group;
    if (per < 2) per = 2;
    out->svec = kg % per == 0 && (uintptr_t)sc->data % (2 * per) == 0 && (uintptr_t)bi->data % (2 * per) == 0 &&
                out->s_exp % per == 0 && out->b_exp % per == 0;
    out->blk = out->svec && aligned16(sc->data) && aligned16(bi->data) && out->s_exp % 8 == 0 && out->b_exp % 8 == 0;
    return AQ_OK;
}

aq_status check_moe_sizes(int64_t T, int top_k, int64_t K, int64_t N) {
    if (T > aq::moe::MAX_TOKENS)
        return fail(AQ_ERR_UNSUPPORTED, "%lld tokens (up to %d; aq_qmm_t_grouped takes more)", (long long)T, aq::moe::MAX_TOKENS);
    if (top_k < 1 || top_k > aq::moe::MAX_TOPK) return fail(AQ_ERR_UNSUPPORTED, "top_k=%d (1..%d)", top_k, aq::moe::MAX_TOPK);
    if (K < 0 || K > (1 << 20) || N < 0 || N > (1 << 20))
        return fail(AQ_ERR_UNSUPPORTED, "model size %lld, experts of %lld rows (up to 2^20)", (long long)K, (long long)N);
    return AQ_OK;
}

}  // namespace

// ===========================================================================
// exported C ABI
// ===========================================================================

AQ_API const char* aq_status_string(aq_status s) {
    switch (s) {
        case AQ_OK: return "AQ_OK";
        case AQ_ERR_NULL: return "AQ_ERR_NULL";
        case AQ_ERR_DTYPE: return "AQ_ERR_DTYPE";
        case AQ_ERR_RANK: return "AQ_ERR_RANK";
        case AQ_ERR_SHAPE: return "AQ_ERR_SHAPE";
        case AQ_ERR_STRIDE: return "AQ_ERR_STRIDE";
        case AQ_ERR_BITS: return "AQ_ERR_BITS";
        case AQ_ERR_GROUP: return "AQ_ERR_GROUP";
        case AQ_ERR_ALIGN: return "AQ_ERR_ALIGN";
        case AQ_ERR_UNSUPPORTED: return "AQ_ERR_UNSUPPORTED";
        case AQ_ERR_OVERLAP: return "AQ_ERR_OVERLAP";
        case AQ_ERR_CUDA: return "AQ_ERR_CUDA";
        case AQ_ERR_DEVICE: return "AQ_ERR_DEVICE";
        case AQ_ERR_TIMEOUT: return "AQ_ERR_TIMEOUT";
        case AQ_ERR_INDEX: return "AQ_ERR_INDEX";
    }
    return "AQ_ERR_UNKNOWN";
}

AQ_API const char* aq_last_error_message(void) { return g_msg; }

AQ_API int aq_version(void) { return 100; }

AQ_API aq_status aq_plan_linear(const aq_view* x, const aq_view* wq, const aq_view* scales,
                                const aq_view* biases, int group, int bits, const aq_view* y, int force_qmv,
                                aq_plan* out) {
    g_msg[0] = 0;
    if (!out) return fail(AQ_ERR_NULL, "plan output is NULL");
    Resolved R;
    aq_status st = resolve_linear(x, wq, scales, biases, group, bits, y, force_qmv, &R);
    if (st != AQ_OK) return st;
    *out = R.plan;
    if (R.plan.regime == AQ_REGIME_QMV && R.mma_why) snprintf(g_msg, sizeof g_msg, "%s", R.mma_why);
    return AQ_OK;
}

AQ_API aq_status aq_qmm_t(const aq_view* x, const aq_view* wq, const aq_view* scales, const aq_view* biases,
                          int group, int bits, const aq_view* y, void* stream) {
    g_msg[0] = 0;
    return run_linear(x, wq, scales, biases, group, bits, y, stream, 0);
}

AQ_API aq_status aq_qmv(const aq_view* x, const aq_view* wq, const aq_view* scales, const aq_view* biases,
                        int group, int bits, const aq_view* y, void* stream) {
    g_msg[0] = 0;
    return run_linear(x, wq, scales, biases, group, bits, y, stream, 1);
}

AQ_API aq_status aq_quantize(const aq_view* w, int group, int bits, const aq_view* wq, const aq_view* scales,
                             const aq_view* biases, void* stream) {
    g_msg[0] = 0;
    aq_status st = check_quant_views(w, group, bits, wq, scales, biases, false);
    if (st != AQ_OK) return st;
    if (numel(w) == 0) return AQ_OK;
    if ((st = check_device()) != AQ_OK) return st;
    aq::QuantArgs a;
    memset(&a, 0, sizeof a);
    a.w = w->data;
    a.wq = (uint32_t*)wq->data;
    a.scales = scales->data;
    a.biases = biases->data;
    a.w_row = w->stride[0];
    a.wq_row = wq->stride[0];
    a.s_row = scales->stride[0];
    a.b_row = biases->stride[0];
    a.N = w->shape[0];
    a.K = w->shape[1];
    a.group = group;
    a.bits = bits;
    cudaError_t e = aq::launch_quantize(a, (aq::DT)w->dtype, (aq::DT)scales->dtype, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "quantize launch");
    return AQ_OK;
}

AQ_API aq_status aq_dequantize(const aq_view* wq, const aq_view* scales, const aq_view* biases, int group,
                               int bits, const aq_view* w_out, void* stream) {
    g_msg[0] = 0;
    aq_status st = check_quant_views(w_out, group, bits, wq, scales, biases, true);
    if (st != AQ_OK) return st;
    if (numel(w_out) == 0) return AQ_OK;
    if ((st = check_device()) != AQ_OK) return st;
    aq::QuantArgs a;
    memset(&a, 0, sizeof a);
    a.w = w_out->data;
    a.wq = (uint32_t*)wq->data;
    a.scales = scales->data;
    a.biases = biases->data;
    a.w_row = w_out->stride[0];
    a.wq_row = wq->stride[0];
    a.s_row = scales->stride[0];
    a.b_row = biases->stride[0];
    a.N = w_out->shape[0];
    a.K = w_out->shape[1];
    a.group = group;
    a.bits = bits;
    cudaError_t e = aq::launch_dequantize(a, (aq::DT)w_out->dtype, (aq::DT)scales->dtype, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "dequantize launch");
    return AQ_OK;
}

AQ_API aq_status aq_qmm_t_grouped(const aq_view* x_sorted, const int64_t* offsets, int n_experts,
                                  const aq_view* wq_bank, const aq_view* s_bank, const aq_view* b_bank, int group,
                                  int bits, const aq_view* y_sorted, void* stream) {
    g_msg[0] = 0;
    aq_status st;
    if ((st = check_view(x_sorted, "x_sorted", 2, 2)) != AQ_OK) return st;
    if ((st = check_view(wq_bank, "wq_bank", 3, 3)) != AQ_OK) return st;
    if ((st = check_view(s_bank, "s_bank", 3, 3)) != AQ_OK) return st;
    if ((st = check_view(b_bank, "b_bank", 3, 3)) != AQ_OK) return st;
    if ((st = check_view(y_sorted, "y_sorted", 2, 2)) != AQ_OK) return st;
    if ((st = check_output(y_sorted, "y_sorted")) != AQ_OK) return st;
    if ((st = check_bits_group(bits, group)) != AQ_OK) return st;
    if (!offsets) return fail(AQ_ERR_NULL, "offsets is NULL");
    if (n_experts <= 0 || wq_bank->shape[0] != n_experts || s_bank->shape[0] != n_experts ||
        b_bank->shape[0] != n_experts)
        return fail(AQ_ERR_SHAPE, "bank leading dim must equal n_experts");
    if (!is_half(x_sorted->dtype)) return fail(AQ_ERR_DTYPE, "x_sorted must be bf16 or f16");
    if (wq_bank->dtype != AQ_U32) return fail(AQ_ERR_DTYPE, "wq_bank must be u32");
    if (s_bank->dtype != x_sorted->dtype || b_bank->dtype != x_sorted->dtype)
        return fail(AQ_ERR_DTYPE, "scale/bias banks must have x's dtype");
    if (y_sorted->dtype != x_sorted->dtype && y_sorted->dtype != AQ_F32)
        return fail(AQ_ERR_DTYPE, "y_sorted must have x's dtype or f32");
    const int64_t T = x_sorted->shape[0], K = x_sorted->shape[1], N = wq_bank->shape[1];
    if (K % group != 0) return fail(AQ_ERR_GROUP, "K not a multiple of group");
    if (wq_bank->shape[2] != K * bits / 32) return fail(AQ_ERR_SHAPE, "wq_bank last dim must be K*bits/32");
    if (s_bank->shape[1] != N || b_bank->shape[1] != N || s_bank->shape[2] != K / group ||
        b_bank->shape[2] != K / group)
        return fail(AQ_ERR_SHAPE, "scale/bias banks must be [E, N, K/group]");
    if (y_sorted->shape[0] != T || y_sorted->shape[1] != N) return fail(AQ_ERR_SHAPE, "y_sorted must be [T, N]");
    if (numel(wq_bank) > 0 && !aligned16(wq_bank->data)) return fail(AQ_ERR_ALIGN, "wq_bank must be 16-byte aligned");
    if (overlaps(y_sorted, x_sorted) || overlaps(y_sorted, wq_bank) || overlaps(y_sorted, s_bank) ||
        overlaps(y_sorted, b_bank))
        return fail(AQ_ERR_OVERLAP, "y_sorted overlaps an input");
    if (T == 0 || N == 0) return AQ_OK;
    if ((st = check_device()) != AQ_OK) return st;
    aq::MmaProblem mp;
    memset(&mp, 0, sizeof mp);
    mp.x = x_sorted->data;
    mp.y = y_sorted->data;
    mp.wq = (const uint32_t*)wq_bank->data;
    mp.scales = s_bank->data;
    mp.biases = b_bank->data;
    mp.M = T;
    mp.N = N;
    mp.K = K;
    mp.x_row = x_sorted->stride[0];
    mp.y_row = y_sorted->stride[0];
    mp.nb[0] = mp.nb[1] = 1;
    mp.w_row = wq_bank->stride[1];
    mp.group = group;
    mp.bits = bits;
    mp.xdt = (aq::DT)x_sorted->dtype;
    mp.ydt = (aq::DT)y_sorted->dtype;
    mp.offsets = offsets;
    mp.n_experts = n_experts;
    mp.w_expert = wq_bank->stride[0];
    mp.s_expert = s_bank->stride[0];
    mp.b_expert = b_bank->stride[0];
    if (s_bank->stride[1] != K / group || b_bank->stride[1] != K / group)
        return fail(AQ_ERR_UNSUPPORTED, "scale/bias bank rows must be contiguous");
    const char* why = nullptr;
    if (!aq::mma_supported(mp, &why)) return fail(AQ_ERR_UNSUPPORTED, "grouped kernel: %s", why);
    cudaError_t e = aq::launch_mma(mp, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "grouped kernel launch");
    return AQ_OK;
}

AQ_API aq_status aq_device_error(void* stream) {
    g_msg[0] = 0;
    int v = 0;
    cudaError_t e = aq::read_and_clear_device_error(&v, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "reading the device error word");
    if (v & aq::DEVERR_TIMEOUT) {
        static const struct { int bit; const char* name; } at[] = {
            {aq::DEVERR_AT_WARP_X, "warp-level kernel x staging"}, {aq::DEVERR_AT_WARP_SB, "warp-level kernel scale/bias staging"},
            {aq::DEVERR_AT_WARP_W, "warp-level kernel W ring"},
            {aq::DEVERR_AT_TC_WFREE, "small-M W producer (expanders)"}, {aq::DEVERR_AT_TC_XFREE, "small-M x producer (MMA commit)"},
            {aq::DEVERR_AT_TC_XFULL, "small-M MMA issuer (x copy)"}, {aq::DEVERR_AT_TC_AFULL, "small-M MMA issuer (expanders)"},
            {aq::DEVERR_AT_TC_DFREE, "small-M MMA issuer (folds)"}, {aq::DEVERR_AT_TC_WFULL, "small-M expanders (W copy)"},
            {aq::DEVERR_AT_TC_SDONE_E, "small-M expanders (MMA commit)"}, {aq::DEVERR_AT_TC_SDONE_F, "small-M folds (MMA commit)"},
            {aq::DEVERR_AT_TC_FOLD, "small-M folds (folds, x or cluster)"},
            {aq::DEVERR_AT_PF_W, "prefill W producer"}, {aq::DEVERR_AT_PF_X, "prefill x producer"},
            {aq::DEVERR_AT_PF_MMA, "prefill MMA issuer"}, {aq::DEVERR_AT_PF_EXP, "prefill expanders"},
            {aq::DEVERR_AT_PF_FOLD, "prefill folds"}, {aq::DEVERR_AT_CHECK, "bounded-wait self-check"}};
        char where[480];
        where[0] = 0;
        for (const auto& a : at)
            if (v & a.bit) {
                if (where[0]) strncat(where, ", ", sizeof where - strlen(where) - 1);
                strncat(where, a.name, sizeof where - strlen(where) - 1);
            }
        return fail(AQ_ERR_TIMEOUT, "a kernel's bounded wait expired (code %d; at: %s)", v, where[0] ? where : "unrecorded");
    }
    if (v & aq::DEVERR_INDEX) return fail(AQ_ERR_INDEX, "a row id was outside the table (code %d)", v);
    if (v != 0) return fail(AQ_ERR_CUDA, "unknown device error code %d", v);
    return AQ_OK;
}

AQ_API aq_status aq_qmm_t_multi(const aq_view* x, int n, const aq_view* const* wq, const aq_view* const* scales,
                                const aq_view* const* biases, int group, int bits, float rms_eps,
                                const aq_view* const* y, void* stream) {
    g_msg[0] = 0;
    if (n < 1 || n > 3) return fail(AQ_ERR_UNSUPPORTED, "n=%d matrices (1..3 supported)", n);
    if (!(rms_eps >= 0.0f)) return fail(AQ_ERR_SHAPE, "rms_eps must be >= 0");
    if (!wq || !scales || !biases || !y) return fail(AQ_ERR_NULL, "NULL array of views");
    Resolved R[3];
    bool all_warp = true;
    for (int j = 0; j < n; ++j) {
        aq_status st = resolve_linear(x, wq[j], scales[j], biases[j], group, bits, y[j], 0, &R[j]);
        if (st != AQ_OK) return st;
    }
    // no output may overlap another output or another matrix's inputs
    for (int j = 0; j < n; ++j)
        for (int k = 0; k < n; ++k) {
            if (j == k) continue;
            if (overlaps(y[j], y[k]) || overlaps(y[j], wq[k]) || overlaps(y[j], scales[k]) || overlaps(y[j], biases[k]))
                return fail(AQ_ERR_OVERLAP, "y[%d] overlaps an input or output of matrix %d", j, k);
        }
    if (R[0].plan.total_rows == 0) return AQ_OK;
    for (int j = 0; j < n && all_warp; ++j) {
        bool ok = false;
        aq_status st = resolve_fused_part(x, wq[j], scales[j], biases[j], group, bits, y[j], "aq_qmm_t_multi", &R[j],
                                          &ok);
        if (st != AQ_OK) ok = false;
        all_warp = ok && R[j].plan.M == R[0].plan.M && R[j].plan.x_row_stride == R[0].plan.x_row_stride;
    }
    if (rms_eps > 0.0f && !all_warp)
        return fail(AQ_ERR_UNSUPPORTED, "an RMS-normalised input needs the warp-level kernel (up to 32 rows, "
                                        "2/4/8-bit codes, 16-byte aligned rows)");
    if (!all_warp || (n == 1 && rms_eps == 0.0f)) {
        // one plain call per matrix, in order, on the same stream
        for (int j = 0; j < n; ++j) {
            aq_status st = run_linear(x, wq[j], scales[j], biases[j], group, bits, y[j], stream, 0);
            if (st != AQ_OK) return st;
        }
        return AQ_OK;
    }
    aq::MmaProblem mp = R[0].mp;
    mp.nseg = n;
    mp.rms_eps = rms_eps;
    for (int j = 0; j < n; ++j) {
        mp.seg_wq[j] = R[j].mp.wq;
        mp.seg_scales[j] = R[j].mp.scales;
        mp.seg_biases[j] = R[j].mp.biases;
        mp.seg_y[j] = R[j].mp.y;
        mp.seg_N[j] = R[j].mp.N;
        mp.seg_w_row[j] = R[j].mp.w_row;
        mp.seg_y_row[j] = R[j].mp.y_row;
    }
    if (!aq::warp_mma_supported(mp)) return fail(AQ_ERR_UNSUPPORTED, "fused projections: too many row blocks");
    return launch_fused(mp, stream);
}

AQ_API aq_status aq_qmm_t_swiglu(const aq_view* x, const aq_view* wq_gate, const aq_view* s_gate,
                                 const aq_view* b_gate, const aq_view* wq_up, const aq_view* s_up,
                                 const aq_view* b_up, int group, int bits, float rms_eps, const aq_view* y,
                                 void* stream) {
    g_msg[0] = 0;
    if (!(rms_eps >= 0.0f)) return fail(AQ_ERR_SHAPE, "rms_eps must be >= 0");
    Resolved Rg, Ru;
    bool okg = false, oku = false;
    aq_status st = resolve_fused_part(x, wq_gate, s_gate, b_gate, group, bits, y, "aq_qmm_t_swiglu", &Rg, &okg);
    if (st != AQ_OK) return st;
    st = resolve_fused_part(x, wq_up, s_up, b_up, group, bits, y, "aq_qmm_t_swiglu", &Ru, &oku);
    if (st != AQ_OK) return st;
    if (Ru.plan.N != Rg.plan.N) return fail(AQ_ERR_SHAPE, "gate and up matrices must have the same N");
    if (Rg.plan.total_rows == 0 || Rg.plan.N == 0) return AQ_OK;
    if (!okg || !oku)
        return fail(AQ_ERR_UNSUPPORTED,
                    "aq_qmm_t_swiglu runs on the warp-level kernel only (up to 32 rows, 2/4/8-bit codes, "
                    "16-byte aligned rows)");
    aq::MmaProblem mp = Rg.mp;
    mp.nseg = 2;
    mp.glu = 1;
    mp.rms_eps = rms_eps;
    const Resolved* parts[2] = {&Rg, &Ru};
    for (int j = 0; j < 2; ++j) {
        mp.seg_wq[j] = parts[j]->mp.wq;
        mp.seg_scales[j] = parts[j]->mp.scales;
        mp.seg_biases[j] = parts[j]->mp.biases;
        mp.seg_y[j] = Rg.mp.y;
        mp.seg_N[j] = parts[j]->mp.N;
        mp.seg_w_row[j] = parts[j]->mp.w_row;
        mp.seg_y_row[j] = Rg.mp.y_row;
    }
    if (!aq::warp_mma_supported(mp)) return fail(AQ_ERR_UNSUPPORTED, "gate/up: too many row blocks");
    return launch_fused(mp, stream);
}

AQ_API aq_status aq_qmm_t_residual(const aq_view* x, const aq_view* wq, const aq_view* scales,
                                   const aq_view* biases, int group, int bits, const aq_view* r, const aq_view* y,
                                   void* stream) {
    g_msg[0] = 0;
    Resolved R, Rr;
    bool ok = false, okr = false;
    aq_status st = resolve_fused_part(x, wq, scales, biases, group, bits, y, "aq_qmm_t_residual", &R, &ok);
    if (st != AQ_OK) return st;
    if ((st = check_view(r, "r", 1, 4)) != AQ_OK) return st;
    if (r->dtype != y->dtype) return fail(AQ_ERR_DTYPE, "r must have y's dtype");
    // r has y's shape and folds the same way; it is read as an input, so it may be y itself
    // (the same view: each element is read and then written by the same thread) but must not
    // overlap y otherwise, nor the other inputs
    const bool same = r->data == y->data && r->rank == y->rank &&
                      memcmp(r->shape, y->shape, sizeof(int64_t) * y->rank) == 0 &&
                      memcmp(r->stride, y->stride, sizeof(int64_t) * y->rank) == 0;
    if (!same) {
        st = resolve_fused_part(x, wq, scales, biases, group, bits, r, "aq_qmm_t_residual (r)", &Rr, &okr);
        if (st != AQ_OK) return st;
        if (overlaps(r, y)) return fail(AQ_ERR_OVERLAP, "r overlaps y (other than being the same view)");
    } else {
        Rr = R;
    }
    if (R.plan.total_rows == 0 || R.plan.N == 0) return AQ_OK;
    if (!ok)
        return fail(AQ_ERR_UNSUPPORTED,
                    "aq_qmm_t_residual runs on the warp-level kernel only (up to 32 rows, 2/4/8-bit codes, "
                    "16-byte aligned rows)");
    aq::MmaProblem mp = R.mp;
    mp.r = r->data;
    mp.r_row = Rr.plan.y_row_stride;
    return launch_fused(mp, stream);
}

AQ_API aq_status aq_dequantize_rows(const aq_view* wq, const aq_view* scales, const aq_view* biases, int group,
                                    int bits, const int64_t* ids, int64_t n_ids, const aq_view* out,
                                    void* stream) {
    g_msg[0] = 0;
    aq_status st;
    if ((st = check_view(out, "out", 2, 2)) != AQ_OK) return st;
    if (n_ids < 0) return fail(AQ_ERR_SHAPE, "n_ids < 0");
    if (out->shape[0] != n_ids) return fail(AQ_ERR_SHAPE, "out must have n_ids rows");
    if ((st = check_output(out, "out")) != AQ_OK) return st;
    if ((st = check_view(wq, "wq", 2, 2)) != AQ_OK) return st;
    if ((st = check_view(scales, "scales", 2, 2)) != AQ_OK) return st;
    if ((st = check_view(biases, "biases", 2, 2)) != AQ_OK) return st;
    if ((st = check_bits_group(bits, group)) != AQ_OK) return st;
    if (!(out->dtype == AQ_F32 || is_half(out->dtype))) return fail(AQ_ERR_DTYPE, "out must be f32, bf16 or f16");
    if (wq->dtype != AQ_U32) return fail(AQ_ERR_DTYPE, "wq must be u32");
    if (!is_half(scales->dtype) || biases->dtype != scales->dtype)
        return fail(AQ_ERR_DTYPE, "scales/biases must be bf16 or f16 (same dtype)");
    const int64_t V = wq->shape[0], K = out->shape[1];
    if (K % group != 0) return fail(AQ_ERR_GROUP, "K=%lld not a multiple of group=%d", (long long)K, group);
    if (wq->shape[1] != K * bits / 32) return fail(AQ_ERR_SHAPE, "wq must be [V, K*bits/32]");
    if (scales->shape[0] != V || scales->shape[1] != K / group || biases->shape[0] != V ||
        biases->shape[1] != K / group)
        return fail(AQ_ERR_SHAPE, "scales/biases must be [V, K/group]");
    if (numel(wq) > 0 && !aligned16(wq->data)) return fail(AQ_ERR_ALIGN, "wq data must be 16-byte aligned");
    if (overlaps(out, wq) || overlaps(out, scales) || overlaps(out, biases))
        return fail(AQ_ERR_OVERLAP, "out overlaps the table");
    if (n_ids == 0 || out->shape[1] == 0) return AQ_OK;
    if (!ids) return fail(AQ_ERR_NULL, "ids is NULL");
    if ((st = check_device()) != AQ_OK) return st;
    aq::QuantArgs a;
    memset(&a, 0, sizeof a);
    a.w = out->data;
    a.wq = (uint32_t*)wq->data;
    a.scales = scales->data;
    a.biases = biases->data;
    a.w_row = out->stride[0];
    a.wq_row = wq->stride[0];
    a.s_row = scales->stride[0];
    a.b_row = biases->stride[0];
    a.N = n_ids;
    a.K = out->shape[1];
    a.group = group;
    a.bits = bits;
    a.ids = ids;
    a.V = wq->shape[0];
    cudaError_t e = aq::device_error_ptr(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = aq::launch_dequantize(a, (aq::DT)out->dtype, (aq::DT)scales->dtype, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "row gather launch");
    return AQ_OK;
}

AQ_API aq_status aq_qmv_gathered(const aq_view* x, const int64_t* x_ids, const int64_t* w_ids, int64_t n_rows,
                                 const aq_view* wq_bank, const aq_view* s_bank, const aq_view* b_bank, int group,
                                 int bits, const aq_view* y, void* stream) {
    g_msg[0] = 0;
    aq_status st;
    if ((st = check_view(x, "x", 2, 2)) != AQ_OK) return st;
    if ((st = check_view(wq_bank, "wq_bank", 3, 3)) != AQ_OK) return st;
    if ((st = check_view(s_bank, "s_bank", 3, 3)) != AQ_OK) return st;
    if ((st = check_view(b_bank, "b_bank", 3, 3)) != AQ_OK) return st;
    if ((st = check_view(y, "y", 2, 2)) != AQ_OK) return st;
    if ((st = check_output(y, "y")) != AQ_OK) return st;
    if ((st = check_bits_group(bits, group)) != AQ_OK) return st;
    if (!is_half(x->dtype)) return fail(AQ_ERR_DTYPE, "x must be bf16 or f16");
    if (wq_bank->dtype != AQ_U32) return fail(AQ_ERR_DTYPE, "wq_bank must be u32");
    if (s_bank->dtype != x->dtype || b_bank->dtype != x->dtype)
        return fail(AQ_ERR_DTYPE, "scale/bias banks must have x's dtype");
    if (y->dtype != x->dtype && y->dtype != AQ_F32) return fail(AQ_ERR_DTYPE, "y must have x's dtype or f32");
    const int64_t T = x->shape[0], K = x->shape[1], E = wq_bank->shape[0], N = wq_bank->shape[1];
    if (n_rows < 0) return fail(AQ_ERR_SHAPE, "n_rows < 0");
    if (K % group != 0) return fail(AQ_ERR_GROUP, "K not a multiple of group");
    if (wq_bank->shape[2] != K * bits / 32) return fail(AQ_ERR_SHAPE, "wq_bank last dim must be K*bits/32");
    if (s_bank->shape[0] != E || b_bank->shape[0] != E || s_bank->shape[1] != N || b_bank->shape[1] != N ||
        s_bank->shape[2] != K / group || b_bank->shape[2] != K / group)
        return fail(AQ_ERR_SHAPE, "scale/bias banks must be [E, N, K/group]");
    if (y->shape[0] != n_rows || y->shape[1] != N) return fail(AQ_ERR_SHAPE, "y must be [n_rows, N]");
    if (numel(wq_bank) > 0) {
        const int64_t need = (bits == 4 || bits == 8) ? 4 : (bits == 2 || bits == 6) ? 2 : 1;  // words
        if (!aligned16(wq_bank->data) || wq_bank->stride[0] % need != 0 || (N > 1 && wq_bank->stride[1] % need != 0))
            return fail(AQ_ERR_ALIGN, "wq_bank rows must be %lld-byte aligned", (long long)(need * 4));
    }
    if (overlaps(y, x) || overlaps(y, wq_bank) || overlaps(y, s_bank) || overlaps(y, b_bank))
        return fail(AQ_ERR_OVERLAP, "y overlaps an input");
    if (n_rows == 0 || N == 0) return AQ_OK;
    if (!x_ids || !w_ids) return fail(AQ_ERR_NULL, "x_ids / w_ids is NULL");
    if (n_rows > 65535) return fail(AQ_ERR_UNSUPPORTED, "more than 65535 gathered rows per call");
    if ((st = check_device()) != AQ_OK) return st;
    aq::QmvArgs a;
    memset(&a, 0, sizeof a);
    a.x = x->data;
    a.wq = (const uint32_t*)wq_bank->data;
    a.scales = s_bank->data;
    a.biases = b_bank->data;
    a.y = y->data;
    a.x_row = x->stride[0];
    a.y_row = y->stride[0];
    a.w_row = wq_bank->stride[1];
    a.s_row = s_bank->stride[1];
    a.b_row = b_bank->stride[1];
    a.M = 1;
    a.N = N;
    a.K = K;
    a.log2g = log2i(group);
    a.xvec = (aligned16(x->data) && (T <= 1 || x->stride[0] % 8 == 0)) ? 1 : 0;
    a.bshape1 = 1;
    a.xb[0] = x->stride[0];
    a.yb[0] = y->stride[0];
    a.wb[0] = wq_bank->stride[0];
    a.sb[0] = s_bank->stride[0];
    a.bb[0] = b_bank->stride[0];
    a.x_ids = x_ids;
    a.w_ids = w_ids;
    a.x_rows = T;
    a.w_entries = E;
    cudaError_t e = aq::device_error_ptr(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = aq::launch_qmv(a, bits, (aq::DT)x->dtype, (aq::DT)y->dtype, n_rows, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "gathered GEMV launch");
    return AQ_OK;
}

AQ_API aq_status aq_check_bounded_wait(uint64_t budget_ns, void* stream) {
    g_msg[0] = 0;
    if (budget_ns == 0 || budget_ns > 1000000000ull) return fail(AQ_ERR_SHAPE, "budget_ns must be in (0, 1e9]");
    aq_status st = check_device();
    if (st != AQ_OK) return st;
    cudaError_t e = aq::launch_bounded_wait_check(budget_ns, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "bounded-wait check launch");
    return AQ_OK;
}

AQ_API aq_status aq_kv_append(const aq_view* k, const aq_view* v, const int64_t* slots, int group, int bits,
                              const aq_view* k_wq, const aq_view* k_scales, const aq_view* k_biases, const aq_view* v_wq,
                              const aq_view* v_scales, const aq_view* v_biases, const aq_view* k_out, const aq_view* v_out,
                              void* stream) {
    g_msg[0] = 0;
    aq_status st;
    if ((st = check_view(k, "k", 3, 3)) != AQ_OK) return st;
    if ((st = check_view(v, "v", 3, 3)) != AQ_OK) return st;
    if ((st = check_cache_bits(bits, group)) != AQ_OK) return st;
    if (!is_half(k->dtype) || v->dtype != k->dtype) return fail(AQ_ERR_DTYPE, "k and v must be bf16 or f16 (same dtype)");
    const int64_t T = k->shape[0], H = k->shape[1], D = k->shape[2];
    if (v->shape[0] != T || v->shape[1] != H || v->shape[2] != D) return fail(AQ_ERR_SHAPE, "v must have k's shape");
    if (D % group != 0) return fail(AQ_ERR_GROUP, "head size %lld not a multiple of group=%d", (long long)D, group);
    aq::kv::AppendArgs a;
    memset(&a, 0, sizeof a);
    if ((st = check_cache_side(k_wq, k_scales, k_biases, "k cache", k->dtype, D, group, &a.side[0])) != AQ_OK) return st;
    if ((st = check_cache_side(v_wq, v_scales, v_biases, "v cache", k->dtype, D, group, &a.side[1])) != AQ_OK) return st;
    if (k_wq->shape[1] != H) return fail(AQ_ERR_SHAPE, "the cache must have k's %lld heads", (long long)H);
    for (int i = 0; i < 3; ++i)
        if (v_wq->shape[i] != k_wq->shape[i]) return fail(AQ_ERR_SHAPE, "the v cache must have the k cache's shape");
    const aq_view* outs[8] = {k_wq, k_scales, k_biases, v_wq, v_scales, v_biases, k_out, v_out};
    const aq_view* ins[2] = {k, v};
    for (int j = 0; j < 2; ++j) {
        const aq_view* o = outs[6 + j];
        if (!o) continue;
        if ((st = check_view(o, j ? "v_out" : "k_out", 3, 3)) != AQ_OK) return st;
        if (o->dtype != k->dtype) return fail(AQ_ERR_DTYPE, "k_out/v_out must have k's dtype");
        if (o->shape[0] != T || o->shape[1] != H || o->shape[2] != D) return fail(AQ_ERR_SHAPE, "k_out/v_out must have k's shape");
    }
    for (int i = 0; i < 8; ++i) {
        if (!outs[i]) continue;
        if ((st = check_output(outs[i], i < 6 ? "cache" : "k_out/v_out")) != AQ_OK) return st;
        for (int j = 0; j < 2; ++j)
            if (overlaps(outs[i], ins[j])) return fail(AQ_ERR_OVERLAP, "an output overlaps k or v");
        for (int j = 0; j < i; ++j)
            if (outs[j] && overlaps(outs[i], outs[j]) && !interleave(outs[i], outs[j]))
                return fail(AQ_ERR_OVERLAP, "outputs overlap each other");
    }
    if (T == 0 || H == 0 || D == 0) return AQ_OK;
    if (!slots) return fail(AQ_ERR_NULL, "slots is NULL");
    if (H * (D / 8) > (1 << 24) || k_wq->shape[2] > 0x7fffffff) return fail(AQ_ERR_UNSUPPORTED, "rows too large");
    if ((st = check_device()) != AQ_OK) return st;
    for (int j = 0; j < 2; ++j) {
        const aq_view *x = ins[j], *o = outs[6 + j];
        auto vec = [&](const aq_view* t) {
            return aligned16(t->data) && (T <= 1 || t->stride[0] % 8 == 0) && (H <= 1 || t->stride[1] % 8 == 0);
        };
        a.x[j] = (const uint16_t*)x->data;
        a.x_tok[j] = x->stride[0];
        a.x_head[j] = x->stride[1];
        a.xvec[j] = vec(x) ? 1 : 0;
        if (o) {
            a.out[j] = (uint16_t*)o->data;
            a.o_tok[j] = o->stride[0];
            a.o_head[j] = o->stride[1];
            a.ovec[j] = vec(o) ? 1 : 0;
        }
    }
    a.slots = slots;
    a.T = T;
    a.H = (int)H;
    a.D = (int)D;
    a.S = (int)k_wq->shape[2];
    a.nslots = k_wq->shape[0] * k_wq->shape[2];
    a.log2g = log2i(group);
    cudaError_t e = aq::device_error_ptr(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = aq::kv::launch_append(a, k->dtype == AQ_BF16, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "cache append launch");
    return AQ_OK;
}

AQ_API aq_status aq_kv_attention_workspace(const aq_view* q, const aq_view* k_wq, int64_t max_pages, size_t* bytes) {
    g_msg[0] = 0;
    if (!bytes) return fail(AQ_ERR_NULL, "bytes is NULL");
    aq_status st = check_attention_q(q, k_wq, max_pages);
    if (st != AQ_OK) return st;
    const aq::kv::AttnShape s = attention_shape(q, k_wq, max_pages);
    *bytes = numel(q) > 0 && s.split ? (s.o_floats + s.ml_floats) * sizeof(float) : 0;
    return AQ_OK;
}

AQ_API aq_status aq_kv_attention(const aq_view* q, const aq_view* k_wq, const aq_view* k_scales, const aq_view* k_biases,
                                 const aq_view* v_wq, const aq_view* v_scales, const aq_view* v_biases, int group, int bits,
                                 const int64_t* pages, int64_t pages_row, int64_t max_pages, const int64_t* lengths,
                                 float scale, int window, const aq_view* out, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    g_msg[0] = 0;
    aq_status st;
    if ((st = check_attention_q(q, k_wq, max_pages)) != AQ_OK) return st;
    if ((st = check_cache_bits(bits, group)) != AQ_OK) return st;
    const int64_t B = q->shape[0], Tq = q->shape[1], Hq = q->shape[2], D = q->shape[3], H = k_wq->shape[1];
    if (D % group != 0) return fail(AQ_ERR_GROUP, "head size %lld not a multiple of group=%d", (long long)D, group);
    aq::kv::AttnArgs a;
    memset(&a, 0, sizeof a);
    if ((st = check_cache_side(k_wq, k_scales, k_biases, "k cache", q->dtype, D, group, &a.k)) != AQ_OK) return st;
    if ((st = check_cache_side(v_wq, v_scales, v_biases, "v cache", q->dtype, D, group, &a.v)) != AQ_OK) return st;
    for (int i = 0; i < 3; ++i)
        if (v_wq->shape[i] != k_wq->shape[i]) return fail(AQ_ERR_SHAPE, "the v cache must have the k cache's shape");
    if ((st = check_view(out, "out", 4, 4)) != AQ_OK) return st;
    if (out->dtype != q->dtype) return fail(AQ_ERR_DTYPE, "out must have q's dtype");
    for (int i = 0; i < 4; ++i)
        if (out->shape[i] != q->shape[i]) return fail(AQ_ERR_SHAPE, "out must have q's shape");
    if ((st = check_output(out, "out")) != AQ_OK) return st;
    if (window < 0) return fail(AQ_ERR_SHAPE, "window < 0");
    if (!(scale - scale == 0.0f)) return fail(AQ_ERR_SHAPE, "scale must be finite");
    const aq::kv::AttnShape s = attention_shape(q, k_wq, max_pages);
    const size_t need = numel(q) > 0 && s.split ? (s.o_floats + s.ml_floats) * sizeof(float) : 0;
    aq_view ws;
    memset(&ws, 0, sizeof ws);
    ws.data = workspace;
    ws.dtype = AQ_F32;
    ws.rank = 1;
    ws.shape[0] = (int64_t)(need / 4);
    ws.stride[0] = 1;
    const aq_view* ins[7] = {q, k_wq, k_scales, k_biases, v_wq, v_scales, v_biases};
    for (const aq_view* v : ins) {
        if (overlaps(out, v)) return fail(AQ_ERR_OVERLAP, "out overlaps an input");
        if (need && overlaps(&ws, v)) return fail(AQ_ERR_OVERLAP, "the workspace overlaps an input");
    }
    if (need && overlaps(&ws, out)) return fail(AQ_ERR_OVERLAP, "the workspace overlaps out");
    if (numel(q) == 0) return AQ_OK;
    if (need) {
        if (!workspace) return fail(AQ_ERR_NULL, "workspace is NULL");
        if (workspace_bytes < need)
            return fail(AQ_ERR_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
        if (!aligned16(workspace)) return fail(AQ_ERR_ALIGN, "workspace must be 16-byte aligned");
    }
    if (!lengths || (!pages && max_pages > 0)) return fail(AQ_ERR_NULL, "pages / lengths is NULL");
    if (pages_row < 0) return fail(AQ_ERR_STRIDE, "pages_row < 0");
    if ((st = check_device()) != AQ_OK) return st;
    const int64_t S = k_wq->shape[2], kg = D / group;
    a.q = (const uint16_t*)q->data;
    a.q_b = q->stride[0]; a.q_t = q->stride[1]; a.q_h = q->stride[2];
    a.out = (uint16_t*)out->data;
    a.o_b = out->stride[0]; a.o_t = out->stride[1]; a.o_h = out->stride[2];
    a.ovec = ((uintptr_t)out->data & 7) == 0 && (B <= 1 || a.o_b % 4 == 0) && (Tq <= 1 || a.o_t % 4 == 0) &&
             (Hq <= 1 || a.o_h % 4 == 0);
    a.pages = pages;
    a.pages_row = pages_row;
    a.max_pages = max_pages;
    a.P = k_wq->shape[0];
    a.lengths = lengths;
    a.B = (int)B; a.Tq = (int)Tq; a.Hq = (int)Hq; a.Hkv = (int)H; a.S = (int)S;
    a.rep = (int)(Hq / H);
    a.rows = (int)(Hq / H * Tq);
    a.rtiles = s.rtiles;
    a.window = window;
    a.scale_log2 = scale * 1.4426950408889634f;
    // tiles of 16 tokens copy as whole pieces: pages of whole tiles, scales and biases dense per head and page
    bool fast = S > 0 && S % 16 == 0;
    for (const aq::kv::Side* d : {&a.k, &a.v})
        fast = fast && d->s_slot == kg && d->b_slot == kg && aligned16(d->scales) && aligned16(d->biases) &&
               d->s_page % 8 == 0 && d->s_head % 8 == 0 && d->b_page % 8 == 0 && d->b_head % 8 == 0;
    // ... and page ids and strides (in bytes) of 32 bits
    const int64_t lim = 0xffffffffll;
    fast = fast && a.P < lim;
    for (const aq::kv::Side* d : {&a.k, &a.v})
        fast = fast && d->w_page * 4 <= lim && d->w_slot * 4 <= lim && d->s_page * 2 <= lim && d->b_page * 2 <= lim;
    a.k_page = (uint32_t)(a.k.w_page * 4);
    a.k_slot = (uint32_t)(a.k.w_slot * 4);
    a.v_page = (uint32_t)(a.v.w_page * 4);
    a.v_slot = (uint32_t)(a.v.w_slot * 4);
    a.fast = fast ? 1 : 0;
    a.scp = kg > 1 ? 1 : 0;
    for (const aq::kv::Side* d : {&a.k, &a.v}) {
        const uintptr_t at = (uintptr_t)d->scales | (uintptr_t)d->biases;
        if (at % (2 * kg) != 0) a.scp = 0;
        for (int64_t x : {d->s_page, d->s_head, d->s_slot, d->b_page, d->b_head, d->b_slot})
            if (x % kg != 0) a.scp = 0;
    }
    const int unit = aq::kv::unit_tokens((int)D, s.nt);
    a.unit_slots = S > 0 ? (int)(unit % S) : 0;
    a.split = s.split;
    a.part_o = (float*)workspace;
    a.part_ml = (float*)workspace + s.o_floats;
    cudaError_t e = aq::device_error_ptr(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = aq::kv::launch_attention(a, s, (int)D, group, q->dtype == AQ_BF16, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "cache attention launch");
    return AQ_OK;
}

AQ_API aq_status aq_moe_swiglu_workspace(int64_t tokens, int top_k, int64_t k, int64_t n, size_t* bytes) {
    g_msg[0] = 0;
    if (!bytes) return fail(AQ_ERR_NULL, "bytes is NULL");
    if (tokens < 0) return fail(AQ_ERR_SHAPE, "tokens < 0");
    aq_status st = check_moe_sizes(tokens, top_k, k, n);
    if (st != AQ_OK) return st;
    *bytes = aq::moe::Layout(tokens, top_k, k, n).bytes;
    return AQ_OK;
}

AQ_API aq_status aq_moe_swiglu(const aq_view* x, const aq_view* logits, int top_k, int norm_topk, const aq_view* wq_gate,
                               const aq_view* s_gate, const aq_view* b_gate, const aq_view* wq_up, const aq_view* s_up,
                               const aq_view* b_up, const aq_view* wq_down, const aq_view* s_down, const aq_view* b_down,
                               int group, int bits, float rms_eps, const aq_view* r, const aq_view* y, void* workspace,
                               size_t workspace_bytes, void* stream) {
    g_msg[0] = 0;
    aq_status st;
    if ((st = check_view(x, "x", 2, 2)) != AQ_OK) return st;
    if ((st = check_view(logits, "logits", 2, 2)) != AQ_OK) return st;
    if ((st = check_view(y, "y", 2, 2)) != AQ_OK) return st;
    if ((st = check_output(y, "y")) != AQ_OK) return st;
    if ((st = check_bits_group(bits, group)) != AQ_OK) return st;
    if (!(bits == 2 || bits == 4 || bits == 8) || (bits == 2 && group == 32))
        return fail(AQ_ERR_UNSUPPORTED, "the layer takes 4- and 8-bit codes, and 2-bit codes in groups of 64 or 128");
    if (!is_half(x->dtype)) return fail(AQ_ERR_DTYPE, "x must be bf16 or f16");
    if (!(logits->dtype == AQ_F32 || is_half(logits->dtype))) return fail(AQ_ERR_DTYPE, "logits must be f32, bf16 or f16");
    if (y->dtype != x->dtype && y->dtype != AQ_F32) return fail(AQ_ERR_DTYPE, "y must have x's dtype or f32");
    if (!(rms_eps >= 0.0f) || !(rms_eps - rms_eps == 0.0f)) return fail(AQ_ERR_SHAPE, "rms_eps must be finite and >= 0");
    const int64_t T = x->shape[0], K = x->shape[1], E = logits->shape[1];
    if (logits->shape[0] != T) return fail(AQ_ERR_SHAPE, "logits must have x's %lld rows", (long long)T);
    if (y->shape[0] != T || y->shape[1] != K) return fail(AQ_ERR_SHAPE, "y must have x's shape");
    if (!wq_gate || wq_gate->rank != 3) return check_view(wq_gate, "gate", 3, 3);
    const int64_t N = wq_gate->shape[1];
    if ((st = check_moe_sizes(T, top_k, K, N)) != AQ_OK) return st;
    if (E < 1 || E > aq::moe::MAX_EXPERTS) return fail(AQ_ERR_UNSUPPORTED, "%lld experts (1..%d)", (long long)E, aq::moe::MAX_EXPERTS);
    if (top_k > E) return fail(AQ_ERR_SHAPE, "top_k=%d of %lld experts", top_k, (long long)E);
    aq::moe::Args a;
    memset(&a, 0, sizeof a);
    if ((st = check_bank(wq_gate, s_gate, b_gate, "gate", x->dtype, E, N, K, group, bits, &a.gate)) != AQ_OK) return st;
    if ((st = check_bank(wq_up, s_up, b_up, "up", x->dtype, E, N, K, group, bits, &a.up)) != AQ_OK) return st;
    if ((st = check_bank(wq_down, s_down, b_down, "down", x->dtype, E, K, N, group, bits, &a.down)) != AQ_OK) return st;
    a.gate.svec = a.up.svec = a.gate.svec && a.up.svec;
    if (r) {
        if ((st = check_view(r, "r", 2, 2)) != AQ_OK) return st;
        if (r->dtype != y->dtype) return fail(AQ_ERR_DTYPE, "r must have y's dtype");
        if (r->shape[0] != T || r->shape[1] != K) return fail(AQ_ERR_SHAPE, "r must have y's shape");
        if (overlaps(r, y) && !same_view(r, y)) return fail(AQ_ERR_OVERLAP, "r overlaps y (other than being the same view)");
    }
    const aq::moe::Layout lay(T, top_k, K, N);
    const size_t need = lay.bytes;
    aq_view ws;
    memset(&ws, 0, sizeof ws);
    ws.data = workspace;
    ws.dtype = AQ_F32;
    ws.rank = 1;
    ws.shape[0] = (int64_t)(need / 4);
    ws.stride[0] = 1;
    // x is read before the first element of y is written, so y may be x itself
    if (overlaps(y, x) && !same_view(y, x)) return fail(AQ_ERR_OVERLAP, "y overlaps x (other than being the same view)");
    const aq_view* ins[10] = {logits, wq_gate, s_gate, b_gate, wq_up, s_up, b_up, wq_down, s_down, b_down};
    for (const aq_view* v : ins) {
        if (overlaps(y, v)) return fail(AQ_ERR_OVERLAP, "y overlaps an input");
        if (overlaps(&ws, v)) return fail(AQ_ERR_OVERLAP, "the workspace overlaps an input");
    }
    if (overlaps(&ws, x) || overlaps(&ws, y) || (r && overlaps(&ws, r))) return fail(AQ_ERR_OVERLAP, "the workspace overlaps x, r or y");
    if (T == 0 || K == 0) return AQ_OK;
    if (N == 0) return fail(AQ_ERR_SHAPE, "experts without rows");
    if (!workspace) return fail(AQ_ERR_NULL, "workspace is NULL");
    if (workspace_bytes < need) return fail(AQ_ERR_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if (!aligned16(workspace)) return fail(AQ_ERR_ALIGN, "workspace must be 16-byte aligned");
    if ((st = check_device()) != AQ_OK) return st;
    a.x = (const uint16_t*)x->data;
    a.x_row = x->stride[0];
    a.logits = logits->data;
    a.l_row = logits->stride[0];
    a.ldt = logits->dtype;
    a.T = (int)T;
    a.E = (int)E;
    a.topk = top_k;
    a.norm = norm_topk != 0;
    a.K = (int)K;
    a.N = (int)N;
    uint8_t* w = (uint8_t*)workspace;
    a.entries = (int*)w;
    a.pairs = (uint16_t*)(w + lay.pairs);
    a.weight = (float*)(w + lay.weight);
    a.hmax = (unsigned*)(w + lay.hmax);
    a.xh = (uint16_t*)(w + lay.xh);
    a.xfac = (float*)(w + lay.xfac);
    a.h = (uint16_t*)(w + lay.h);
    a.hscale = (float*)(w + lay.hscale);
    a.y = y->data;
    a.y_row = y->stride[0];
    a.ydt = y->dtype;
    a.r = r ? r->data : nullptr;
    a.r_row = r ? r->stride[0] : 0;
    a.rms_eps = rms_eps;
    cudaError_t e = aq::device_error_ptr(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word");
    e = aq::moe::launch(a, bits, group, x->dtype == AQ_BF16, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "mixture-of-experts launch");
    return AQ_OK;
}
