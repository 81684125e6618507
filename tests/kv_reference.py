"""Plain 64-bit counterparts of the key/value cache calls, and seeded caches, for the tests."""
import numpy as np
import torch

import oracle


def dname(dtype):
    return {torch.bfloat16: "bf16", torch.float16: "f16"}[dtype]


def make_cache(P, H, S, D, group, dtype, seed, std=1.0, layout="phs"):
    """A quantized cache of normal values: (codes [P, H, S, D] float64, (wq, scales, biases)) on the CPU.  layout "psh"
    stores slots outside heads and returns transposed views."""
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(P * H * S, D, generator=g) * std
    Q = oracle.quantize(w.numpy(), group, 4, dname(dtype))
    wq = torch.from_numpy(Q.packed.view(np.int32).copy())
    sc = torch.from_numpy(Q.scale_bits.view(np.int16).copy()).view(dtype)
    bi = torch.from_numpy(Q.bias_bits.view(np.int16).copy()).view(dtype)
    t = [x.view(P, H, S, -1) for x in (wq, sc, bi)]
    if layout == "psh":
        t = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in t]
    return tuple(t)


def to_dev(side, device="cuda"):
    """A copy on the device with the same strides."""
    out = []
    for x in side:
        y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=device)
        y.copy_(x)
        out.append(y)
    return tuple(out)


def codes(wq):
    """Packed 4-bit words [..., W] to codes [..., 8 W] in float64."""
    w = wq.to(torch.int64) & 0xFFFFFFFF
    return torch.stack([(w >> (4 * i)) & 15 for i in range(8)], -1).flatten(-2).double()


def parts(side, group):
    """(scale * code, bias) per element, float64."""
    wq, sc, bi = side
    D = wq.shape[-1] * 8
    at = torch.arange(D) // group
    return codes(wq) * sc.double()[..., at], bi.double()[..., at]


def attention(q, kc, vc, pages, lengths, group, scale, window=0):
    """(out, bound): the formula in float64, and how far a result may be from it element by element.

    bound = u |out| + (2^-11 + 2 delta) A: the output's rounding u (half a step of its type); the rounding of a probability
    times a scale to 11 bits (2^-11 of every term); and delta, the error of a score in fp32.  A = sum_j p_j (|s| code + |b|),
    for f16, where codes count from 7 or 8 (|code - 8| <= max(code, 8)), sum_j p_j (|s| max(code, 8) + |b|).
    delta = 2^-20 scale max_j sum_d |q_d| (1040 |s_jd| + |b_jd|): the codes carry an offset of at most 1024 through fp32 sums
    of 16 products per step, at most 8 steps a group, each off by at most 2^-23 of the magnitudes summed.  exp, the sums of p
    and the joins of partial sums are within a few 2^-22, which 2^-20 of the same magnitudes covers (a 2^-16 floor below)."""
    B, Tq, Hq, D = q.shape
    H, S = kc[0].shape[1], kc[0].shape[2]
    rep = Hq // H
    out = torch.zeros(B, Tq, Hq, D, dtype=torch.float64)
    bound = torch.zeros_like(out)
    u = torch.finfo(q.dtype).eps / 2
    qd = q.double()
    at = torch.arange(D) // group
    for b in range(B):
        n = int(lengths[b])
        if n <= 0:
            continue
        t = torch.arange(n)
        pg, sl = pages[b][t // S], t % S
        for h in range(H):
            ks, kb = parts(tuple(x[pg, h, sl] for x in kc), group)
            vs, vb = parts(tuple(x[pg, h, sl] for x in vc), group)
            va = torch.maximum(vs.abs(), 8 * vc[1][pg, h, sl].double().abs()[:, at]) if q.dtype == torch.float16 else vs.abs()
            mag = 1040 * kc[1][pg, h, sl].double().abs()[:, at] + kb.abs()
            for i in range(Tq):
                pos = n - Tq + i
                lo = max(0, pos - window + 1) if window else 0
                if pos < 0:
                    continue
                r = slice(lo, pos + 1)
                x = qd[b, i, h * rep:(h + 1) * rep]
                p = torch.softmax(x @ (ks + kb)[r].T * scale, -1)
                o = p @ (vs + vb)[r]
                A = p @ (va + vb.abs())[r]
                delta = 2.0 ** -20 * abs(scale) * (x.abs() @ mag[r].T).amax(-1, keepdim=True) + 2.0 ** -16
                out[b, i, h * rep:(h + 1) * rep] = o
                bound[b, i, h * rep:(h + 1) * rep] = u * o.abs() + (2.0 ** -11 + 2 * delta) * A
    # results below the type's normal range are rounded to its subnormal step
    return out, bound + torch.finfo(q.dtype).tiny * torch.finfo(q.dtype).eps


def page_table(lengths, S, seed, spare=1):
    """Distinct pages per sequence in a random order: (pages [B, max], P)."""
    used = [-(-max(0, int(n)) // S) for n in lengths]
    P = sum(used) + spare
    order = torch.randperm(P, generator=torch.Generator().manual_seed(seed))
    pages = torch.zeros(len(used), max(1, max(used)), dtype=torch.int64)
    at = 0
    for b, k in enumerate(used):
        pages[b, :k] = order[at:at + k]
        at += k
    return pages, P
