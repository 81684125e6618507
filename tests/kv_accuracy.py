"""Attention over a 4-bit cache in 64 bits, with two bounds on what may differ: element by element, and root mean square.

The kernel's sums per element of the output, with codes q, scales s, biases b of a token j's value and p_j its probability:
    out = sum_j (p_j s_j)(q_j - c_j) + sum_j p_j (b_j + c_j s_j),   c_j = 8 or 7.
Its errors, relative to the magnitudes M = sum_j p_j (|s_j| w_j + |b_j + 7.5 s_j| + |s_j|/2), w_j = max(|q_j - 8|, |q_j - 7|), and
A = sum_j p_j (15 |s_j| + |b_j|) (codes and the middle of the codes enter the sums each for itself):
  - the output's rounding: at most u |out|, u half a step of the type;
  - p_j s_j rounded to 11 bits (bf16) or 22 (f16, two numbers of 11): at most r = 2^-11 or 2^-22 of each term, independent from
    token to token: rms r / sqrt 3 sqrt(sum_j (p_j s_j w_j)^2);
  - the score of token j in fp32: delta_j = 2^-20 scale sum_d |q_d| (15 |s_jd| + |b_jd|) (MMAs of 16 products, at most 8 a group,
    each within 2^-23 of the magnitudes summed, then one fused step a group, the scaling and the exponential's argument), which
    moves p_j by 2 delta_j of itself at most (numerator and sum), plus 2^-20 for the exponential and the joins; as rms 2^-22 of the same
    magnitudes, of p_j v_j, independent from token to token (what moves all alike leaves p as it is);
  - the sums over tokens: every tile's MMAs are cut at 2^-23 of the magnitudes that meet in them, twice (the middle, then the codes),
    mirror images of one another, and the tiles' results are added in fp32, rounded to nearest: 2^-22 A.
"""
import torch

from tests.accuracy import MARGIN, misses  # noqa: F401


def values(side, page_ids, head, slots, group):
    """(codes, scales, biases) [tokens, D] in float64, of one head."""
    wq, sc, bi = (x[page_ids, head, slots] for x in side)
    w = wq.to(torch.int64) & 0xFFFFFFFF
    q = torch.stack([(w >> (4 * i)) & 15 for i in range(8)], -1).flatten(-2).double()
    at = torch.arange(q.shape[-1], device=q.device) // group
    return q, sc.double()[:, at], bi.double()[:, at]


def attention(q, kc, vc, pages, lengths, group, window=0, which=None, weights=None):
    """(out, bound, rms): the formula in float64, the elementwise bound and, without the output's rounding, the rms allowance of every
    element; which: the sequences to do (the others' rows stay zero); weights(p s): the probabilities times scales as they are
    carried, if not exactly.  Tensors on any device."""
    B, Tq, Hq, D = q.shape
    H, S = kc[0].shape[1], kc[0].shape[2]
    rep = Hq // H
    scale = D ** -0.5
    u = torch.finfo(q.dtype).eps / 2
    r = 2.0 ** -22 if q.dtype == torch.float16 else 2.0 ** -11
    out, bound, rms = (torch.zeros(q.shape, dtype=torch.float64, device=q.device) for _ in range(3))
    for b in range(B) if which is None else which:
        n = int(lengths[b])
        for h in range(H) if n > 0 else ():
            first = max(0, n - Tq - window + 1) if window else 0
            t = torch.arange(first, n, device=q.device)
            at = pages[b].to(q.device)[t // S], h, t % S
            kq, ks, kb = values(kc, *at, group)
            vq, vs, vb = values(vc, *at, group)
            k, kmag = ks * kq + kb, 15 * ks.abs() + kb.abs()
            v, w = vs * vq + vb, vs.abs() * torch.maximum((vq - 8).abs(), (vq - 7).abs())
            m, a = w + (vb + 7.5 * vs).abs() + vs.abs() / 2, 15 * vs.abs() + vb.abs()
            for i in range(Tq):
                pos = n - Tq + i
                if pos < 0:
                    continue
                lo = (max(0, pos - window + 1) if window else 0) - first
                z = slice(lo, pos + 1 - first)
                rows = slice(h * rep, (h + 1) * rep)
                x = q[b, i, rows].double()
                p = torch.softmax(x @ k[z].T * scale, -1)
                delta = 2.0 ** -20 * scale * (x.abs() @ kmag[z].T)
                o, A = p @ v[z], p @ a[z]
                if weights is not None:
                    o = p @ (vb + 7.5 * vs)[z] + torch.einsum("rtd,td->rd", weights(p[:, :, None] * vs[z]), vq[z] - 7.5)
                out[b, i, rows] = o
                bound[b, i, rows] = (u * o.abs() + r * (p @ w[z]) + (2 * delta.amax(-1, keepdim=True) + 2.0 ** -20) * (p @ m[z])
                                     + 2.0 ** -22 * A)
                sq = (p ** 2) @ (r ** 2 / 3 * w[z] ** 2) + ((p * delta / 4) ** 2) @ (v[z] ** 2)
                rms[b, i, rows] = torch.sqrt(sq + (2.0 ** -22 * A) ** 2)
    return out, bound + torch.finfo(q.dtype).tiny * torch.finfo(q.dtype).eps, rms

