"""A mixture-of-experts layer in 64 bits, with two bounds on what may differ: element by element, and root mean square.

y = r + sum_j w_j Wd_j h_j, h = silu(g) u, g = n x Wg^T, u = n x Wu^T.  With |W| <= |s| code + |b| = mag (codes enter the sums each for
itself), the errors are:
  - y's rounding: half a step of its type;
  - a product's sum: MMAs of 16 products, at most 8 a group, each cut at 2^-23 of the magnitudes summed, then a fused step a group: at
    most e = 2^-19 mag |x| (of 2^4 steps one after another), and 2^-22 mag |x| as rms (cuts of group sums of either sign);
  - h: w (1.1 |u| e_g + |silu(g)| e_u) from its sums, 2^-18 |h| (rms 2^-20) from the exponential and the divisions, and its rounding to 11
    bits (y bf16) or 22 (f16, f32), r = 2^-11 or 2^-22: at most r |h|, rms r |h| / sqrt 3, independent from column to column; where an
    f16 number is subnormal 2^-32 of the token's largest;
  - the down product: as the first ones, of h; the weight w within 2^-21 of itself.
"""
import torch

from tests.accuracy import MARGIN, misses  # noqa: F401


class Bank:
    """64-bit values and magnitudes of a quantized bank [E, N, K] = (wq, scales, biases), on its device."""

    def __init__(self, side, group, bits):
        wq, sc, bi = side
        w = wq.to(torch.int64) & 0xFFFFFFFF
        q = torch.stack([(w >> (bits * i)) & (2 ** bits - 1) for i in range(32 // bits)], -1).flatten(-2).double()
        s, b = (t.double().repeat_interleave(group, -1) for t in (sc, bi))
        self.v, self.mag = s * q + b, s.abs() * q + b.abs()


def layer(x, logits, top_k, banks, ydt, norm=True, rms_eps=0.0, r=None, carried=None):
    """(y, bound, rms); rms without y's rounding.  carried(h): the activations as they pass to the down product, if not exactly."""
    gate, up, down = banks
    xs = x.double()
    if rms_eps > 0:
        xs = xs / torch.sqrt((xs ** 2).mean(-1, keepdim=True) + rms_eps)
    y = r.double().clone() if r is not None else torch.zeros_like(xs)
    bound, var = torch.zeros_like(xs), torch.zeros_like(xs)
    part = 2.0 ** -11 if ydt == torch.bfloat16 else 2.0 ** -22
    order = torch.sort(logits.double(), dim=-1, descending=True, stable=True)
    for t in range(x.shape[0]):
        ids, top = order.indices[t, :top_k], order.values[t, :top_k]
        w = torch.softmax(top, 0) if norm else torch.softmax(logits[t].double(), 0)[ids]
        for e, we in zip(ids.tolist(), w):
            g, u = gate.v[e] @ xs[t], up.v[e] @ xs[t]
            mg, mu = gate.mag[e] @ xs[t].abs(), up.mag[e] @ xs[t].abs()
            a = g * torch.sigmoid(g)
            h = we * a * u
            first = lambda c: we * (1.1 * u.abs() * c * mg + a.abs() * c * mu)
            d, wd = down.v[e], down.mag[e]
            o = d @ (h if carried is None else carried(h))
            y[t] += o
            eh = first(2.0 ** -19) + (part + 2.0 ** -18) * h.abs() + 2.0 ** -32 * h.abs().max()
            bound[t] += d.abs() @ eh + 2.0 ** -19 * (wd @ (h.abs() + eh)) + 2.0 ** -21 * o.abs()
            rh = first(2.0 ** -22) ** 2 + (part ** 2 / 3 + 2.0 ** -40) * h ** 2
            var[t] += d ** 2 @ rh + (2.0 ** -22 * (wd @ h.abs())) ** 2 + (2.0 ** -21 * o) ** 2
    u = torch.finfo(ydt).eps / 2
    return y, bound + u * (y.abs() + bound) + torch.finfo(ydt).tiny * torch.finfo(ydt).eps, var.sqrt()
