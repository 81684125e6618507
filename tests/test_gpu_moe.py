"""GPU tests of the mixture-of-experts layer (aq_moe_swiglu) against the formula in 64 bits.

Tolerance.  y = r + sum_j w_j Wd (silu(g) u), all sums fp32.  Rounding y is half a step of its type.  g and u are sums of
K products, s D + b X per group (D sums codes times x, X sums x): each is off by at most
e1 = 2^-19 sum_k |n x_k| (|s| (128 + code) + |b|) (MMAs of 16 products, at most 8 a group, each within 2^-23 of the
magnitudes summed, and the folds of K/G groups over four warps, 2^-24 each of at most 2^4 of them one after another).
h = w silu(g) u is off by |w| (|u| 1.1 e1 + |silu(g)| e1) (|silu'| <= 1.1); it is carried as f16 with a power of two per 16
values (per row when multiplied), off by half a step of 11 bits, 2^-11 |h|, or where it is a subnormal by 2^-25 / 2^13 = 2^-38
of the largest of its row times the code's weight, at most 2^6: 2^-32; __expf and the divisions are within 2^-18 of h.  The down product adds 2^-19 sum |h| (|s| (128 + code) + |b|) and weighs
the errors of h with |Wd|.
"""
import numpy as np
import pytest
import torch

import oracle
from group_wise_affine_qmv_b200 import aq, inputs
from tests.parity import dtype_name, to_device_quant

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda"
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


class Bank:
    """A quantized bank [E, N, K]: device tensors, and float64 values and magnitudes on the CPU."""

    def __init__(self, E, N, K, group, bits, dtype, seed, std=0.02):
        Q = oracle.quantize(inputs.normal((E, N, K), std, seed=seed).numpy(), group, bits, dtype_name(torch.empty(0, dtype=dtype)))
        self.dev = to_device_quant(Q, DEV, dtype)
        self.v = torch.from_numpy(Q.dequant()).double().view(E, N, K)
        s = self.dev[1].double().cpu().abs().repeat_interleave(group, -1)
        b = self.dev[2].double().cpu().abs().repeat_interleave(group, -1)
        self.mag = self.v.abs() + 2 * b + 128 * s     # >= |s| (128 + code) + |b|


def reference(x, logits, top_k, banks, norm, rms_eps, r, ydt):
    gate, up, down = banks
    x64, z = x.double(), logits.double()
    T, K = x.shape
    n = 1 / torch.sqrt((x64 ** 2).mean(-1, keepdim=True) + rms_eps) if rms_eps > 0 else torch.ones(T, 1, dtype=torch.float64)
    y = r.double().clone() if r is not None else torch.zeros(T, K, dtype=torch.float64)
    err = torch.zeros(T, K, dtype=torch.float64)
    for t in range(T):
        row = [(-np.inf if v == -np.inf else v) for v in z[t].tolist()]
        ids = [e for e in sorted(range(len(row)), key=lambda e: (-row[e], e))[:top_k] if row[e] != -np.inf]
        if not ids:
            continue
        top = z[t, ids[0]]
        p = torch.exp(z[t, ids] - top)
        w = p / (p.sum() if norm else torch.exp(z[t] - top).sum())
        xt = x64[t] * n[t]
        for e, we in zip(ids, w):
            g, u = gate.v[e] @ xt, up.v[e] @ xt
            eg, eu = (2.0 ** -19 * (m.mag[e] @ xt.abs()) for m in (gate, up))
            s = g * torch.sigmoid(g)
            h = we * s * u
            eh = we * (u.abs() * 1.1 * eg + s.abs() * eu + eg * eu) + (2.0 ** -11 + 2.0 ** -18) * h.abs() + 2.0 ** -32 * h.abs().max()
            y[t] += down.v[e] @ h
            err[t] += down.v[e].abs() @ eh + 2.0 ** -19 * (down.mag[e] @ (h.abs() + eh))
    u = torch.finfo(ydt).eps / 2
    return y, u * (y.abs() + err) + err + 2.0 ** -22 * y.abs() + torch.finfo(ydt).tiny * torch.finfo(ydt).eps


def setup(T, E, K, N, group, bits, dtype, seed=0):
    banks = (Bank(E, N, K, group, bits, dtype, seed), Bank(E, N, K, group, bits, dtype, seed + 1),
             Bank(E, K, N, group, bits, dtype, seed + 2))
    x = inputs.normal((T, K), 1.0, dtype, seed=seed + 3)
    logits = inputs.normal((T, E), 1.5, F32, seed=seed + 4)
    return banks, x, logits


def call(banks, x, logits, top_k, group, bits, **kw):
    kw = {k: v.to(DEV) if isinstance(v, torch.Tensor) and not v.is_cuda else v for k, v in kw.items()}
    y = aq.aq_moe_swiglu(x.to(DEV), logits.to(DEV), top_k, *[b.dev for b in banks], group, bits, **kw)
    aq.aq_device_error()
    return y


def close(y, want, bound):
    err = (y.double().cpu() - want).abs()
    assert torch.all(err <= bound), (err / bound).max().item()


@pytest.mark.parametrize("T,E,top_k,K,N,group,bits,dtype,norm,rms,res,ydt", [
    (1, 4, 1, 128, 64, 64, 4, BF, True, 0.0, False, BF),
    (1, 8, 8, 96, 160, 32, 4, F16, True, 0.0, True, F16),
    (3, 16, 2, 256, 128, 128, 4, BF, False, 1e-6, True, BF),
    (5, 6, 3, 1408, 96, 32, 8, BF, True, 1e-6, False, F32),
    (2, 40, 4, 160, 352, 32, 8, F16, False, 0.0, False, F32),
    (17, 2, 2, 192, 192, 64, 8, F16, True, 1e-5, True, F16),      # 17 tokens per expert: a second block of one
    (64, 3, 2, 128, 256, 128, 8, BF, True, 0.0, True, BF),        # up to 64 tokens of one expert
    (64, 64, 6, 256, 128, 64, 4, BF, True, 1e-6, True, F32),
    (33, 130, 5, 64, 64, 64, 2, BF, True, 0.0, False, BF),        # more than 128 experts
    (4, 512, 16, 128, 128, 128, 2, F16, False, 0.0, False, F16),
    (9, 5, 5, 640, 384, 128, 4, F16, True, 0.0, False, F16),      # every expert for every token, odd numbers of groups
])
def test_layer_matches_the_formula(T, E, top_k, K, N, group, bits, dtype, norm, rms, res, ydt):
    banks, x, logits = setup(T, E, K, N, group, bits, dtype, seed=T + E)
    r = inputs.normal((T, K), 1.0, ydt, seed=99) if res else None
    y = call(banks, x, logits, top_k, group, bits, norm_topk=norm, rms_eps=rms, residual=r, out_dtype=ydt)
    close(y, *reference(x, logits, top_k, banks, norm, rms, r, ydt))


@pytest.mark.parametrize("T,E,top_k,K,N,group,bits,dtype", [
    (40, 64, 4, 256, 512, 64, 4, BF),       # more than two gate/up items per CTA that fits: a warp has items of its own
    (64, 8, 2, 160, 1024, 32, 8, F16),      # the same with 16 tokens an entry and rows of odd numbers of groups
    (48, 40, 3, 192, 512, 64, 2, BF),
    (64, 4, 2, 2112, 1216, 32, 4, BF),      # rows whose scales do not fit a warp's block
    (64, 4, 2, 96, 8224, 32, 8, BF),        # and those of the down bank
    (30, 32, 4, 384, 640, 128, 8, F16),
])
def test_many_items(T, E, top_k, K, N, group, bits, dtype):
    banks, x, logits = setup(T, E, K, N, group, bits, dtype, seed=T + K)
    y = call(banks, x, logits, top_k, group, bits, out_dtype=F32)
    close(y, *reference(x, logits, top_k, banks, True, 0.0, None, F32))
    # scales and biases one element past a 16-byte boundary
    odd = []
    for b in banks:
        wq, *sb = b.dev
        flat = [torch.zeros(t.numel() + 1, dtype=t.dtype, device=DEV) for t in sb]
        for f, t in zip(flat, sb):
            f[1:] = t.flatten()
        odd.append((wq, *[f[1:].view(t.shape) for f, t in zip(flat, sb)]))
    z = aq.aq_moe_swiglu(x.to(DEV), logits.to(DEV), top_k, *odd, group, bits, out_dtype=F32)
    aq.aq_device_error()
    close(z, *reference(x, logits, top_k, banks, True, 0.0, None, F32))


def test_ties_infinities_and_empty_rows():
    T, E, K, N, group, bits = 6, 40, 128, 64, 64, 4
    banks, x, logits = setup(T, E, K, N, group, bits, BF, seed=50)
    logits[0] = 0.25                                   # all equal: experts 0, 1, 2
    logits[1, 3:] = float("-inf")                      # only three experts allowed, one more is not chosen
    logits[1, 1] = float("-inf")
    logits[2] = float("-inf")                          # no expert
    logits[3] = torch.finfo(F32).min                   # a mask's lowest value everywhere: equal again
    logits[4] = 0.0
    logits[4, 1::2] = -0.0                             # the two zeros tie
    logits[5, 39] = 80.0                               # one expert takes all
    r = inputs.normal((T, K), 1.0, BF, seed=51)
    for norm in (True, False):
        for res in (None, r):
            y = call(banks, x, logits, 3, group, bits, norm_topk=norm, residual=res)
            close(y, *reference(x, logits, 3, banks, norm, 0.0, res, BF))
            assert torch.equal(y[2].cpu(), torch.zeros(K, dtype=BF) if res is None else r[2])
    for dt in (BF, F16):                               # logits of 16 bits, where ties are common
        lg = (logits.clamp(-100, 100) * 2).round() / 2
        lg[2] = float("-inf")
        y = call(banks, x, lg.to(dt), 3, group, bits)
        close(y, *reference(x, lg.to(dt), 3, banks, True, 0.0, None, BF))


def test_a_broken_token_leaves_the_others_alone():
    T, E, K, N, group, bits = 5, 8, 128, 128, 64, 8
    banks, x, logits = setup(T, E, K, N, group, bits, BF, seed=60)
    base = call(banks, x, logits, 3, group, bits)
    for what in ("logit", "x", "inf"):
        x2, l2 = x.clone(), logits.clone()
        if what == "logit":
            l2[2, 4] = float("nan")
        else:
            x2[2, 7] = float("nan") if what == "x" else float("inf")
        y = call(banks, x2, l2, 3, group, bits)
        keep = [0, 1, 3, 4]
        assert torch.equal(y[keep], base[keep]) and torch.all(torch.isnan(y[2])), what


def test_the_same_call_gives_the_same_bits():
    T, E, K, N, group, bits = 40, 6, 256, 192, 64, 4
    banks, x, logits = setup(T, E, K, N, group, bits, F16, seed=70)
    full = call(banks, x, logits, 2, group, bits, out_dtype=F32)
    for _ in range(5):
        assert torch.equal(full, call(banks, x, logits, 2, group, bits, out_dtype=F32))


def test_strided_operands_and_in_place_update():
    T, E, K, N, group, bits = 7, 5, 256, 128, 64, 8
    banks, x, logits = setup(T, E, K, N, group, bits, BF, seed=80)
    base = call(banks, x, logits, 2, group, bits, rms_eps=1e-6, residual=x)
    wide = torch.zeros(T, K + 24, dtype=BF, device=DEV)
    wide[:, 8:8 + K] = x.to(DEV)
    wl = torch.full((T, E + 3), 50.0, device=DEV)
    wl[:, 1:1 + E] = logits.to(DEV)
    out = torch.full((T, K + 5), 3.0, dtype=BF, device=DEV)
    xs = wide[:, 8:8 + K]
    y = aq.aq_moe_swiglu(xs, wl[:, 1:1 + E], 2, *[b.dev for b in banks], group, bits, rms_eps=1e-6, residual=xs, out=out[:, 2:2 + K])
    assert torch.equal(y, base) and torch.all(out[:, :2] == 3.0) and torch.all(out[:, 2 + K:] == 3.0)
    # banks as slices of larger ones, rows and experts apart
    big = []
    for b in banks:
        wq, sc, bi = b.dev
        w2 = torch.zeros(E, wq.shape[1] + 2, wq.shape[2] + 4, dtype=torch.int32, device=DEV)
        w2[:, 1:-1, :wq.shape[2]] = wq
        s2, b2 = (torch.zeros(E, t.shape[1] + 1, t.shape[2], dtype=BF, device=DEV) for t in (sc, bi))
        s2[:, 1:], b2[:, 1:] = sc, bi
        big.append((w2[:, 1:-1, :wq.shape[2]], s2[:, 1:], b2[:, 1:]))
    y = aq.aq_moe_swiglu(xs, logits.to(DEV), 2, *big, group, bits, rms_eps=1e-6, residual=xs)
    assert torch.equal(y, base)
    aq.aq_moe_swiglu(xs, logits.to(DEV), 2, *[b.dev for b in banks], group, bits, rms_eps=1e-6, residual=xs, out=xs)
    assert torch.equal(xs, base) and torch.all(wide[:, :8] == 0) and torch.all(wide[:, 8 + K:] == 0)
    aq.aq_device_error()


def test_captured_replayed_and_on_two_streams():
    T, E, K, N, group, bits = 4, 8, 512, 256, 64, 4
    banks, x, logits = setup(T, E, K, N, group, bits, BF, seed=90)
    dx, dl = x.to(DEV), logits.to(DEV)
    dev = [b.dev for b in banks]
    base = call(banks, x, logits, 2, group, bits)
    other = call(banks, x.flip(0), logits.flip(0), 2, group, bits)
    out = torch.empty_like(dx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        aq.aq_moe_swiglu(dx, dl, 2, *dev, group, bits, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, base)
    dx.copy_(x.flip(0))
    dl.copy_(logits.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, other)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for s, o in zip(streams, outs):
            with torch.cuda.stream(s):
                o.append(aq.aq_moe_swiglu(dx, dl, 2, *dev, group, bits))
    torch.cuda.synchronize()
    assert all(torch.equal(o, other) for o in outs[0] + outs[1])
    aq.aq_device_error()


def test_layer_after_layer_on_one_stream():
    """Each call's kernels start early next to the one before: a chain gives what the calls one at a time give."""
    T, E, K, N, group, bits = 3, 12, 256, 128, 64, 4
    layers = [setup(T, E, K, N, group, bits, BF, seed=100 + 10 * i) for i in range(3)]
    router = Bank(1, E, K, group, 8, BF, 140)
    rw = tuple(t[0] for t in router.dev)

    def step(h, banks, sync):
        lg = aq.aq_qmm_t(h, *rw, group, 8, out_dtype=F32)
        if sync:
            torch.cuda.synchronize()
        h = aq.aq_moe_swiglu(h, lg, 2, *[b.dev for b in banks], group, bits, rms_eps=1e-6, residual=h)
        if sync:
            torch.cuda.synchronize()
        return h

    x = layers[0][1].to(DEV)
    want = x
    for _ in range(4):
        for banks, _, _ in layers:
            want = step(want, banks, True)
    for _ in range(5):
        h = x
        for _ in range(4):
            for banks, _, _ in layers:
                h = step(h, banks, False)
        assert torch.equal(h, want)
    aq.aq_device_error()


def test_no_tokens():
    banks, x, logits = setup(1, 4, 128, 64, 64, 4, BF)
    y = call(banks, x[:0], logits[:0], 2, 64, 4)
    assert y.shape == (0, 128)


def test_tensors_of_another_device_are_refused():
    banks, x, logits = setup(2, 4, 128, 64, 64, 4, BF)
    dev = [b.dev for b in banks]
    for i in range(3):
        mixed = list(dev)
        mixed[i] = (dev[i][0], dev[i][1].cpu(), dev[i][2])
        with pytest.raises(ValueError):
            aq.aq_moe_swiglu(x.to(DEV), logits.to(DEV), 2, *mixed, 64, 4)
    with pytest.raises(ValueError):
        aq.aq_moe_swiglu(x.to(DEV), logits, 2, *dev, 64, 4)
