"""GPU tests of the 4-bit key/value cache: aq_kv_append and aq_kv_attention.

The append is held bit for bit to the oracle's quantizer, the attention element by element to the
formula in 64 bits within the bound that tests/kv_reference.py derives.
"""
import numpy as np
import pytest
import torch

import oracle
from group_wise_affine_qmv_b200 import aq, inputs
from tests import kv_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def _expect(x, group):
    """(words, scales, biases) of x [T, H, D]: the formula step by step in fp32.  Against the oracle's quantizer, whose
    scale is (max - min) / 15, stored scales and biases are within a step of their type and codes within one, the latter
    only where the value lies halfway between two codes."""
    T, H, D = x.shape
    f = x.float().numpy().reshape(T, H, D // group, group)
    lo, hi = f.min(-1, keepdims=True), f.max(-1, keepdims=True)
    s = (hi - lo) * (np.float32(1) / np.float32(15))
    q = np.rint(np.divide(f - lo, s, out=np.zeros_like(f), where=s != 0)).astype(np.int64)
    assert q.max() <= 15
    words = (q.reshape(T, H, D // 8, 8) << (4 * np.arange(8))).sum(-1).astype(np.uint32).view(np.int32)
    out = (torch.from_numpy(words), torch.from_numpy(s[..., 0]).to(x.dtype), torch.from_numpy(lo[..., 0]).to(x.dtype))
    Q = oracle.quantize(x.reshape(T * H, D).float().numpy(), group, 4, ref.dname(x.dtype))
    os_, ob = (torch.from_numpy(b.view(np.int16).copy()).view(x.dtype).view(T, H, -1) for b in (Q.scale_bits, Q.bias_bits))
    assert torch.equal(ob, out[2])
    assert (os_.view(torch.int16).int() - out[1].view(torch.int16).int()).abs().max() <= 1
    oq = ref.codes(torch.from_numpy(Q.packed.view(np.int32).copy()).view(T, H, -1)).numpy().reshape(q.shape)
    off = np.nonzero(oq != q)
    exact = ((f - lo).astype(np.float64) * 15 / np.where(s != 0, hi - lo, 1).astype(np.float64))[off]
    assert np.all(np.abs(oq - q)[off] == 1) and np.all(np.abs(exact - np.floor(exact) - 0.5) < 1e-6)
    return out


def _blank(P, H, S, D, group, dtype, layout="phs"):
    shape = (P, H, S) if layout == "phs" else (P, S, H)
    t = [torch.full((*shape, D // 8), 0x5A5A5A5A, dtype=torch.int32, device=DEV),
         torch.full((*shape, D // group), 7.0, dtype=dtype, device=DEV),
         torch.full((*shape, D // group), -7.0, dtype=dtype, device=DEV)]
    return tuple(x if layout == "phs" else x.transpose(1, 2) for x in t)


def _check_append(k, v, slots, kc, vc, group, outs=(None, None)):
    S = kc[0].shape[2]
    for x, side, blank, o in ((k, kc, _blank(*kc[0].shape[:3], k.shape[2], group, k.dtype), outs[0]),
                              (v, vc, _blank(*kc[0].shape[:3], k.shape[2], group, k.dtype), outs[1])):
        want = [b.cpu().clone() for b in blank]
        exp = _expect(x.cpu(), group)
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < want[0].shape[0] * S:
                for w, e in zip(want, exp):
                    w[s // S, :, s % S] = e[t]
        for got, w in zip(side, want):
            g, w = got.cpu().contiguous(), w.contiguous()
            if g.dtype != torch.int32:
                g, w = g.view(torch.int16), w.view(torch.int16)
            assert torch.equal(g, w)
        if o is not None:
            at = torch.arange(x.shape[2]) // group
            vals = torch.from_numpy(np.asarray(ref.codes(exp[0]))).float()
            # fp32: s * q is exact (8 or 11 bits times 4), so one addition rounds, as the fma does
            w = (exp[1].float()[..., at] * vals + exp[2].float()[..., at]).to(x.dtype)
            assert torch.equal(o.cpu(), w)


@pytest.mark.parametrize("T,H,D,group,S,dtype", [
    (1, 1, 64, 32, 1, BF), (1, 8, 128, 64, 16, F16), (33, 3, 96, 32, 7, BF), (32, 8, 128, 64, 64, BF),
    (257, 2, 256, 128, 48, F16), (1000, 5, 128, 128, 32, BF), (5, 1, 64, 64, 8, F16)])
def test_append_matches_the_formula(T, H, D, group, S, dtype):
    P = -(-T // S) + 2
    kv = inputs.normal((T, 2, H, D), 1.0, dtype, seed=T + D).to(DEV)
    k, v = kv[:, 0], kv[:, 1]
    kc, vc = (_blank(P, H, S, D, group, dtype) for _ in range(2))
    slots = torch.randperm(P * S, generator=torch.Generator().manual_seed(T))[:T]
    if T > 2:
        slots[T // 2] = -1
    ko, vo = torch.empty(T, H, D, dtype=dtype, device=DEV), torch.empty(T, H, D, dtype=dtype, device=DEV)
    aq.aq_kv_append(k, v, slots.to(DEV), kc, vc, group, 4, k_out=ko, v_out=vo)
    aq.aq_device_error()
    _check_append(k, v, slots, kc, vc, group, (ko, vo))


def test_append_ties_constant_groups_and_values_of_every_size():
    T, H, D, group = 6, 2, 128, 64
    k = torch.randn(T, H, D, generator=torch.Generator().manual_seed(5))
    k[0] = 3.25                                              # constant: scale 0
    k[1] = (torch.arange(H * D) % 31).view(H, D) * 0.5        # exact halves between codes
    k[2] *= 1e30
    k[3] *= 1e-30
    k[4, :, ::2] = 0.0
    k = k.to(BF)
    v = (-k).flip(0).contiguous()
    kc, vc = (_blank(1, H, 16, D, group, BF) for _ in range(2))
    slots = torch.arange(T) * 2 + 1
    aq.aq_kv_append(k.to(DEV), v.to(DEV), slots.to(DEV), kc, vc, group, 4)
    aq.aq_device_error()
    _check_append(k, v, slots, kc, vc, group)


def test_append_strides_layouts_and_interleaved_halves():
    T, H, D, group, S = 11, 4, 64, 32, 5
    base = inputs.normal((T, H * D * 2 + 3), 1.0, BF, seed=1).to(DEV)
    k = base[:, 1:1 + H * D].unflatten(1, (H, D))             # rows at odd addresses
    v = base[:, H * D + 2:H * D * 2 + 2].unflatten(1, (H, D)).flip(1).transpose(0, 1).contiguous().transpose(0, 1)
    slots = torch.randperm(4 * S, generator=torch.Generator().manual_seed(2))[:T]
    kc, vc = (_blank(4, H, S, D, group, BF, "psh") for _ in range(2))
    ko = torch.full((T, H, D + 1), 9.0, dtype=BF, device=DEV)
    aq.aq_kv_append(k, v, slots.to(DEV), kc, vc, group, 4, k_out=ko[..., 1:])
    aq.aq_device_error()
    _check_append(k, v, slots, kc, vc, group, (ko[..., 1:], None))
    assert torch.all(ko[..., 0] == 9.0)
    both = [torch.stack([a, a], 1) for a in _blank(4, H, S, D, group, BF)]   # [P, 2, H, S, ..]
    kc, vc = (tuple(t[:, i] for t in both) for i in range(2))
    aq.aq_kv_append(k, v, slots.to(DEV), kc, vc, group, 4)
    aq.aq_device_error()
    _check_append(k, v, slots, kc, vc, group)


def test_append_slot_outside_the_cache_is_flagged_and_not_stored():
    T, H, D, group, S = 4, 2, 64, 64, 4
    k, v = (inputs.normal((T, H, D), 1.0, F16, seed=s) for s in (1, 2))
    kc, vc = (_blank(2, H, S, D, group, F16) for _ in range(2))
    slots = torch.tensor([3, 8, -5, 7])                       # 8 = P * S
    aq.aq_kv_append(k.to(DEV), v.to(DEV), slots.to(DEV), kc, vc, group, 4)
    with pytest.raises(aq.AQError) as ei:
        aq.aq_device_error()
    assert ei.value.name == "AQ_ERR_INDEX"
    _check_append(k, v, slots, kc, vc, group)
    aq.aq_device_error()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _case(B, Hq, H, D, group, S, Tq, lengths, dtype, seed=0, layout="phs", std=1.0):
    pages, P = ref.page_table(lengths, S, seed)
    kc = ref.make_cache(P, H, S, D, group, dtype, seed + 1, layout=layout)
    vc = ref.make_cache(P, H, S, D, group, dtype, seed + 2, std=std, layout=layout)
    q = inputs.normal((B, Tq, Hq, D), 1.0, dtype, seed=seed + 3)
    return q, kc, vc, pages, torch.tensor(lengths, dtype=torch.int64)


def _run(q, kc, vc, pages, lengths, group, **kw):
    out = aq.aq_kv_attention(q.to(DEV), ref.to_dev(kc), ref.to_dev(vc), pages.to(DEV), lengths.to(DEV), group, 4, **kw)
    aq.aq_device_error()
    return out


def _close(out, want, bound):
    err = (out.double().cpu() - want).abs()
    worst = (err / bound.clamp_min(1e-300)).max().item()
    assert torch.all(err <= bound), worst


CASES = [
    # B, Hq, H, D, group, S, Tq, lengths, dtype, window
    (1, 1, 1, 64, 64, 16, 1, [1], BF, 0),
    (1, 2, 1, 128, 64, 16, 1, [16], F16, 0),
    (2, 16, 8, 128, 64, 16, 1, [300, 17], BF, 0),
    (3, 8, 8, 128, 32, 32, 1, [0, 65, 640], F16, 0),
    (2, 32, 4, 128, 128, 64, 1, [1000, 63], BF, 0),
    (2, 7, 1, 64, 32, 16, 1, [129, 64], BF, 0),
    (2, 12, 4, 256, 32, 16, 1, [200, 48], F16, 0),
    (1, 8, 2, 256, 128, 128, 1, [700], BF, 0),
    (1, 4, 4, 256, 64, 16, 3, [90], BF, 0),
    (3, 8, 2, 128, 64, 16, 5, [3, 5, 77], BF, 0),          # shorter than the queries: rows that see nothing
    (2, 16, 2, 64, 64, 16, 4, [100, 31], F16, 0),          # 32 query rows: four column tiles
    (2, 24, 2, 128, 32, 16, 7, [210, 6], BF, 0),           # 84 rows: several row tiles
    (1, 20, 2, 256, 64, 32, 2, [130], F16, 0),             # 20 rows at head size 256
    (2, 4, 2, 128, 64, 16, 1, [500, 40], BF, 33),
    (2, 4, 2, 64, 32, 16, 6, [300, 4], F16, 1),            # every query sees itself alone
    (2, 6, 2, 128, 128, 16, 9, [257, 256], BF, 100),
    (3, 4, 2, 128, 64, 1, 1, [37, 1, 18], BF, 0),          # pages of one slot
    (2, 4, 2, 64, 64, 24, 2, [100, 25], F16, 50),          # pages that end inside a tile
    (2, 4, 1, 256, 64, 10, 1, [95, 200], BF, 0),
]


@pytest.mark.parametrize("B,Hq,H,D,group,S,Tq,lengths,dtype,window", CASES)
def test_attention_matches_the_formula(B, Hq, H, D, group, S, Tq, lengths, dtype, window):
    q, kc, vc, pages, n = _case(B, Hq, H, D, group, S, Tq, lengths, dtype, seed=D + S)
    out = _run(q, kc, vc, pages, n, group, window=window)
    want, bound = ref.attention(q, kc, vc, pages, n, group, D ** -0.5, window)
    _close(out, want, bound)
    for b, m in enumerate(lengths):
        assert torch.all(out[b, :max(0, Tq - m)] == 0)


@pytest.mark.parametrize("layout,S", [("psh", 16), ("psh", 5), ("phs", 5)])
def test_attention_layouts_give_the_same_bits(layout, S):
    """Token-major storage and pages of any size: the same result as the dense layout, bit for bit."""
    lengths = [140, 33]
    q, kc, vc, pages, n = _case(2, 8, 4, 128, 64, 16, 1, lengths, BF, seed=3)
    base = _run(q, kc, vc, pages, n, 64)
    # the same tokens in a cache of another page size and layout
    P2 = 2 * -(-140 // S)
    pages2 = torch.arange(P2).flip(0).view(2, -1)
    k2, v2 = (ref.make_cache(P2, 4, S, 128, 64, BF, 9, layout=layout) for _ in range(2))
    for src, dst in ((kc, k2), (vc, v2)):
        for b, m in enumerate(lengths):
            t = torch.arange(m)
            for a, d in zip(src, dst):
                d[pages2[b][t // S], :, t % S] = a[pages[b][t // 16], :, t % 16]
    out = _run(q, k2, v2, pages2, n, 64)
    assert torch.equal(out, base)


@pytest.mark.parametrize("D,group", [(128, 64), (128, 32), (256, 32), (256, 64), (64, 64)])
def test_attention_scales_past_their_boundary(D, group):
    """Scales and biases that start one element past where a row of them could be copied whole."""
    q, kc, vc, pages, n = _case(2, 8, 4, D, group, 16, 1, [150, 37], F16, seed=12)
    base = _run(q, kc, vc, pages, n, group)

    def past(side):
        dev = list(ref.to_dev(side))
        for i in (1, 2):
            flat = torch.zeros(dev[i].numel() + 1, dtype=dev[i].dtype, device=DEV)
            flat[1:] = dev[i].flatten()
            dev[i] = flat[1:].view(dev[i].shape)
        return tuple(dev)

    out = aq.aq_kv_attention(q.to(DEV), past(kc), past(vc), pages.to(DEV), n.to(DEV), group, 4)
    aq.aq_device_error()
    assert torch.equal(out, base)


def test_attention_strided_queries_outputs_and_table():
    q, kc, vc, pages, n = _case(2, 6, 3, 64, 32, 16, 2, [70, 19], BF, seed=4)
    base = _run(q, kc, vc, pages, n, 32)
    big = torch.zeros(2, 2, 9, 67, dtype=BF, device=DEV)
    qs = big[:, :, 1:7, 2:66]
    qs.copy_(q)
    store = torch.full((6, 2, 2, 65), 3.0, dtype=BF, device=DEV)
    o = store.permute(1, 2, 0, 3)[..., 1:]
    wide = torch.zeros(2, pages.shape[1] + 3, dtype=torch.int64, device=DEV)
    wide[:, :pages.shape[1]] = pages.to(DEV)
    aq.aq_kv_attention(qs, ref.to_dev(kc), ref.to_dev(vc), wide[:, :pages.shape[1]], n.to(DEV), 32, 4, out=o)
    aq.aq_device_error()
    assert torch.equal(o, base)
    assert torch.all(store[..., 0] == 3.0)


def test_attention_long_contexts_are_split_and_repeat_bit_for_bit():
    for B, Hq, H, D, group, S, lengths in ((1, 8, 2, 128, 64, 64, [9001]), (3, 4, 2, 64, 64, 16, [5000, 1, 2049]),
                                           (1, 2, 1, 256, 128, 32, [4097])):
        q, kc, vc, pages, n = _case(B, Hq, H, D, group, S, 1, lengths, F16, seed=6)
        a = _run(q, kc, vc, pages, n, group)
        want, bound = ref.attention(q, kc, vc, pages, n, group, D ** -0.5)
        _close(a, want, bound)
        assert torch.equal(a, _run(q, kc, vc, pages, n, group))


def test_attention_many_sequences_share_the_ctas():
    """More items than CTAs, lengths from nothing to several pages: CTAs begin and end inside items."""
    g = torch.Generator().manual_seed(5)
    for B, Hq, H, D, group, S, Tq, window in ((70, 16, 8, 128, 64, 16, 1, 0), (150, 8, 4, 64, 32, 8, 2, 0),
                                              (97, 20, 5, 256, 128, 32, 3, 40)):
        lengths = torch.randint(0, 300, (B,), generator=g).tolist()
        lengths[3], lengths[7] = 0, 1
        q, kc, vc, pages, n = _case(B, Hq, H, D, group, S, Tq, lengths, BF, seed=8)
        a = _run(q, kc, vc, pages, n, group, window=window)
        _close(a, *ref.attention(q, kc, vc, pages, n, group, D ** -0.5, window))
        assert torch.equal(a, _run(q, kc, vc, pages, n, group, window=window))


def test_attention_a_warp_walks_many_tiles():
    """Contexts so long that every warp of a full device has more tiles than it fetches page numbers for at once; the
    pages repeat, which keeps the cache small."""
    B, Hq, H, D, group, S = 2, 16, 8, 64, 64, 16
    lengths = [130001, 120007]
    kc = ref.make_cache(64, H, S, D, group, F16, 31)
    vc = ref.make_cache(64, H, S, D, group, F16, 32)
    g = torch.Generator().manual_seed(33)
    pages = torch.randint(0, 64, (B, -(-max(lengths) // S)), generator=g)
    q = inputs.normal((B, 1, Hq, D), 1.0, F16, seed=34)
    n = torch.tensor(lengths)
    _close(_run(q, kc, vc, pages, n, group), *ref.attention(q, kc, vc, pages, n, group, D ** -0.5))


def test_attention_ignores_what_lies_behind_a_sequence():
    """Stale slots of the last page with NaN and infinite scales, pages past the end, other sequences' pages."""
    q, kc, vc, pages, n = _case(2, 4, 2, 128, 64, 16, 3, [37, 2], BF, seed=7)
    base = _run(q, kc, vc, pages, n, 64, window=0)
    for side in (kc, vc):
        for b, m in enumerate(n.tolist()):
            last = pages[b][(m - 1) // 16]
            side[1][last, :, (m - 1) % 16 + 1:] = float("nan")
            side[2][last, :, (m - 1) % 16 + 1:] = float("inf")
            side[0][last, :, (m - 1) % 16 + 1:] = -1
    pages = torch.cat([pages, torch.full((2, 2), 1 << 40)], 1)   # ids that no length reaches
    assert torch.equal(_run(q, kc, vc, pages, n, 64), base)


def test_attention_window_hides_broken_old_tokens():
    q, kc, vc, pages, n = _case(1, 2, 1, 64, 64, 16, 2, [100], F16, seed=8)
    base = _run(q, kc, vc, pages, n, 64, window=20)
    for side in (kc, vc):
        for t in range(100 - 2 - 20 + 1):                        # before the first query's window
            side[1][pages[0][t // 16], :, t % 16] = float("nan")
            side[2][pages[0][t // 16], :, t % 16] = float("-inf")
    assert torch.equal(_run(q, kc, vc, pages, n, 64, window=20), base)


def test_attention_a_broken_token_reaches_only_queries_that_see_it():
    """NaN in a token: queries at or after it give NaN, earlier ones of the same run stay as they were."""
    q, kc, vc, pages, n = _case(1, 2, 1, 128, 128, 16, 4, [50], BF, seed=9)
    base = _run(q, kc, vc, pages, n, 128)
    kc[1][pages[0][48 // 16], :, 48 % 16] = float("nan")         # the third of the four query tokens
    out = _run(q, kc, vc, pages, n, 128)
    assert torch.equal(out[:, :2], base[:, :2]) and torch.all(torch.isnan(out[:, 2:]))
    kc[1][pages[0][48 // 16], :, 48 % 16] = 1.0
    vc[1][pages[0][48 // 16], :, 48 % 16] = float("nan")
    out = _run(q, kc, vc, pages, n, 128)
    assert torch.all(torch.isfinite(out[:, :2])) and torch.all(torch.isnan(out[:, 2:]))


def test_attention_a_broken_value_inside_a_tile_that_earlier_queries_see():
    q, kc, vc, pages, n = _case(1, 2, 1, 64, 32, 16, 4, [60], BF, seed=15)
    base = _run(q, kc, vc, pages, n, 32)
    for a, x in ((1, float("inf")), (2, float("nan"))):           # token 58 of tile 48..63: queries at 56..59
        old = vc[a].clone()
        vc[a][pages[0][3], :, 10] = x
        out = _run(q, kc, vc, pages, n, 32)
        assert torch.equal(out[:, :2], base[:, :2]) and not torch.any(torch.isfinite(out[:, 2:]))
        vc[a].copy_(old)


@pytest.mark.parametrize("dtype", [BF, F16])
def test_attention_scales_of_every_size(dtype):
    """Value scales that differ by 2^12 between tokens, large and tiny scores, queries of very different sizes."""
    q, kc, vc, pages, n = _case(2, 8, 2, 128, 64, 16, 1, [300, 45], dtype, seed=10)
    g = torch.Generator().manual_seed(1)
    f = 2.0 ** torch.randint(-6, 7, vc[1].shape[:3], generator=g)
    vc = (vc[0], (vc[1].float() * f[..., None]).to(dtype), (vc[2].float() * f[..., None]).to(dtype))
    q = q.clone()
    q[:, :, 0] *= 40.0
    q[:, :, 1] *= 2.0 ** -10
    q[:, :, 2] = 0.0
    q[:, :, 3, ::7] *= 30.0
    out = _run(q, kc, vc, pages, n, 64)
    want, bound = ref.attention(q, kc, vc, pages, n, 64, 128 ** -0.5)
    _close(out, want, bound)
    for scale in (0.0, -0.2, 1.5):
        out = _run(q, kc, vc, pages, n, 64, scale=scale)
        want, bound = ref.attention(q, kc, vc, pages, n, 64, scale)
        _close(out, want, bound)


def test_attention_scores_that_grow_along_the_context():
    """The running reference has to move again and again: keys that grow along the sequence."""
    q, kc, vc, pages, n = _case(1, 4, 1, 64, 64, 16, 1, [1500], BF, seed=11)
    for t in range(1500):
        for a in (1, 2):
            kc[a][pages[0][t // 16], :, t % 16] *= 0.02 * (t + 1)
    out = _run(q, kc, vc, pages, n, 64)
    want, bound = ref.attention(q, kc, vc, pages, n, 64, 64 ** -0.5)
    _close(out, want, bound)


def test_attention_bad_pages_and_lengths_are_flagged():
    q, kc, vc, pages, n = _case(2, 2, 1, 64, 64, 16, 1, [40, 20], BF, seed=12)
    P = kc[0].shape[0]
    dev = (q.to(DEV), ref.to_dev(kc), ref.to_dev(vc))
    base = _run(q, kc, vc, pages, n, 64)
    for bad in (P, -1, 1 << 40):
        p2 = pages.clone()
        p2[0, 1] = bad
        out = aq.aq_kv_attention(*dev, p2.to(DEV), n.to(DEV), 64, 4)
        with pytest.raises(aq.AQError) as ei:
            aq.aq_device_error()
        assert ei.value.name == "AQ_ERR_INDEX"
        assert torch.equal(out[1], base[1]) and torch.all(torch.isfinite(out[0]))
    for lens in ([1 << 40, 20], [-3, 20]):
        out = aq.aq_kv_attention(*dev, pages.to(DEV), torch.tensor(lens).to(DEV), 64, 4)
        with pytest.raises(aq.AQError) as ei:
            aq.aq_device_error()
        assert ei.value.name == "AQ_ERR_INDEX"
        assert torch.equal(out[1], base[1])
    assert torch.all(out[0] == 0)
    aq.aq_device_error()


def test_attention_empty_calls():
    q, kc, vc, pages, n = _case(2, 2, 1, 64, 64, 16, 1, [0, 0], BF, seed=13)
    assert torch.all(_run(q, kc, vc, pages, n, 64) == 0)
    assert torch.all(_run(q, kc, vc, pages[:, :0], n, 64) == 0)
    e = aq.aq_kv_attention(q[:0].to(DEV), ref.to_dev(kc), ref.to_dev(vc), pages[:0].to(DEV), n[:0].to(DEV), 64, 4)
    assert e.shape == (0, 1, 2, 64)
    aq.aq_kv_append(q[:0, 0].to(DEV)[:, :1], q[:0, 0].to(DEV)[:, :1], n[:0].to(DEV), ref.to_dev(kc), ref.to_dev(vc), 64, 4)
    aq.aq_device_error()


def test_attention_captured_replayed_and_on_two_streams():
    q, kc, vc, pages, n = _case(2, 8, 4, 128, 64, 16, 1, [700, 90], BF, seed=14)
    dq, dk, dv, dp, dn = q.to(DEV), ref.to_dev(kc), ref.to_dev(vc), pages.to(DEV), n.to(DEV)
    base = _run(q, kc, vc, pages, n, 64)
    other = _run(q.flip(0), kc, vc, pages.flip(0), n.flip(0), 64)
    out = torch.empty_like(dq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        aq.aq_kv_attention(dq, dk, dv, dp, dn, 64, 4, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, base)
    dq.copy_(q.flip(0))
    dp.copy_(pages.flip(0))
    dn.copy_(n.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, other)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for s, o in zip(streams, outs):
            with torch.cuda.stream(s):
                o.append(aq.aq_kv_attention(dq, dk, dv, dp, dn, 64, 4))
    torch.cuda.synchronize()
    assert all(torch.equal(o, other) for o in outs[0] + outs[1])
    aq.aq_device_error()


@pytest.mark.parametrize("S", [64, 63])
def test_caches_past_four_gigabytes(S):
    """Offsets of more than 32 bits: appended to and read from the last pages of a large cache as from a small one."""
    P, H, D, group, T = 140000, 8, 128, 64, 150
    k, v = (inputs.normal((T, H, D), 1.0, BF, seed=s).to(DEV) for s in (40, 41))
    q = inputs.normal((1, 1, 16, D), 1.0, BF, seed=42).to(DEV)
    n = torch.tensor([T], device=DEV)
    got = []
    for pages in (P, 4):
        kc, vc = (tuple(torch.zeros(pages, H, S, w, dtype=t, device=DEV) for w, t in ((D // 8, torch.int32), (D // group, BF), (D // group, BF)))
                  for _ in range(2))
        ids = torch.tensor([[pages - 1, pages - 3, pages - 2]], device=DEV)
        t = torch.arange(T, device=DEV)
        aq.aq_kv_append(k, v, ids[0, t // S] * S + t % S, kc, vc, group, 4)
        got.append(aq.aq_kv_attention(q, kc, vc, ids, n, group, 4))
        assert all(int(x[:pages - 3].count_nonzero()) == 0 for c in (kc, vc) for x in c)
        del kc, vc
    assert torch.equal(got[0], got[1]) and got[0].abs().max() > 0
    aq.aq_device_error()
    torch.cuda.empty_cache()


def test_tensors_of_another_device_are_refused():
    q, kc, vc, pages, n = _case(1, 2, 1, 64, 64, 16, 1, [20], BF)
    dk, dv = ref.to_dev(kc), ref.to_dev(vc)
    with pytest.raises(ValueError):
        aq.aq_kv_attention(q.to(DEV), (dk[0], dk[1].cpu(), dk[2]), dv, pages.to(DEV), n.to(DEV), 64, 4)
    with pytest.raises(ValueError):
        aq.aq_kv_append(q[0].to(DEV), q[0], n.to(DEV), dk, dv, 64, 4)
    aq.aq_device_error()


def test_append_then_attention_token_by_token():
    """A prompt and then single tokens: the cache as appended gives what the whole sequence's own keys and values give."""
    B, Hq, H, D, group, S, n0, steps = 2, 4, 2, 128, 64, 16, 30, 6
    k, v = (inputs.normal((B, n0 + steps, H, D), 1.0, BF, seed=s) for s in (20, 21))
    q = inputs.normal((B, steps, Hq, D), 1.0, BF, seed=22)
    pages, P = ref.page_table([n0 + steps] * B, S, 1)
    kc, vc = (_blank(P, H, S, D, group, BF) for _ in range(2))

    def slots(t0, t1):
        t = torch.arange(t0, t1)
        return torch.stack([pages[b][t // S] * S + t % S for b in range(B)]).reshape(-1).to(DEV)

    def put(t0, t1):
        aq.aq_kv_append(k[:, t0:t1].reshape(-1, H, D).to(DEV), v[:, t0:t1].reshape(-1, H, D).to(DEV), slots(t0, t1), kc, vc,
                        group, 4)

    put(0, n0)
    got = []
    for i in range(steps):
        put(n0 + i, n0 + i + 1)
        n = torch.full((B,), n0 + i + 1, dtype=torch.int64, device=DEV)
        got.append(aq.aq_kv_attention(q[:, i:i + 1].to(DEV), kc, vc, pages.to(DEV), n, group, 4))
    aq.aq_device_error()
    side = [tuple(x.cpu() for x in c) for c in (kc, vc)]
    want, bound = ref.attention(q, *side, pages, torch.full((B,), n0 + steps), group, D ** -0.5)
    _close(torch.cat(got, 1), want, bound)
