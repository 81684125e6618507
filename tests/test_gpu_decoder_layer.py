"""A decoder layer of the quantized calls as a server runs it: projections, the key/value cache, attention over it, the
output projection, the router and the experts; a prompt and then single tokens, eager and captured."""
import pytest
import torch

from group_wise_affine_qmv_b200 import aq, inputs
from tests import kv_reference as ref
from tests import test_gpu_moe as moe

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
HID, HQ, H, D, S, GROUP, BITS, E, TOPK, INTER = 256, 8, 2, 64, 16, 64, 4, 12, 3, 128
EPS = 1e-6


class Layer:
    def __init__(self, seed):
        self.qkv = [moe.Bank(1, n, HID, GROUP, BITS, BF, seed + i) for i, n in enumerate((HQ * D, H * D, H * D))]
        self.o = moe.Bank(1, HID, HQ * D, GROUP, BITS, BF, seed + 3)
        self.router = moe.Bank(1, E, HID, GROUP, 8, BF, seed + 4, std=0.2)
        self.experts = [moe.Bank(E, n, k, GROUP, BITS, BF, seed + 5 + i)
                        for i, (n, k) in enumerate(((INTER, HID), (INTER, HID), (HID, INTER)))]

    def step(self, x, B, kc, vc, slots, pages, lengths, keep=None):
        """x [B * T, HID], the T newest tokens of each sequence, through the layer; keep collects what each call gave."""
        one = lambda b: tuple(t[0] for t in b.dev)
        T = x.shape[0] // B
        q, k, v = aq.aq_qmm_t_multi(x, [one(b) for b in self.qkv], GROUP, BITS, rms_eps=EPS)
        aq.aq_kv_append(k.view(-1, H, D), v.view(-1, H, D), slots, kc, vc, GROUP, BITS)
        a = aq.aq_kv_attention(q.view(B, T, HQ, D), kc, vc, pages, lengths, GROUP, BITS)
        h = aq.aq_qmm_t_residual(a.view(-1, HQ * D), *one(self.o), GROUP, BITS, x)
        z = aq.aq_qmm_t(h, *one(self.router), GROUP, 8, out_dtype=F32)
        y = aq.aq_moe_swiglu(h, z, TOPK, *[b.dev for b in self.experts], GROUP, BITS, rms_eps=EPS, residual=h)
        if keep is not None:
            keep.update(q=q, a=a, h=h, z=z, y=y)
        return y


def cache(P):
    side = ref.make_cache(P, H, S, D, GROUP, BF, 3)
    return tuple(torch.zeros_like(t, device=DEV) for t in side)


def slots_of(pages, t0, t1):
    t = torch.arange(t0, t1)
    return torch.stack([p[t // S] * S + t % S for p in pages]).reshape(-1).to(DEV)


def test_prompt_and_tokens_through_two_layers():
    B, n0, steps = 3, 20, 6          # twice 30 tokens (the calls with a norm or a residual take up to 32), then 3 at a time
    layers = [Layer(300), Layer(320)]
    pages, P = ref.page_table([n0 + steps] * B, S, 7)
    caches = [(cache(P), cache(P)) for _ in layers]
    dpages = pages.to(DEV)
    x = inputs.normal((B, n0 + steps, HID), 1.0, BF, seed=77).to(DEV)

    def run(t0, t1, check):
        h = x[:, t0:t1].reshape(-1, HID)
        n = torch.full((B,), t1, dtype=torch.int64, device=DEV)
        for layer, (kc, vc) in zip(layers, caches):
            got = {}
            h = layer.step(h, B, kc, vc, slots_of(pages, t0, t1), dpages, n, got)
            if check:                # each call against the formula of what it was given
                aq.aq_device_error()
                sides = [tuple(t.cpu() for t in c) for c in (kc, vc)]
                T = t1 - t0
                want, bound = ref.attention(got["q"].view(B, T, HQ, D).cpu(), *sides, pages, n.cpu(), GROUP, D ** -0.5)
                err = (got["a"].cpu().double() - want).abs()
                assert torch.all(err <= bound), (err / bound).max()
                hh = got["h"].cpu()
                moe.close(got["y"], *moe.reference(hh, got["z"].cpu(), TOPK, layer.experts, True, EPS, hh, BF))
        return h

    run(0, n0 // 2, True)
    run(n0 // 2, n0, True)
    want = [run(n0 + i, n0 + i + 1, i % 3 == 0).clone() for i in range(steps)]

    # the same tokens again from a captured step: slots, lengths and the tokens are read anew by every replay
    xs = torch.zeros(B, HID, dtype=BF, device=DEV)
    slots = torch.full((B,), -1, dtype=torch.int64, device=DEV)
    n = torch.zeros(B, dtype=torch.int64, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h = xs
        for layer, (kc, vc) in zip(layers, caches):
            h = layer.step(h, B, kc, vc, slots, dpages, n)
    for i in range(steps):
        t = n0 + i
        xs.copy_(x[:, t])
        slots.copy_(slots_of(pages, t, t + 1))
        n.fill_(t + 1)
        graph.replay()
        assert torch.equal(h, want[i]), i
    # sequences of a padded batch: no slot, no length; the first one is not touched by them
    slots[1:] = -1
    n[1:] = 0
    graph.replay()
    assert torch.equal(h[0], want[-1][0])
    aq.aq_device_error()
