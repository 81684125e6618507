"""GPU tests of aq_moe_swiglu's accuracy against the formula in 64 bits, within the bounds that tests/moe_accuracy.py derives."""
import pytest
import torch

from group_wise_affine_qmv_b200 import aq
from tests import moe_accuracy as acc

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda"
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def quantized(E, N, K, group, bits, dtype, gen):
    sides = aq.aq_quantize(torch.randn(E * N, K, generator=gen, device=DEV).mul_(0.02).to(dtype), group, bits)
    return tuple(t.view(E, N, -1) for t in sides)


# one part of an activation (bf16 y), two (f16 and f32 y); scales that come as blocks and stage by stage, tiles of one and two
# blocks of 8 tokens, few items (shared by a CTA's warps) and many
@pytest.mark.parametrize("dtype,ydt", [(BF, BF), (BF, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("T,E,top_k,K,N,group,bits", [
    (1, 8, 2, 512, 256, 64, 4),
    (2, 16, 2, 1024, 512, 64, 4),
    (5, 12, 4, 352, 224, 32, 8),
    (24, 3, 2, 384, 512, 128, 8),
    (40, 64, 4, 256, 512, 64, 4),
    (64, 6, 2, 160, 1024, 32, 8),
    (7, 16, 3, 512, 640, 64, 2),
    (33, 24, 4, 512, 512, 128, 2),
    (16, 4, 2, 128, 8224, 32, 4),
])
def test_errors_stay_near_the_output_rounding(T, E, top_k, K, N, group, bits, dtype, ydt):
    gen = torch.Generator(device=DEV).manual_seed(T + K)
    sides = [quantized(E, n, k, group, bits, dtype, gen) for n, k in ((N, K), (N, K), (K, N))]
    x = torch.randn(T, K, generator=gen, device=DEV).to(dtype)
    logits = torch.randn(T, E, generator=gen, device=DEV) * 1.5
    banks = [acc.Bank(s, group, bits) for s in sides]
    for kw in (dict(), dict(norm_topk=False, rms_eps=1e-6)):
        y = aq.aq_moe_swiglu(x, logits, top_k, *sides, group, bits, out_dtype=ydt, **kw)
        aq.aq_device_error()
        want, bound, rms = acc.layer(x, logits, top_k, banks, ydt, norm=kw.get("norm_topk", True), rms_eps=kw.get("rms_eps", 0.0))
        off, err = acc.misses(y, want, bound, rms)
        assert off == 0 and err < acc.MARGIN, (off, err)


def test_f32_outputs_do_not_depend_on_how_a_bf16_x_is_typed():
    """The same numbers as bf16 and as f16 inputs: an f32 layer is as exact for either."""
    T, E, top_k, K, N, group, bits = 9, 8, 2, 512, 512, 64, 4
    gen = torch.Generator(device=DEV).manual_seed(1)
    # values, scales and biases that both types hold: codes of a bf16 bank whose scales are powers of two
    sides = []
    for n, k in ((N, K), (N, K), (K, N)):
        wq = quantized(E, n, k, group, bits, BF, gen)[0]
        sc = torch.full((E, n, k // group), 2.0 ** -8, device=DEV)
        sides.append((wq, sc, sc * -7.5))
    x = torch.randn(T, K, generator=gen, device=DEV).to(BF)
    logits = torch.randn(T, E, generator=gen, device=DEV)
    ys = []
    for dtype in (BF, F16):
        typed = [(w, s.to(dtype), b.to(dtype)) for w, s, b in sides]
        ys.append(aq.aq_moe_swiglu(x.to(dtype), logits, top_k, *typed, group, bits, out_dtype=F32).double())
    aq.aq_device_error()
    want, _, rms = acc.layer(x, logits, top_k, [acc.Bank(s, group, bits) for s in sides], F32)
    for y in ys:
        assert (y - want).square().mean().sqrt() < acc.MARGIN * (rms.square().mean() + (2.0 ** -24 * want).square().mean()).sqrt()


def test_top_k_past_32_bits_is_refused():
    gen = torch.Generator(device=DEV).manual_seed(2)
    sides = [quantized(4, n, k, 64, 4, BF, gen) for n, k in ((64, 128), (64, 128), (128, 64))]
    x = torch.randn(2, 128, generator=gen, device=DEV).to(BF)
    for k in ((1 << 32) + 2, -(1 << 32) + 2):
        with pytest.raises(aq.AQError):
            aq.aq_moe_swiglu(x, torch.randn(2, 4, device=DEV), k, *sides, 64, 4)
