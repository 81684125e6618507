"""The second half of a decoder layer as the README has it: router and experts both read the normalised hidden state."""
import pytest
import torch

from group_wise_affine_qmv_b200 import aq
from tests import moe_accuracy as acc

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def test_router_and_experts_read_the_normalised_state():
    T, E, top_k, K, N, G, eps = 5, 12, 3, 256, 128, 64, 1e-6
    gen = torch.Generator(device=DEV).manual_seed(1)

    def bank(E, N, K, bits, std):
        return tuple(t.view(E, N, -1) for t in aq.aq_quantize(torch.randn(E * N, K, generator=gen, device=DEV).mul_(std).to(BF), G, bits))

    experts = [bank(E, n, k, 4, 0.02) for n, k in ((N, K), (N, K), (K, N))]
    router = tuple(t[0] for t in bank(1, E, K, 8, 0.2))
    # rows of different sizes: what is not normalised weighs experts differently
    h = (torch.randn(T, K, generator=gen, device=DEV) * torch.tensor([0.1, 0.5, 1.0, 4.0, 20.0], device=DEV)[:, None]).to(BF)
    z, = aq.aq_qmm_t_multi(h, [router], G, 8, out_dtype=F32, rms_eps=eps)
    y = aq.aq_moe_swiglu(h, z, top_k, *experts, G, 4, rms_eps=eps, residual=h, out_dtype=BF)
    aq.aq_device_error()
    w = acc.Bank(tuple(t[None] for t in router), G, 8)
    hn = h.double() / torch.sqrt((h.double() ** 2).mean(-1, keepdim=True) + eps)
    # sums in fp32 of K products: 2^-19 of their magnitudes (as for the layer's own), the norm within 2^-21
    want, mag = hn @ w.v[0].T, hn.abs() @ w.mag[0].T
    assert torch.all((z - want).abs() <= 2.0 ** -19 * mag + 2.0 ** -21 * want.abs())
    want, bound, rms = acc.layer(h, z, top_k, [acc.Bank(s, G, 4) for s in experts], BF, rms_eps=eps, r=h)
    off, err = acc.misses(y, want, bound, rms)
    assert off == 0 and err < acc.MARGIN, (off, err)
