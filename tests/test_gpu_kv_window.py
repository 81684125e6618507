"""GPU tests of pages that a sliding window has left behind: their entries are not read, whatever the layout."""
import pytest
import torch

from group_wise_affine_qmv_b200 import aq
from tests import kv_accuracy as acc
from tests import kv_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("S,layout", [(1, "phs"), (5, "phs"), (8, "phs"), (8, "psh"), (16, "psh"), (16, "phs"), (48, "phs"), (64, "phs")])
@pytest.mark.parametrize("gone", [-1, 1 << 40])
def test_pages_before_the_window_may_be_gone(S, layout, gone):
    H, Hq, D, group, Tq = 2, 4, 128, 64, 3
    lengths, window = [77, 300, 15, 41, 1100], 20
    pages, P = ref.page_table(lengths, S, 1)
    kc, vc = (ref.make_cache(P, H, S, D, group, BF, s, layout=layout) for s in (2, 3))
    q = torch.randn(len(lengths), Tq, Hq, D, generator=torch.Generator().manual_seed(4)).to(BF)
    freed = pages.clone()
    for b, n in enumerate(lengths):
        freed[b, :max(0, n - Tq - window + 1) // S] = gone
        freed[b, -(-n // S):] = gone
    assert (freed != pages).any()
    dev = [ref.to_dev(c) for c in (kc, vc)]
    L = torch.tensor(lengths, device=DEV)
    a, b = (aq.aq_kv_attention(q.to(DEV), *dev, t.to(DEV), L, group, 4, window=window) for t in (pages, freed))
    aq.aq_device_error()
    assert torch.equal(a, b)
    want, bound, rms = acc.attention(q, kc, vc, pages, lengths, group, window)
    off, err = acc.misses(b, want, bound, rms)
    assert off == 0 and err < acc.MARGIN, (off, err)


def test_a_page_that_a_query_sees_is_still_flagged():
    H, D, group, S, n, window, Tq = 2, 64, 32, 8, 77, 20, 3
    pages, P = ref.page_table([n], S, 1)
    dev = [ref.to_dev(ref.make_cache(P, H, S, D, group, F16, s)) for s in (2, 3)]
    q = torch.randn(1, Tq, 4, D, generator=torch.Generator().manual_seed(4)).to(F16)
    pages[0, (n - Tq - window + 1) // S] = -1
    aq.aq_kv_attention(q.to(DEV), *dev, pages.to(DEV), torch.tensor([n], device=DEV), group, 4, window=window)
    with pytest.raises(aq.AQError) as ei:
        aq.aq_device_error()
    assert ei.value.name == "AQ_ERR_INDEX"


def test_a_window_past_32_bits_sees_every_token():
    H, D, group, S, n, Tq = 2, 64, 32, 16, 77, 3
    pages, P = ref.page_table([n], S, 1)
    dev = [ref.to_dev(ref.make_cache(P, H, S, D, group, F16, s)) for s in (2, 3)]
    q = torch.randn(1, Tq, 4, D, generator=torch.Generator().manual_seed(4)).to(F16).to(DEV)
    run = lambda w: aq.aq_kv_attention(q, *dev, pages.to(DEV), torch.tensor([n], device=DEV), group, 4, window=w)
    whole = run(0)
    for w in (1 << 30, (1 << 31) - 1, 1 << 31, (1 << 32) + 5, (1 << 63) - 1):
        assert torch.equal(run(w), whole), w
    for w in (-1, -(1 << 32) + 5):
        with pytest.raises(aq.AQError):
            run(w)
    aq.aq_device_error()
