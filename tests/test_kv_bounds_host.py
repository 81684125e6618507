"""The attention tests' bounds tell a right result from wrong ones, at the sizes that they are used at: on the CPU, the formula's
own result passes, and results that leave tokens out, read a wrong page or count nothing do not."""
import pytest
import torch

from tests import kv_accuracy as acc
from tests import kv_reference as ref

BF, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("B,Hq,H,D,group,S,n,dtype", [
    (1, 8, 2, 128, 64, 64, 9001, F16), (1, 8, 2, 128, 64, 64, 9001, BF), (1, 4, 2, 256, 64, 32, 4097, BF), (2, 4, 2, 64, 32, 16, 700, BF)])
def test_bounds_reject_results_that_leave_something_out(B, Hq, H, D, group, S, n, dtype):
    pages, P = ref.page_table([n] * B, S, 5)
    kc, vc = ref.make_cache(P, H, S, D, group, dtype, 1), ref.make_cache(P, H, S, D, group, dtype, 2)
    q = torch.randn(B, 1, Hq, D, generator=torch.Generator().manual_seed(3)).to(dtype)
    L = torch.full((B,), n)
    want, bound, rms = acc.attention(q, kc, vc, pages, L, group)

    def wrong(got):
        off, err = acc.misses(got.to(dtype), want, bound, rms)
        return off > 0 and err > 2 * acc.MARGIN

    off, err = acc.misses(want.to(dtype), want, bound, rms)
    assert off == 0 and err < acc.MARGIN
    assert wrong(torch.zeros_like(want))
    assert wrong(acc.attention(q, kc, vc, pages, L // 2, group)[0])            # half of the context
    assert wrong(acc.attention(q, kc, vc, pages, L - n // 18, group)[0])       # without the last eighteenth
    assert wrong(acc.attention(q, kc, vc, pages, L, group, window=n - n // 18)[0])
    swapped = pages.clone()
    swapped[:, -(n // S) // 2] = pages[:, 0]                                   # one page read twice, another not at all
    assert acc.misses(acc.attention(q, kc, vc, swapped, L, group)[0].to(dtype), want, bound, rms)[1] > acc.MARGIN


def to_11_bits(x):
    m, e = torch.frexp(x)
    return torch.ldexp((m * 2.0 ** 11).round() / 2.0 ** 11, e)


@pytest.mark.parametrize("D,group,S,n", [(128, 64, 64, 1500), (64, 32, 16, 700)])
def test_bounds_reject_f16_results_from_one_f16_number_a_weight(D, group, S, n):
    """p s carried in 11 bits, as bf16 outputs have it, is a miss for f16 ones."""
    for dtype, fine in ((F16, False), (BF, True)):
        pages, P = ref.page_table([n], S, 6)
        kc, vc = ref.make_cache(P, 2, S, D, group, dtype, 1), ref.make_cache(P, 2, S, D, group, dtype, 2)
        q = torch.randn(1, 1, 8, D, generator=torch.Generator().manual_seed(3)).to(dtype)
        want, bound, rms = acc.attention(q, kc, vc, pages, [n], group)
        got = acc.attention(q, kc, vc, pages, [n], group, weights=to_11_bits)[0]
        assert (acc.misses(got.to(dtype), want, bound, rms)[1] < acc.MARGIN) == fine
