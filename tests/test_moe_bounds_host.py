"""The expert layer's bounds tell a right result from wrong ones: on the CPU, the formula's own result passes, and results without an
expert, of zeros, or through activations of too few bits do not."""
import pytest
import torch

import oracle
from tests import moe_accuracy as acc
from tests import kv_reference as ref
import numpy as np

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def bank(E, N, K, group, bits, dtype, seed):
    w = torch.randn(E, N, K, generator=torch.Generator().manual_seed(seed)) * 0.02
    Q = oracle.quantize(w.numpy(), group, bits, ref.dname(dtype))
    wq = torch.from_numpy(Q.packed.view(np.int32).copy()).view(E, N, -1)
    return acc.Bank((wq, *(torch.from_numpy(t.view(np.int16).copy()).view(dtype).view(E, N, -1) for t in (Q.scale_bits, Q.bias_bits))), group, bits)


def to_11_bits(x):
    m, e = torch.frexp(x)
    return torch.ldexp((m * 2.0 ** 11).round() / 2.0 ** 11, e)


@pytest.mark.parametrize("T,E,top_k,K,N,group,bits,dtype,ydt", [
    (4, 8, 2, 256, 256, 64, 4, BF, BF), (4, 8, 2, 256, 256, 64, 4, F16, F16), (5, 6, 3, 160, 352, 32, 8, BF, F32),
    (4, 8, 2, 256, 256, 64, 2, F16, F32), (5, 6, 3, 160, 352, 32, 8, F16, F16)])
def test_bounds_reject_results_that_leave_something_out(T, E, top_k, K, N, group, bits, dtype, ydt):
    banks = [bank(E, n, k, group, bits, dtype, i) for i, (n, k) in enumerate(((N, K), (N, K), (K, N)))]
    g = torch.Generator().manual_seed(9)
    x, logits = torch.randn(T, K, generator=g).to(dtype), torch.randn(T, E, generator=g)
    want, bound, rms = acc.layer(x, logits, top_k, banks, ydt)

    def wrong(got):
        off, err = acc.misses(got.to(ydt), want, bound, rms)
        return off > 0 and err > 2 * acc.MARGIN

    off, err = acc.misses(want.to(ydt), want, bound, rms)
    assert off == 0 and err < acc.MARGIN
    assert wrong(torch.zeros_like(want))
    assert wrong(acc.layer(x, logits, top_k - 1, banks, ydt)[0])
    assert wrong(acc.layer(x, logits, top_k, banks, ydt, norm=False)[0])
    few = acc.layer(x, logits, top_k, banks, ydt, carried=to_11_bits)[0]
    assert (acc.misses(few.to(ydt), want, bound, rms)[1] < acc.MARGIN) == (ydt == BF)
