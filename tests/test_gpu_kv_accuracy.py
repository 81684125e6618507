"""GPU tests of aq_kv_attention's accuracy against the formula in 64 bits, within the bounds that tests/kv_accuracy.py derives:
contexts that a CTA walks whole, value channels far from zero, and every type, head size and group."""
import pytest
import torch

from group_wise_affine_qmv_b200 import aq
from tests import kv_accuracy as acc

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16


def fill(x, group):
    """A cache of what aq_kv_append stores for x [P, H, S, D]."""
    P, H, S, D = x.shape
    new = lambda: (torch.zeros(P, H, S, D // 8, dtype=torch.int32, device=DEV), torch.zeros(P, H, S, D // group, dtype=x.dtype, device=DEV),
                   torch.zeros(P, H, S, D // group, dtype=x.dtype, device=DEV))
    side, spare = new(), new()
    tok = x.transpose(1, 2).reshape(P * S, H, D)
    aq.aq_kv_append(tok, tok, torch.arange(P * S, device=DEV), side, spare, group, 4)
    return side


def case(B, Hq, H, D, group, S, lengths, dtype, Tq=1, far=0.0, shared=False, seed=0):
    """shared: all sequences read the same pages, in the same random order."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    used = [-(-n // S) for n in lengths]
    P = max(used) if shared else sum(used)
    kc = fill(torch.randn(P, H, S, D, generator=g, device=DEV).to(dtype), group)
    v = torch.randn(P, H, S, D, generator=g, device=DEV)
    v[..., ::32] += far
    vc = fill(v.to(dtype), group)
    order = torch.randperm(P, generator=torch.Generator().manual_seed(seed))
    pages = torch.zeros(B, max(used), dtype=torch.int64)
    at = 0
    for b, k in enumerate(used):
        pages[b, :k] = order[at:at + k]
        at += 0 if shared else k
    q = torch.randn(B, Tq, Hq, D, generator=g, device=DEV).to(dtype)
    return q, kc, vc, pages.to(DEV), torch.tensor(lengths, device=DEV)


def check(args, group, which=None, window=0, keep=slice(None)):
    q, kc, vc, pages, lengths = args
    out = aq.aq_kv_attention(q, kc, vc, pages, lengths, group, 4, window=window)
    aq.aq_device_error()
    want, bound, rms = acc.attention(q, kc, vc, pages, lengths.tolist(), group, window, which)
    rows = slice(None) if which is None else list(which)
    off, err = acc.misses(*(x[rows][..., keep] for x in (out, want, bound, rms)))
    assert off == 0 and err < acc.MARGIN, (off, err)


# more items than CTAs fit the device: a CTA walks whole contexts, all of an element's sum in one place
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("H,D,group,n,far", [
    (8, 128, 64, 131072, 0.0),
    (8, 64, 32, 65536, 0.0),
    (8, 256, 128, 32771, 0.0),
    (8, 128, 64, 8192, 20.0),
    (8, 128, 64, 8192, -20.0),
    (8, 128, 32, 65536, 20.0),
])
def test_a_long_context_in_one_cta(H, D, group, n, far, dtype):
    args = case(64, H, H, D, group, 64, [n] * 64, dtype, far=far, shared=True, seed=n)
    # channels around zero next to some far from it: those that the far ones leave few codes
    keep = torch.arange(D, device=DEV) % 32 != 0 if far else slice(None)
    check(args, group, which=range(0, 64, 21), keep=keep)


# query rows in tiles of 8, 16 and 32
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("Hq,Tq", [(4, 5), (8, 3), (32, 2)])
def test_many_rows_over_a_long_context(Hq, Tq, dtype):
    check(case(72, Hq, 4, 128, 64, 64, [24576] * 72, dtype, Tq=Tq, far=20.0, shared=True, seed=Hq), 64, which=(0, 71),
          keep=torch.arange(128, device=DEV) % 32 != 0)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("Hq,H,D,group,S,lengths,Tq,window", [
    (8, 2, 128, 64, 64, [9001], 1, 0),
    (4, 2, 256, 64, 32, [4097, 3], 1, 0),
    (4, 2, 256, 32, 16, [700, 2113], 3, 0),
    (6, 2, 64, 32, 16, [700, 31, 1500], 2, 0),
    (4, 4, 64, 64, 48, [5000], 1, 0),
    (16, 4, 128, 128, 128, [9001, 0, 4096], 1, 0),
    (16, 4, 128, 32, 8, [2500, 801], 4, 1024),
    (14, 2, 128, 64, 1, [1200, 517], 1, 0),
    (8, 2, 128, 64, 64, [130001], 1, 0),
])
def test_errors_stay_near_the_output_rounding(Hq, H, D, group, S, lengths, Tq, window, dtype):
    check(case(len(lengths), Hq, H, D, group, S, lengths, dtype, Tq=Tq, seed=sum(lengths)), group, window=window)
