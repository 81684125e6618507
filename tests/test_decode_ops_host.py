"""Refusals of the key/value cache and mixture-of-experts calls (CPU only: nothing is launched)."""
import ctypes

import pytest
import torch

from group_wise_affine_qmv_b200 import aq

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def lib():
    from group_wise_affine_qmv_b200 import build
    build.build()
    return aq.load_library()


def side(P=3, H=2, S=16, D=128, group=64, dtype=BF):
    return [torch.zeros(P, H, S, D // 8, dtype=torch.int32), torch.zeros(P, H, S, D // group, dtype=dtype),
            torch.zeros(P, H, S, D // group, dtype=dtype)]


def V(t):
    return None if t is None else ctypes.byref(aq.view(t))


def no_device():
    """Calls that pass every check end at the missing device here; where there is one they would launch on host memory."""
    if torch.cuda.is_available():
        pytest.skip("a valid call on host memory: only where no launch can follow")


def name(lib, st):
    return lib.aq_status_string(st).decode()


def odd(shape, dtype):
    """A tensor of this shape whose data is not 16-byte aligned."""
    n = 1
    for s in shape:
        n *= s
    t = torch.zeros(n + 1, dtype=dtype)[1:].view(shape)
    assert t.data_ptr() % 16
    return t


# ---------------------------------------------------------------------------

@pytest.mark.parametrize("case,status", [
    ("null", "AQ_ERR_NULL"), ("slots", "AQ_ERR_NULL"), ("rank", "AQ_ERR_RANK"), ("dtype", "AQ_ERR_DTYPE"), ("f32", "AQ_ERR_DTYPE"),
    ("vshape", "AQ_ERR_SHAPE"), ("bits8", "AQ_ERR_UNSUPPORTED"), ("bits7", "AQ_ERR_BITS"), ("group", "AQ_ERR_GROUP"),
    ("gmod", "AQ_ERR_GROUP"), ("words", "AQ_ERR_SHAPE"), ("heads", "AQ_ERR_SHAPE"), ("sdtype", "AQ_ERR_DTYPE"),
    ("sshape", "AQ_ERR_SHAPE"), ("vcache", "AQ_ERR_SHAPE"), ("align", "AQ_ERR_ALIGN"), ("wstride", "AQ_ERR_ALIGN"),
    ("inner", "AQ_ERR_STRIDE"), ("expand", "AQ_ERR_OVERLAP"), ("same", "AQ_ERR_OVERLAP"), ("kout", "AQ_ERR_SHAPE"),
    ("koutk", "AQ_ERR_OVERLAP"), ("koutdt", "AQ_ERR_DTYPE"),
])
def test_append_refusals(lib, case, status):
    T, H, D, group, bits = 4, 2, 128, 64, 4
    k, v, slots = torch.zeros(T, H, D, dtype=BF), torch.zeros(T, H, D, dtype=BF), torch.zeros(T, dtype=torch.int64)
    kc, vc, ko, vo = side(), side(), None, None
    sp = slots.data_ptr()
    if case == "null":
        kc[0] = None
    elif case == "slots":
        sp = 0
    elif case == "rank":
        k = torch.zeros(T, H * D, dtype=BF)
    elif case == "dtype":
        v = v.to(F16)
    elif case == "f32":
        k, v = k.float(), v.float()
    elif case == "vshape":
        v = torch.zeros(T + 1, H, D, dtype=BF)
    elif case == "bits8":
        bits = 8
    elif case == "bits7":
        bits = 7
    elif case == "group":
        group = 16
    elif case == "gmod":
        k = v = torch.zeros(T, H, 96, dtype=BF)
    elif case == "words":
        kc[0] = torch.zeros(3, 2, 16, 20, dtype=torch.int32)
    elif case == "heads":
        kc, vc = side(H=4), side(H=4)
    elif case == "sdtype":
        kc[1] = kc[1].to(F16)
    elif case == "sshape":
        kc[2] = torch.zeros(3, 2, 16, 4, dtype=BF)
    elif case == "vcache":
        vc = side(P=2)
    elif case == "align":
        kc[0] = odd((3, 2, 16, 16), torch.int32)
    elif case == "wstride":
        kc[0] = torch.zeros(3, 2, 16, 18, dtype=torch.int32)[..., :16]
    elif case == "inner":
        k = torch.zeros(T, D, H, dtype=BF).transpose(1, 2)
    elif case == "expand":
        kc[0] = torch.zeros(1, 2, 16, 16, dtype=torch.int32).expand(3, 2, 16, 16)
    elif case == "same":
        vc[1] = kc[1]
    elif case == "kout":
        ko = torch.zeros(T, H, D + 8, dtype=BF)
    elif case == "koutk":
        ko = k
    elif case == "koutdt":
        vo = torch.zeros(T, H, D, dtype=F16)
    st = lib.aq_kv_append(V(k), V(v), sp, group, bits, *[V(t) for t in kc + vc], V(ko), V(vo), None)
    assert name(lib, st) == status, lib.aq_last_error_message()


def test_append_accepts_interleaved_halves_up_to_the_launch(lib):
    """Key and value halves of one buffer do not count as overlapping; halves that meet do."""
    no_device()
    k = torch.zeros(2, 2, 128, dtype=BF)
    slots = torch.zeros(2, dtype=torch.int64)

    def call(a, b):
        st = lib.aq_kv_append(V(k), V(k.clone()), slots.data_ptr(), 64, 4, *[V(t) for t in a + b], None, None, None)
        return name(lib, st)

    full = [torch.stack([t, t], 1) for t in side()]                     # [P, 2, H, S, ..]
    got = call([t[:, 0] for t in full], [t[:, 1] for t in full])
    assert got in ("AQ_ERR_CUDA", "AQ_ERR_DEVICE")                      # every check passed; there is no device here
    full = [torch.cat([t, t], -1) for t in side()]                      # halves of a row
    got = call([t[..., :t.shape[-1] // 2] for t in full], [t[..., t.shape[-1] // 2:] for t in full])
    assert got in ("AQ_ERR_CUDA", "AQ_ERR_DEVICE")
    w = torch.zeros(3, 2, 16, 20, dtype=torch.int32)
    a, b = side(), side()
    a[0], b[0] = w[..., :16], w[..., 4:]
    assert call(a, b) == "AQ_ERR_OVERLAP"


# ---------------------------------------------------------------------------

def attention(lib, q, kc, vc, out, group=64, bits=4, pages=True, lengths=True, max_pages=64, scale=1.0, window=0, ws="fit", row=2,
              short=0):
    need = ctypes.c_size_t()
    ids = torch.zeros(8, dtype=torch.int64)
    if ws == "fit":
        st = lib.aq_kv_attention_workspace(V(q), V(kc[0]), max_pages, ctypes.byref(need))
        if st:
            return name(lib, st)
        ws = torch.zeros(need.value + 16, dtype=torch.uint8)
        off = -ws.data_ptr() % 16
        ptr = ws.data_ptr() + off
    else:
        need.value = 1 << 40
        ptr = ws
    st = lib.aq_kv_attention(V(q), *[V(t) for t in kc + vc], group, bits, ids.data_ptr() if pages else None, row, max_pages,
                             ids.data_ptr() if lengths else None, scale, window, V(out), ptr, need.value - short, None)
    return name(lib, st)


@pytest.mark.parametrize("case,status", [
    ("ok", None), ("null", "AQ_ERR_NULL"), ("rank", "AQ_ERR_RANK"), ("f32", "AQ_ERR_DTYPE"), ("d", "AQ_ERR_UNSUPPORTED"),
    ("heads", "AQ_ERR_SHAPE"), ("bits", "AQ_ERR_UNSUPPORTED"), ("group", "AQ_ERR_GROUP"), ("gmod", "AQ_ERR_GROUP"),
    ("sdtype", "AQ_ERR_DTYPE"), ("vcache", "AQ_ERR_SHAPE"), ("outshape", "AQ_ERR_SHAPE"), ("outdtype", "AQ_ERR_DTYPE"),
    ("outq", "AQ_ERR_OVERLAP"), ("outself", "AQ_ERR_OVERLAP"), ("window", "AQ_ERR_SHAPE"), ("nan", "AQ_ERR_SHAPE"),
    ("inf", "AQ_ERR_SHAPE"), ("pages", "AQ_ERR_NULL"), ("lengths", "AQ_ERR_NULL"), ("row", "AQ_ERR_STRIDE"),
    ("wsnull", "AQ_ERR_NULL"), ("wsshort", "AQ_ERR_SHAPE"), ("wsodd", "AQ_ERR_ALIGN"), ("wsq", "AQ_ERR_OVERLAP"),
    ("maxpages", "AQ_ERR_SHAPE"), ("toolong", "AQ_ERR_UNSUPPORTED"), ("align", "AQ_ERR_ALIGN"), ("nohead", "AQ_ERR_SHAPE"),
])
def test_attention_refusals(lib, case, status):
    if status is None:
        no_device()
    q, kc, vc = torch.zeros(2, 1, 4, 128, dtype=BF), side(), side()
    out, kw = torch.zeros(2, 1, 4, 128, dtype=BF), {}
    if case == "null":
        vc[2] = None
    elif case == "rank":
        q = q[0]
    elif case == "f32":
        q = q.float()
    elif case == "d":
        q, kc, vc = torch.zeros(2, 1, 4, 96, dtype=BF), side(D=96, group=32), side(D=96, group=32)
    elif case == "heads":
        q = torch.zeros(2, 1, 3, 128, dtype=BF)
    elif case == "bits":
        kw["bits"] = 8
    elif case == "group":
        kw["group"] = 48
    elif case == "gmod":
        q, kc, vc = torch.zeros(2, 1, 4, 64, dtype=BF), side(D=64), side(D=64)
        kw["group"] = 128
    elif case == "sdtype":
        vc[1] = vc[1].to(F16)
    elif case == "vcache":
        vc = side(S=32)
    elif case == "outshape":
        out = out[:1]
    elif case == "outdtype":
        out = out.float()
    elif case == "outq":
        out = q
    elif case == "outself":
        out = torch.zeros(1, 1, 4, 128, dtype=BF).expand(2, 1, 4, 128)
    elif case == "window":
        kw["window"] = -1
    elif case in ("nan", "inf"):
        kw["scale"] = float(case)
    elif case == "pages":
        kw["pages"] = False
    elif case == "lengths":
        kw["lengths"] = False
    elif case == "row":
        kw["row"] = -1
    elif case == "wsnull":
        kw["ws"] = None
    elif case == "wsshort":
        kw["short"] = 1
    elif case == "wsodd":
        big = torch.zeros(1 << 22, dtype=torch.uint8)
        kw["ws"] = big.data_ptr() - big.data_ptr() % 16 + 20
    elif case == "wsq":
        kw["ws"] = q.data_ptr()
    elif case == "maxpages":
        kw["max_pages"] = -1
    elif case == "toolong":
        kw["max_pages"] = 1 << 30
    elif case == "align":
        kc[0] = odd((3, 2, 16, 16), torch.int32)
    elif case == "nohead":
        kc, vc = side(H=0), side(H=0)
    got = attention(lib, q, kc, vc, out, **kw)
    assert got == status if status else got in ("AQ_ERR_CUDA", "AQ_ERR_DEVICE"), (got, lib.aq_last_error_message())


def test_attention_refuses_more_pages_than_it_counts(lib):
    q, c = torch.zeros(2, 1, 4, 128, dtype=BF), [t[:1].expand(2 ** 31, *t.shape[1:]) for t in side()]
    assert attention(lib, q, c, c, torch.empty_like(q)) == "AQ_ERR_UNSUPPORTED"


def test_attention_workspace_depends_on_sizes_only(lib):
    def need(B, Tq, Hq, D, H, S, pages):
        n = ctypes.c_size_t()
        q, k = torch.zeros(B, Tq, Hq, D, dtype=BF), torch.zeros(2, H, S, D // 8, dtype=torch.int32)
        assert lib.aq_kv_attention_workspace(V(q), V(k), pages, ctypes.byref(n)) == 0
        return n.value

    assert need(1, 1, 8, 128, 8, 16, 4096) == need(64, 1, 8, 128, 8, 16, 4096)
    assert need(0, 1, 8, 128, 8, 16, 64) == 0
    assert need(1, 1, 8, 128, 8, 16, 1) <= need(1, 1, 8, 128, 8, 16, 4096) < 64 << 20


# ---------------------------------------------------------------------------

def bank(E, N, K, group=64, bits=4, dtype=BF):
    return [torch.zeros(E, N, K * bits // 32, dtype=torch.int32), torch.zeros(E, N, K // group, dtype=dtype),
            torch.zeros(E, N, K // group, dtype=dtype)]


@pytest.mark.parametrize("case,status", [
    ("ok", None), ("inplace", None), ("tokens", "AQ_ERR_UNSUPPORTED"), ("topk0", "AQ_ERR_UNSUPPORTED"), ("topk17", "AQ_ERR_UNSUPPORTED"),
    ("topke", "AQ_ERR_SHAPE"), ("experts", "AQ_ERR_UNSUPPORTED"), ("bits3", "AQ_ERR_UNSUPPORTED"), ("bits2g32", "AQ_ERR_UNSUPPORTED"),
    ("bits", "AQ_ERR_BITS"), ("group", "AQ_ERR_GROUP"), ("kmod", "AQ_ERR_GROUP"), ("nmod", "AQ_ERR_GROUP"), ("xdtype", "AQ_ERR_DTYPE"),
    ("ldtype", "AQ_ERR_DTYPE"), ("ydtype", "AQ_ERR_DTYPE"), ("sdtype", "AQ_ERR_DTYPE"), ("lrows", "AQ_ERR_SHAPE"), ("yshape", "AQ_ERR_SHAPE"),
    ("upshape", "AQ_ERR_SHAPE"), ("downshape", "AQ_ERR_SHAPE"), ("sshape", "AQ_ERR_SHAPE"), ("srows", "AQ_ERR_UNSUPPORTED"),
    ("walign", "AQ_ERR_ALIGN"), ("xodd", None), ("rshape", "AQ_ERR_SHAPE"), ("rdtype", "AQ_ERR_DTYPE"), ("ry", "AQ_ERR_OVERLAP"),
    ("yx", "AQ_ERR_OVERLAP"), ("yself", "AQ_ERR_OVERLAP"), ("ylogits", "AQ_ERR_OVERLAP"), ("eps", "AQ_ERR_SHAPE"), ("epsnan", "AQ_ERR_SHAPE"),
    ("null", "AQ_ERR_NULL"), ("wsnull", "AQ_ERR_NULL"), ("wsshort", "AQ_ERR_SHAPE"), ("wsodd", "AQ_ERR_ALIGN"), ("wsx", "AQ_ERR_OVERLAP"),
    ("xrank", "AQ_ERR_RANK"), ("grank", "AQ_ERR_RANK"),
])
def test_moe_refusals(lib, case, status):
    if status is None:
        no_device()
    T, E, K, N, group, bits, top_k, eps = 3, 6, 128, 192, 64, 4, 2, 0.0
    x, lg, y, r = torch.zeros(T, K, dtype=BF), torch.zeros(T, E), torch.zeros(T, K, dtype=BF), None
    gate, up, down = bank(E, N, K), bank(E, N, K), bank(E, K, N)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    wp, wb = ws.data_ptr() + -ws.data_ptr() % 16, (1 << 20) - 16
    if case == "inplace":
        y = r = x
    elif case == "tokens":
        x, lg, y = torch.zeros(65, K, dtype=BF), torch.zeros(65, E), torch.zeros(65, K, dtype=BF)
    elif case.startswith("topk"):
        top_k = {"topk0": 0, "topk17": 17, "topke": 7}[case]
    elif case == "experts":
        lg = torch.zeros(T, 513)
    elif case == "bits3":
        bits = 3
    elif case == "bits2g32":
        bits, group = 2, 32
    elif case == "bits":
        bits = 1
    elif case == "group":
        group = 40
    elif case == "kmod":
        x, y, gate, up = torch.zeros(T, 96, dtype=BF), torch.zeros(T, 96, dtype=BF), bank(E, N, 96, 32), bank(E, N, 96, 32)
    elif case == "nmod":
        gate, up, down = bank(E, 96, K), bank(E, 96, K), bank(E, K, 96, 32)
    elif case == "xdtype":
        x = x.float()
    elif case == "ldtype":
        lg = lg.to(torch.int32)
    elif case == "ydtype":
        y = y.to(F16)
    elif case == "sdtype":
        up[2] = up[2].to(F16)
    elif case == "lrows":
        lg = lg[:2]
    elif case == "yshape":
        y = torch.zeros(T, N, dtype=BF)
    elif case == "upshape":
        up = bank(E, N - 64, K)
    elif case == "downshape":
        down = bank(E, N, K)
    elif case == "sshape":
        gate[1] = torch.zeros(E, N, 3, dtype=BF)
    elif case == "srows":
        down[1] = torch.zeros(E, K, 4, dtype=BF)[..., :3]
    elif case == "walign":
        gate[0] = odd(gate[0].shape, torch.int32)
    elif case == "xodd":
        x = odd((T, K), BF)
    elif case == "rshape":
        r = torch.zeros(T, N, dtype=BF)
    elif case == "rdtype":
        r = torch.zeros(T, K, dtype=F32)
    elif case == "ry":
        big = torch.zeros(T + 1, K, dtype=BF)
        r, y = big[1:], big[:-1]
    elif case == "yx":
        big = torch.zeros(T + 1, K, dtype=BF)
        x, y = big[1:], big[:-1]
    elif case == "yself":
        y = torch.zeros(1, K, dtype=BF).expand(T, K)
    elif case == "ylogits":
        buf = torch.zeros(T * K, dtype=BF)
        y, lg = buf.view(T, K), buf[:T * E].view(T, E)
    elif case == "eps":
        eps = -1e-6
    elif case == "epsnan":
        eps = float("nan")
    elif case == "null":
        down[0] = None
    elif case == "wsnull":
        wp = None
    elif case == "wsshort":
        n = ctypes.c_size_t()
        assert lib.aq_moe_swiglu_workspace(T, top_k, K, N, ctypes.byref(n)) == 0
        wb = n.value - 1
    elif case == "wsodd":
        wp += 8
    elif case == "wsx":
        wp = x.data_ptr()
    elif case == "xrank":
        x = x[None]
    elif case == "grank":
        gate[0] = gate[0][0]
    st = lib.aq_moe_swiglu(V(x), V(lg), top_k, 1, *[V(t) for t in gate + up + down], group, bits, eps, V(r), V(y), wp, wb, None)
    got = name(lib, st)
    assert got == status if status else got in ("AQ_ERR_CUDA", "AQ_ERR_DEVICE"), (got, lib.aq_last_error_message())


def test_binding_checks_ids():
    q, c = torch.zeros(1, 1, 2, 64, dtype=BF), side(D=64, H=1)
    with pytest.raises(TypeError):
        aq.aq_kv_attention(q, c, c, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int64), 64, 4)
    with pytest.raises(ValueError):
        aq.aq_kv_attention(q, c, c, torch.zeros(2, 2, dtype=torch.int64), torch.zeros(1, dtype=torch.int64), 64, 4)
    with pytest.raises(ValueError):
        aq.aq_kv_append(q[0, 0][None], q[0, 0][None], torch.zeros(2, dtype=torch.int64), c, c, 64, 4)
