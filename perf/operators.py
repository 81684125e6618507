"""Cases and plain forms of the decode-step operators on affine group-quantized data: the 4-bit key/value cache (append
and attention) and the mixture-of-experts layer for a few tokens.

A tensor held in `bits` bits stands for ``scale * q + bias`` with one scale and one bias per `group` consecutive elements;
code i of a row sits at bit ``i * bits`` of its little-endian uint32 words.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ----------------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one user's first decode steps: one query token, a few hundred cached ones; only latency counts
        dict(name="attend_one_short", op="attend", batch=1, hq=16, hkv=8, d=128, group=64, page=16, tq=1, lo=300, hi=300,
             window=0, dtype="bf16"),
        # the 32-sequence decode batch of a 0.6B-class decoder (16 query heads on 8 key/value heads of 128), ragged lengths
        dict(name="attend_batch", op="attend", batch=32, hq=16, hkv=8, d=128, group=64, page=64, tq=1, lo=500, hi=4096,
             window=0, dtype="bf16"),
        # one very long document: the work of a single sequence has to be split over the whole GPU
        dict(name="attend_long", op="attend", batch=1, hq=32, hkv=8, d=128, group=128, page=128, tq=1, lo=131071, hi=131071,
             window=0, dtype="f16"),
        # several new tokens per sequence (a checked draft), wide heads, a sliding window, sequences from empty to long
        dict(name="attend_draft_window", op="attend", batch=8, hq=8, hkv=4, d=256, group=32, page=32, tq=5, lo=0, hi=8190,
             window=1024, dtype="bf16"),
        # the largest: a full serving batch at long context
        dict(name="attend_largest", op="attend", batch=32, hq=32, hkv=8, d=128, group=64, page=64, tq=1, lo=9001, hi=32768,
             window=0, dtype="bf16"),
        # one decode step's new keys and values of the 32-sequence batch
        dict(name="append_decode", op="append", tokens=32, hkv=8, d=128, group=64, page=64, dtype="bf16"),
        # a prompt's keys and values at once
        dict(name="append_prompt", op="append", tokens=8191, hkv=8, d=128, group=32, page=16, dtype="f16"),
        # one token through the 128-expert 8-bit bank
        dict(name="moe_one", op="moe", tokens=1, experts=128, topk=8, k=1408, n=2816, group=32, bits=8, renorm=True, rms=False,
             residual=False, dtype="bf16"),
        # the decode batch of 32 tokens through the same bank: nearly every expert is read
        dict(name="moe_batch", op="moe", tokens=32, experts=128, topk=8, k=1408, n=2816, group=32, bits=8, renorm=True,
             rms=True, residual=True, dtype="bf16"),
        # a small 4-bit layer for two tokens: only latency counts
        dict(name="moe_small", op="moe", tokens=2, experts=16, topk=2, k=1024, n=512, group=64, bits=4, renorm=False, rms=False,
             residual=False, dtype="f16"),
        # the most tokens the layer takes at once, 4-bit experts, normalised input and residual as in a decoder block
        dict(name="moe_64_tokens", op="moe", tokens=64, experts=64, topk=6, k=2048, n=1024, group=64, bits=4, renorm=True,
             rms=True, residual=True, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "moe", "moe", "moe"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "attend":
        d = rng.choice([64, 128, 128, 256])
        group = rng.choice([g for g in (32, 64, 128) if g <= d])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
        batch = _log_int(rng, 1, 48)
        tq = rng.choice([1, 1, 1, 2, 3, 5, 8])
        # cached elements (tokens x heads x head size) up to 1/4 of the largest listed case's
        most = max(64, min(131072, (32 * 32768 * 8 * 128 // 4) // (batch * hkv * d)))
        hi = _log_int(rng, 16, most)
        lo = rng.choice([hi, rng.randrange(0, hi + 1), max(0, hi - hi // 3)])
        window = rng.choice([0, 0, 0, _log_int(rng, 16, 4096)])
        page = rng.choice([1, 8, 16, 16, 32, 48, 64, 64, 128, 256])
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, group=group, page=page, tq=tq, lo=lo, hi=hi, window=window,
                    dtype=dtype)
    if op == "append":
        d = rng.choice([64, 128, 128, 256])
        group = rng.choice([g for g in (32, 64, 128) if g <= d])
        return dict(op=op, tokens=_log_int(rng, 1, 8191), hkv=rng.choice([1, 2, 4, 8]), d=d, group=group,
                    page=rng.choice([1, 8, 16, 32, 48, 64, 128]), dtype=dtype)
    bits = rng.choice([4, 4, 8])
    group = rng.choice([32, 64, 128])
    k = 128 * rng.randrange(4, 17)
    n = 128 * rng.randrange(2, 17)
    # as many experts and tokens as keep the banks and the products below those of the largest listed layer
    experts = rng.choice([e for e in (4, 8, 16, 32, 60, 64, 96, 128) if e <= 16 or e * k * n <= 112 * 1408 * 2816])
    topk = rng.randrange(1, min(8, experts) + 1)
    tokens = min(_log_int(rng, 1, 64), max(1, 256 * 1408 * 2816 // (topk * k * n)))
    return dict(op=op, tokens=tokens, experts=experts, topk=topk, k=k, n=n, group=group, bits=bits, renorm=rng.random() < 0.7, rms=rng.random() < 0.5, residual=rng.random() < 0.5,
                dtype=dtype)


# ----------------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _pack(w, group, bits, sdtype):
    """Group-wise affine quantization of w [..., D] in 32 bits: codes int32 [..., D], scales and biases [..., D / group]."""
    g = w.float().unflatten(-1, (-1, group))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = (hi - lo) / float(2 ** bits - 1)
    q = torch.where(s == 0, torch.zeros_like(g), torch.round((g - lo) / s)).clamp_(0, 2 ** bits - 1)
    return q.flatten(-2).to(torch.int32), s.squeeze(-1).to(sdtype), lo.squeeze(-1).to(sdtype)


def _words(q, bits):
    """Codes [..., D] to packed words [..., D * bits / 32]."""
    per = 32 // bits
    sh = torch.arange(per, device=q.device, dtype=torch.int32) * bits
    return (q.unflatten(-1, (-1, per)) << sh).sum(-1, dtype=torch.int32)


def _quantized(shape, std, group, bits, sdtype, gen, spread=None):
    """A tensor of normal values quantized block by block: (words, scales, biases)."""
    lead, d = shape[:-1], shape[-1]
    rows = math.prod(lead)
    wq = torch.empty(rows, d * bits // 32, dtype=torch.int32, device=DEV)
    sc = torch.empty(rows, d // group, dtype=sdtype, device=DEV)
    bi = torch.empty_like(sc)
    step = max(1, (1 << 27) // d)
    for r in range(0, rows, step):
        w = torch.randn(min(step, rows - r), d, generator=gen, device=DEV) * std
        if spread is not None:
            w *= spread
        q, sc[r:r + step], bi[r:r + step] = _pack(w, group, bits, sdtype)
        wq[r:r + step] = _words(q, bits)
    return wq.view(*lead, -1), sc.view(*lead, -1), bi.view(*lead, -1)


def _lengths(case, seed):
    """Cached tokens per sequence, the new ones among them: spread over [lo, hi], the longest at hi."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    g = torch.Generator()
    g.manual_seed(seed + 1)
    n = torch.randint(lo, hi + 1, (b,), generator=g)
    n[0] = lo
    n[-1] = hi
    return n


def _max_pages(case):
    return max(1, -(-case["hi"] // case["page"]))


def prepare(case, seed):
    g = _gen(seed)
    dt = DT[case["dtype"]]
    if case["op"] == "attend":
        b, hkv, d, page = case["batch"], case["hkv"], case["d"], case["page"]
        mp = _max_pages(case)
        n = _lengths(case, seed)
        total = int(((n + page - 1) // page).sum()) + 1
        # keys have a few channels of several times the others' size
        spread = torch.where(torch.rand(d, generator=g, device=DEV) < 0.05, 4.0, 1.0)
        kc = _quantized((total, hkv, page, d), 1.0, case["group"], 4, dt, g, spread)
        vc = _quantized((total, hkv, page, d), 1.0, case["group"], 4, dt, g)
        # sequences own pages in a random order; entries past a sequence's last page are never used
        order = torch.randperm(total, generator=torch.Generator().manual_seed(seed + 2))
        pages = torch.zeros(b, mp, dtype=torch.int64)
        used = (n + page - 1) // page
        at = torch.cumsum(used, 0) - used
        for i in range(b):
            pages[i, :used[i]] = order[at[i]:at[i] + used[i]]
        q = torch.randn(b, case["tq"], case["hq"], d, generator=g, device=DEV).to(dt)
        return dict(case=case, q=q, kc=kc, vc=vc, pages=pages.to(DEV), lengths=n.to(DEV))
    if case["op"] == "append":
        t, hkv, d, page = case["tokens"], case["hkv"], case["d"], case["page"]
        total = -(-t // page) + 2
        # keys and values as the projections leave them: two slices of one [T, 2 H D] result
        kv = torch.randn(t, 2 * hkv * d, generator=g, device=DEV).to(dt)
        # a prompt fills its pages in order, the pages lie anywhere; a token behind the last sequence has slot -1
        order = torch.randperm(total, generator=torch.Generator().manual_seed(seed + 2)).to(DEV)
        i = torch.arange(t, device=DEV)
        slots = order[i // page] * page + i % page
        if t > 4:
            slots[t // 2] = -1
        caches = [(torch.zeros(total, hkv, page, d // 8, dtype=torch.int32, device=DEV),
                   torch.zeros(total, hkv, page, d // case["group"], dtype=dt, device=DEV),
                   torch.zeros(total, hkv, page, d // case["group"], dtype=dt, device=DEV)) for _ in range(2)]
        return dict(case=case, k=kv[:, :hkv * d].unflatten(-1, (hkv, d)), v=kv[:, hkv * d:].unflatten(-1, (hkv, d)),
                    slots=slots, kc=caches[0], vc=caches[1])
    t, e, k, n, group, bits = (case[x] for x in ("tokens", "experts", "k", "n", "group", "bits"))
    gate, up = (_quantized((e, n, k), 0.02, group, bits, dt, g) for _ in range(2))
    down = _quantized((e, k, n), 0.02, group, bits, dt, g)
    x = torch.randn(t, k, generator=g, device=DEV).to(dt)
    logits = torch.randn(t, e, generator=g, device=DEV) * 1.5
    return dict(case=case, x=x, logits=logits, gate=gate, up=up, down=down, r=x if case["residual"] else None)


# ----------------------------------------------------------------------------------------------------------------------
# the operators
# ----------------------------------------------------------------------------------------------------------------------

def _codes(words, bits):
    """Packed words [..., W] to codes as float [..., W * 32 / bits]."""
    sh = torch.arange(32 // bits, device=words.device, dtype=torch.int32) * bits
    return ((words.unsqueeze(-1) >> sh) & (2 ** bits - 1)).flatten(-2).float()


def _values(t, group, bits):
    """What packed words, scales and biases stand for, in 32 bits."""
    q = _codes(t[0], bits).unflatten(-1, (-1, group))
    return (q * t[1].float().unsqueeze(-1) + t[2].float().unsqueeze(-1)).flatten(-2)


def _attend(s):
    c = s["case"]
    q, pages, n = s["q"], s["pages"], s["lengths"]
    b, tq, hq, d = q.shape
    page, hkv = c["page"], c["hkv"]
    span = torch.arange(pages.shape[1] * page, device=q.device)
    # [B, H, tokens, ...] of the pages in the sequences' order
    seq = [tuple(x[pages].transpose(1, 2).flatten(2, 3) for x in t) for t in (s["kc"], s["vc"])]
    k, v = (_values(t, c["group"], 4) for t in seq)
    qf = q.float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4)          # [B, H, heads, Tq, D]
    score = torch.matmul(qf.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (hq // hkv, tq)) / math.sqrt(d)
    pos = (n[:, None] - tq + torch.arange(tq, device=q.device))[:, None, None, :, None]
    seen = (span <= pos) & ((span > pos - c["window"]) if c["window"] else (span >= 0))
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - top), torch.zeros_like(score))
    p = p / p.sum(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (hq // hkv, tq))
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3).to(q.dtype)


def _append(s):
    c = s["case"]
    # a token without a slot stands back for the last one before it that has a slot, which is then stored twice
    i = torch.arange(c["tokens"], device=DEV)
    src = torch.cummax(torch.where(s["slots"] >= 0, i, torch.zeros_like(i)), 0).values
    page, at = s["slots"][src] // c["page"], s["slots"][src] % c["page"]
    new = [_pack(x, c["group"], 4, x.dtype) for x in (s["k"], s["v"])]
    words = [(_words(q, 4), sc, bi) for q, sc, bi in new]
    outs = [_values(w, c["group"], 4).to(s["k"].dtype) for w in words]
    (kq, ks, kb), (vq, vs, vb) = s["kc"], s["vc"]
    kq[page, :, at], ks[page, :, at], kb[page, :, at] = (x[src] for x in words[0])
    vq[page, :, at], vs[page, :, at], vb[page, :, at] = (x[src] for x in words[1])
    return outs + [ks, kb, vs, vb]


def _moe(s):
    c = s["case"]
    x, logits, k = s["x"].float(), s["logits"], c["topk"]
    order = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids, top = order.indices[:, :k], order.values[:, :k]
    e = torch.exp(top - top[:, :1])
    w = e / (e if c["renorm"] else torch.exp(logits - top[:, :1])).sum(-1, keepdim=True)
    if c["rms"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    gate, up, down = (_values(tuple(a[ids] for a in t), c["group"], c["bits"]) for t in (s["gate"], s["up"], s["down"]))
    xs = x[:, None, :, None]
    g, u = torch.matmul(gate, xs), torch.matmul(up, xs)                            # [T, top-k, N, 1]
    y = (torch.matmul(down, g / (1 + torch.exp(-g)) * u).squeeze(-1) * w.unsqueeze(-1)).sum(1)
    if s["r"] is not None:
        y = s["r"].float() + y
    return y.to(s["x"].dtype)


def run(state):
    c = state["case"]
    if own:
        from group_wise_affine_qmv_b200 import aq
        if c["op"] == "attend":
            return aq.aq_kv_attention(state["q"], state["kc"], state["vc"], state["pages"], state["lengths"], c["group"], 4,
                                      window=c["window"])
        if c["op"] == "append":
            k_out = torch.empty(state["k"].shape, dtype=state["k"].dtype, device=DEV)
            v_out = torch.empty_like(k_out)
            aq.aq_kv_append(state["k"], state["v"], state["slots"], state["kc"], state["vc"], c["group"], 4, k_out=k_out,
                            v_out=v_out)
            return [k_out, v_out, *state["kc"][1:], *state["vc"][1:]]
        return aq.aq_moe_swiglu(state["x"], state["logits"], c["topk"], state["gate"], state["up"], state["down"], c["group"],
                                c["bits"], norm_topk=c["renorm"], rms_eps=1e-6 if c["rms"] else 0.0, residual=state["r"])
    return {"attend": _attend, "append": _append, "moe": _moe}[c["op"]](state)


def work(case):
    if case["op"] == "attend":
        hkv, d, tq = case["hkv"], case["d"], case["tq"]
        # cached tokens that some query sees, at the mean of the lengths' range
        n = (case["lo"] + case["hi"]) / 2
        seen = min(n, case["window"] + tq - 1) if case["window"] else n
        tokens = case["batch"] * max(1.0, seen)
        cache = tokens * hkv * 2 * (d / 2 + 4 * d / case["group"])
        return dict(bytes=cache + 2 * 2 * case["batch"] * tq * case["hq"] * d, flops=4 * tokens * tq * case["hq"] * d)
    if case["op"] == "append":
        e = 2 * case["tokens"] * case["hkv"] * case["d"]
        return dict(bytes=e * (2 + 2 + 0.5 + 4 / case["group"]) + 8 * case["tokens"], flops=8 * e)
    t, k, n = case["tokens"], case["k"], case["n"]
    pairs = t * case["topk"]
    # distinct experts of tokens that choose evenly
    met = case["experts"] * (1 - (1 - case["topk"] / case["experts"]) ** t)
    weights = met * 3 * k * n * (case["bits"] / 8 + 4 / case["group"])
    return dict(bytes=weights + 2 * t * k * (3 if case["residual"] else 2) + 4 * t * case["experts"], flops=pairs * 6 * k * n)


# ----------------------------------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ----------------------------------------------------------------------------------------------------------------------

def _stands_for(words, scales, biases, group, bits):
    """scale * q + bias of every element, code by code, in 64 bits."""
    d = words.shape[-1] * 32 // bits
    out = torch.empty(*words.shape[:-1], d, dtype=torch.float64, device=words.device)
    per = 32 // bits
    w = words.to(torch.int64) & 0xFFFFFFFF
    for i in range(per):
        out[..., i::per] = ((w >> (bits * i)) % (1 << bits)).double()
    at = torch.arange(d, device=words.device) // group
    return out.mul_(scales.double()[..., at]).add_(biases.double()[..., at])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        q = s["q"].double()
        out = torch.zeros_like(q)
        tq, per = case["tq"], case["hq"] // case["hkv"]
        for b, n in enumerate(s["lengths"].tolist()):
            if n == 0:
                continue
            first = max(0, n - tq - case["window"] + 1) if case["window"] else 0
            at = torch.arange(first, n, device=DEV)
            page, slot = s["pages"][b][at // case["page"]], at % case["page"]
            for h in range(case["hkv"]):
                k, v = (_stands_for(*(x[page, h, slot] for x in t), case["group"], 4) for t in (s["kc"], s["vc"]))
                for i in range(tq):
                    pos = n - tq + i
                    if pos < 0:
                        continue
                    a = (max(0, pos - case["window"] + 1) if case["window"] else 0) - first
                    z = pos + 1 - first
                    rows = slice(h * per, (h + 1) * per)
                    p = torch.softmax(q[b, i, rows] @ k[a:z].T * case["d"] ** -0.5, -1)
                    out[b, i, rows] = p @ v[a:z]
        return out
    if case["op"] == "append":
        # the codes are defined by 32-bit arithmetic, where ties are met: the values have no 64-bit counterpart
        found = [None, None]
        on = s["slots"] >= 0
        page, slot = s["slots"][on] // case["page"], s["slots"][on] % case["page"]
        for x, cache in ((s["k"], s["kc"]), (s["v"], s["vc"])):
            w = x[on].double().unflatten(-1, (-1, case["group"]))
            lo, hi = w.min(-1).values, w.max(-1).values
            for src in ((hi - lo) / 15, lo):
                dst = torch.zeros(cache[1].shape, dtype=torch.float64, device=DEV)
                dst[page, :, slot] = src
                found.append(dst)
        return found
    x, z = s["x"].double(), s["logits"].double()
    if case["rms"]:
        x = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + 1e-6)
    y = torch.zeros_like(x) if s["r"] is None else s["r"].double()
    for t in range(case["tokens"]):
        # the largest logits, of equal ones the lower ids
        row = z[t].tolist()
        ids = sorted(range(case["experts"]), key=lambda e: (-row[e], e))[:case["topk"]]
        w = torch.softmax(z[t, ids], 0) if case["renorm"] else torch.softmax(z[t], 0)[ids]
        for e, we in zip(ids, w):
            gate, up, down = (_stands_for(*(a[e] for a in m), case["group"], case["bits"]) for m in (s["gate"], s["up"], s["down"]))
            g = gate @ x[t]
            y[t] += we * (down @ (g * torch.sigmoid(g) * (up @ x[t])))
    return y
