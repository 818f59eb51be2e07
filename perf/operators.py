"""The operators of cached serving: what is measured, in plain form and as the framework's calls.

    write    new keys and values quantised into an 8-bit cache
    read     rows of the 8-bit cache given back in the model's type
    cache    a decoding step over the 8-bit cache
    shared   a decoding step of a batch whose sequences share a prefix

The 8-bit cache holds, for each (sequence, key head, position), the D codes of a
row in e4m3 and one exponent byte b for the whole row: value = code * 2^(b - 127).
The exponent is the smallest for which the row's largest magnitude fits in 448.
"""

import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one decoding step's new token of a mid-size batch: latency alone
        dict(name="write one token", op="write", B=16, Hk=32, n=1, cap=1024, D=128, dtype="bf16", ragged=False),
        # a padded batch of prompts of unlike length, fp16 with narrow heads
        dict(name="write ragged prompts", op="write", B=5, Hk=16, n=1003, cap=2048, D=64, dtype="f16", ragged=True),
        # the keys and values of a long prompt, bound by memory
        dict(name="write long prompt", op="write", B=2, Hk=32, n=4096, cap=8192, D=128, dtype="bf16", ragged=False),
        # a short piece of the cache for a chunk of prompt to attend to
        dict(name="read chunk", op="read", B=3, Hk=8, n=333, cap=1024, D=64, dtype="f16", ragged=True),
        # a whole long cache, handed to a model that keeps 16-bit keys
        dict(name="read whole cache", op="read", B=4, Hk=32, n=8192, cap=8192, D=128, dtype="bf16", ragged=False),
        # one short conversation, grouped heads: latency alone
        dict(name="cache short", op="cache", B=1, H=8, Hk=2, nq=1, cap=1024, D=64, dtype="f16", ragged=True, causal=True),
        # the decoding step that the benchmark times, on the 8-bit cache
        dict(name="cache step", op="cache", B=16, H=32, Hk=32, nq=1, cap=8192, D=128, dtype="bf16", ragged=False, causal=True),
        # drafted tokens checked at once, grouped heads, lengths far apart
        dict(name="cache drafts", op="cache", B=24, H=32, Hk=8, nq=5, cap=16384, D=128, dtype="bf16", ragged=True, causal=True),
        # a few questions about one short text: latency alone
        dict(name="shared short", op="shared", B=3, H=8, Hk=8, nq=1, np=301, cap=64, D=64, dtype="f16", ragged=True, causal=True, own8=False),
        # a batch behind one long instruction, grouped heads
        dict(name="shared step", op="shared", B=64, H=32, Hk=8, nq=1, np=8192, cap=1024, D=128, dtype="bf16", ragged=True, causal=True, own8=False),
        # drafted tokens behind a prefix, the sequences' own part in the 8-bit cache, one key head a query head
        dict(name="shared drafts", op="shared", B=32, H=32, Hk=32, nq=4, np=4096, cap=2048, D=128, dtype="bf16", ragged=True, causal=True, own8=True),
        # many samples of one long document: bound by the products
        dict(name="shared wide", op="shared", B=256, H=32, Hk=4, nq=1, np=32768, cap=256, D=128, dtype="f16", ragged=True, causal=True, own8=True),
    ]


def _span(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("write", "read", "cache", "shared")}
    while True:
        op = rng.choice(("write", "read", "cache", "cache", "shared", "shared"))
        c = dict(op=op, D=rng.choice((64, 128)), ragged=rng.random() < 0.7)
        if op in ("write", "read"):
            c.update(B=_span(rng, 1, 64), Hk=_span(rng, 1, 32), n=_span(rng, 1, 8192), dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
            c["cap"] = c["n"] + _span(rng, 1, 1024)
        else:
            Hk, group = _span(rng, 1, 32), rng.choice((1, 1, 2, 3, 4, 7, 8, 16))
            c.update(Hk=Hk, H=Hk * group, nq=rng.choice((1, 1, 1, 2, 3, 5, 8)), dtype=rng.choice(("bf16", "f16")), causal=rng.random() < 0.8)
            if op == "cache":
                c.update(B=_span(rng, 1, 64), cap=_span(rng, 16, 32768))
            else:
                c.update(B=_span(rng, 2, 256), np=_span(rng, 16, 32768), cap=_span(rng, 8, 2048), own8=rng.random() < 0.5)
            if c["H"] > 64:
                continue
        if _cost(c) <= most[op]:
            return c


def _cost(c):
    """What bounds the draw: bytes, products, and the values that the plain form holds."""
    w = work(c)
    if "nq" not in c:
        return w["bytes"]
    scores = c["B"] * c["H"] * c["nq"] * (c["cap"] + c.get("np", 0))
    return w["bytes"] + w["flops"] / 50 + 4 * scores + 8 * c["B"] * c["Hk"] * c["cap"] * c["D"]


def _mix(case):
    return random.Random(" ".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))


def _counts(case):
    """Where each sequence's rows begin and how many there are (write, read)."""
    r = _mix(case)
    count = [r.randint(case["n"] // 3, case["n"]) if case["ragged"] else case["n"] for _ in range(case["B"])]
    return [r.randint(0, case["cap"] - case["n"]) for _ in count], count


def _lens(case):
    """Each sequence's length in the cache, the new tokens among them."""
    r = _mix(case)
    low = min(case["nq"], case["cap"])
    return [r.randint(low, case["cap"]) if case["ragged"] else case["cap"] for _ in range(case["B"])]


def work(case):
    D, size = case["D"], _BYTES[case["dtype"]]
    if case["op"] in ("write", "read"):
        rows = 2 * case["Hk"] * sum(_counts(case)[1])  # keys and values
        dense = rows if case["op"] == "write" else 2 * case["Hk"] * case["B"] * case["n"]  # read fills what it is not asked for with zeros
        return {"bytes": rows * (D + 1) + dense * D * size + 8 * case["B"], "flops": 2.0 * rows * D}
    lens, nq, own8 = _lens(case), case["nq"], case["op"] == "cache" or case["own8"]
    out = case["B"] * case["H"] * nq
    np_ = case.get("np", 0)
    rows = 2 * case["Hk"] * sum(lens)
    seen = sum(np_ + (n - (nq - 1) / 2 if case["causal"] else n) for n in lens) * case["H"] * nq
    return {"bytes": rows * (D + 1 if own8 else D * size) + 2 * case["Hk"] * np_ * D * size + out * (2 * D * size + 4) + 4 * case["B"], "flops": 4.0 * D * seen}


def _rows(g, shape, dtype):
    """Rows of keys or values: every channel with a spread of its own, a few of them large."""
    gain = torch.rand(shape[-1], generator=g, device="cuda") + 0.5
    gain[torch.randint(0, shape[-1], (2,), generator=g, device="cuda")] = 4.0
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.unbind(0):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * gain)
    return out


def _cache8(g, B, Hk, cap, D):
    codes = [torch.empty(B, Hk, cap, D, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    exps = [torch.empty(B, Hk, cap, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for c, e in zip(codes, exps):
        for b in range(B):
            c[b], e[b] = _quantise(_rows(g, (Hk, cap, D), torch.bfloat16))
    return dict(k=codes[0], v=codes[1], k_exp=exps[0], v_exp=exps[1])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, Hk, cap, D, dtype = case["B"], case["Hk"], case["cap"], case["D"], _TYPES[case["dtype"]]
    s = dict(case=case)

    def int32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    if case["op"] in ("write", "read"):
        start, count = _counts(case)
        s.update(start=int32(start), count=int32(count) if case["ragged"] else None, cache=_cache8(g, B, Hk, cap, D))
        if case["op"] == "write":
            s.update(k=_rows(g, (B, Hk, case["n"], D), dtype), v=_rows(g, (B, Hk, case["n"], D), dtype))
        return s
    s.update(lens=int32(_lens(case)), q=torch.randn(B, case["H"], case["nq"], D, generator=g, device="cuda").to(dtype))
    if case["op"] == "cache" or case["own8"]:
        s["cache"] = _cache8(g, B, Hk, cap, D)
    else:
        s["cache"] = dict(k=_rows(g, (B, Hk, cap, D), dtype), v=_rows(g, (B, Hk, cap, D), dtype))
    if case["op"] == "shared":
        s.update(kp=_rows(g, (Hk, case["np"], D), dtype), vp=_rows(g, (Hk, case["np"], D), dtype))
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import exact_io_aware_37_gb300 as fa

    case, c = s["case"], s["cache"]
    cache = fa.Cache8(c["k"], c["v"], c["k_exp"], c["v_exp"]) if "k_exp" in c else (c["k"], c["v"])
    if case["op"] == "write":
        fa.fa_cache_write(s["k"], s["v"], cache, s["start"], s["count"])
        return c
    if case["op"] == "read":
        return fa.cache_read(cache, s["start"], case["n"], s["count"], dtype=_TYPES[case["dtype"]])
    if case["op"] == "cache":
        return fa.decode_cache(s["q"], cache, s["lens"], causal=case["causal"])
    return fa.decode_shared(s["q"], s["kp"], s["vp"], cache, s["lens"], causal=case["causal"])


def _quantise(x):
    """(codes, exponent bytes) of rows along the last axis; what is not finite becomes NaN."""
    x = x.float()
    mantissa, exponent = torch.frexp(torch.where(x.isfinite(), x.abs(), 0.0).amax(-1))  # amax = mantissa * 2^exponent, mantissa in [0.5, 1)
    e = torch.where(mantissa <= 0.875, exponent - 9, exponent - 8)  # 448 = 0.875 * 2^9
    e = torch.where(mantissa == 0, -127, e).clamp(min=-127)
    return (x * _power(-e)[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _power(e):
    """2^e from its bits: pow() may be off by a rounding."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _values(codes, exps):
    return codes.float() * _power(exps.int() - 127)[..., None]


def _plain(s):
    case, c = s["case"], s["cache"]
    dtype = _TYPES[case["dtype"]]
    if case["op"] in ("write", "read"):
        i = torch.arange(case["n"], device="cuda")
        there = i < (torch.full_like(s["start"], case["n"]) if s["count"] is None else s["count"])[:, None]  # [B, n]
        at = s["start"][:, None] + i
        if case["op"] == "write":
            b, i = there.nonzero(as_tuple=True)
            at = at[b, i]
            for x, codes, exps in ((s["k"], c["k"], c["k_exp"]), (s["v"], c["v"], c["v_exp"])):
                code, e = _quantise(x)
                codes.view(torch.uint8)[b, :, at] = code.view(torch.uint8)[b, :, i]
                exps[b, :, at] = e[b, :, i]
            return c
        at = torch.where(there, at, 0)[:, None, :].expand(-1, case["Hk"], -1)
        rows = at[..., None].expand(-1, -1, -1, case["D"])
        out = []
        for codes, exps in ((c["k"], c["k_exp"]), (c["v"], c["v_exp"])):
            v = _values(codes.view(torch.uint8).gather(2, rows).view(torch.float8_e4m3fn), exps.gather(2, at))
            out.append(torch.where(there[:, None, :, None], v, 0.0).to(dtype))
        return tuple(out)

    # attention: every query's scores over the prefix and over its own sequence, one softmax
    q, lens = s["q"].float(), s["lens"]
    B, H, nq, D = q.shape
    Hk = case["Hk"]
    k, v = (_values(c[x], c[x + "_exp"]) if "k_exp" in c else c[x].float() for x in ("k", "v"))
    q = q.view(B, Hk, H // Hk * nq, D) * D ** -0.5  # the rows of a key head: its query heads' new tokens
    scores = q @ k.transpose(-1, -2)
    np_ = case.get("np", 0)
    if np_:
        flat = q.transpose(0, 1).reshape(Hk, -1, D)
        scores = torch.cat(((flat @ s["kp"].float().transpose(-1, -2)).view(Hk, B, -1, np_).transpose(0, 1), scores), -1)
    j = torch.arange(np_ + case["cap"], device="cuda")
    last = (np_ + lens - 1)[:, None]
    if case["causal"]:
        last = last - nq + 1 + torch.arange(nq, device="cuda").repeat(H // Hk)
    else:
        last = last.expand(-1, q.shape[2])
    seen = (j <= last[..., None])[:, None]  # [B, 1, rows, keys]
    scores = scores.masked_fill(~seen, float("-inf"))
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m.isfinite(), m, 0.0))
    del scores
    l = p.sum(-1, keepdim=True)
    o = p[..., np_:] @ v
    if np_:
        o = o + (p[..., :np_].transpose(0, 1).reshape(Hk, -1, np_) @ s["vp"].float()).view(Hk, B, -1, D).transpose(0, 1)
    o = torch.where(l > 0, o / l, 0.0)
    return o.view(B, H, nq, D).to(dtype), (m + l.log()).view(B, H, nq)


def exact(case, seed):
    """The definitions in 64 bits, one sequence and key head at a time."""
    s = prepare(case, seed)
    c = s["cache"]
    powers = torch.tensor([2.0**i for i in range(-200, 201)], dtype=torch.float64, device="cuda")

    def two(e):
        return powers[(e + 200).long()]

    if case["op"] in ("write", "read"):
        start, count = _counts(case)
        if case["op"] == "write":
            out = {k: c[k].to(torch.float64 if k in ("k", "v") else torch.uint8) for k in c}
            for b in range(case["B"]):
                to = slice(start[b], start[b] + count[b])
                for name in ("k", "v"):
                    x = s[name][b, :, : count[b]].double()
                    e = x.abs().amax(-1).log2().floor() - 8
                    e = torch.where(x.abs().amax(-1) > 448 * two(e), e + 1, e).clamp(min=-127)
                    y = x * two(-e)[..., None]
                    step = two(y.abs().clamp(min=2.0**-6).log2().floor() - 3)  # three bits after the leading one
                    out[name][b, :, to] = (y / step).round() * step
                    out[name + "_exp"][b, :, to] = (e + 127).to(torch.uint8)
            return out
        out = [torch.zeros(case["B"], case["Hk"], case["n"], case["D"], dtype=torch.float64, device="cuda") for _ in range(2)]
        for b in range(case["B"]):
            at = slice(start[b], start[b] + count[b])
            for o, name in zip(out, ("k", "v")):
                o[b, :, : count[b]] = c[name][b, :, at].double() * two(c[name + "_exp"][b, :, at].double() - 127)[..., None]
        return tuple(out)
    if work(case)["flops"] > 4e11:
        return None
    B, H, nq, D = s["q"].shape
    group = H // case["Hk"]
    o = torch.zeros(B, H, nq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, nq), float("-inf"), dtype=torch.float64, device="cuda")
    for h in range(case["Hk"]):
        heads = slice(h * group, (h + 1) * group)
        prefix = [s[x][h].double() for x in ("kp", "vp")] if "kp" in s else [torch.zeros(0, D, dtype=torch.float64, device="cuda")] * 2
        for b, n in enumerate(_lens(case)):
            kv = []
            for x, pre in zip(("k", "v"), prefix):
                t = c[x][b, h, :n].double()
                if "k_exp" in c:
                    t = t * two(c[x + "_exp"][b, h, :n].double() - 127)[:, None]
                kv.append(torch.cat((pre, t)))
            total = kv[0].shape[0]
            t = torch.einsum("gid,jd->gij", s["q"][b, heads].double(), kv[0]) / D ** 0.5
            if case["causal"]:
                late = torch.arange(total, device="cuda")[None] > torch.arange(total - nq, total, device="cuda")[:, None]
                t[:, late] = float("-inf")
            lse[b, heads] = torch.logsumexp(t, -1)
            o[b, heads] = torch.softmax(t, -1).nan_to_num(0.0) @ kv[1]
    return o, lse
