"""The attention side of a served transformer layer, around this library's
sparse linear layers: what each operator is, on which sizes it is measured,
and what it has to compute.

    rope    the QKV projection's rows -> per-head RMS norm and rotation of the
            queries and keys; keys and values appended to the paged cache
    decode  attention of one new token per sequence over the paged cache
    prompt  causal attention of a ragged batch of new tokens over the paged
            cache (which holds them, and any earlier tokens of the sequence)

decode and prompt take a sliding window and a few first tokens that stay
visible.  The cache is [pages, kv heads, page size, head dim] (any strides), in
bf16 or in e4m3 codes with a scale per kv head.

With ``own`` false run() computes an operator in elementary torch operations
in 32 bits; with ``own`` true it calls the library.
"""
import math

import torch

own = False

# ---------------------------------------------------------------------- cases
# 32 query and 8 kv heads of 128: the head layout whose QKV projection is the
# 6144 x 4096 linear of this library's decode measurements.  28 and 4 heads of
# 64 (7 query heads per kv head, which divide no tile evenly) are the odd ones.
_HEADS = dict(hq=32, hkv=8, d=128, page=64, cache="bf16", order="head")
_ODD = dict(hq=28, hkv=4, d=64, page=16, cache="bf16", order="token")


def listed():
    return [
        # one sequence, one new token: the latency of the smallest call
        dict(_HEADS, name="rope-1", op="rope", tokens=1, rot=128, norm=True, pairs="half"),
        # a decode batch into an 8-bit cache (the decode sweep's largest batch)
        dict(_HEADS, name="rope-64-e4m3", op="rope", tokens=64, rot=128, norm=True, pairs="half") | dict(cache="e4m3"),
        # the 3000 tokens of the group-wise linear, rotated in part, in neighbouring pairs, without a norm
        dict(_ODD, name="rope-3000-odd", op="rope", tokens=3000, rot=32, norm=False, pairs="even"),
        # a long prompt: bound by memory
        dict(_HEADS, name="rope-8192", op="rope", tokens=8192, rot=128, norm=True, pairs="half"),
        # one short conversation: the latency of the smallest call
        dict(_HEADS, name="decode-1x1000", op="decode", batch=1, low=1000, high=1000, window=0, sinks=0),
        # one long document: a single row to be spread over the whole GPU
        dict(_HEADS, name="decode-1x131071", op="decode", batch=1, low=131071, high=131071, window=0, sinks=0),
        # a serving batch of very different lengths in an 8-bit cache
        dict(_HEADS, name="decode-64-ragged-e4m3", op="decode", batch=64, low=1, high=16000, window=0, sinks=0)
        | dict(cache="e4m3"),
        # a large batch with a sliding window and sinks, odd heads, small pages, tokens outermost in a page
        dict(_ODD, name="decode-128-window", op="decode", batch=128, low=1, high=9000, window=2000, sinks=4),
        # short prompts of different lengths in one call
        dict(_HEADS, name="prompt-16-short", op="prompt", batch=16, qlow=1, qhigh=200, prefix=0, window=0, sinks=0)
        | dict(page=16),
        # one long prompt: bound by the matrix products
        dict(_HEADS, name="prompt-8192", op="prompt", batch=1, qlow=8192, qhigh=8192, prefix=0, window=0, sinks=0),
        # a longer one under a sliding window with sinks, odd heads
        dict(_ODD, name="prompt-16001-window", op="prompt", batch=1, qlow=16001, qhigh=16001, prefix=0, window=4096,
             sinks=4),
        # pieces of two prompts whose first 14000 tokens are in an 8-bit cache
        dict(_HEADS, name="prompt-piece-e4m3", op="prompt", batch=2, qlow=1500, qhigh=2048, prefix=14000, window=0,
             sinks=0) | dict(cache="e4m3"),
    ]


_MOST_CACHE = 1 << 30     # bytes of keys and values a drawn call reads at most
_MOST_SCORES = 32 * 8192 * 8192  # query heads x queries x keys of a drawn prompt call (padded) at most
_BARRED = 3072            # no size of a drawn case is this


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    while True:
        c = dict(op=rng.choice(("rope", "decode", "prompt")), hkv=rng.choice((1, 2, 4, 8)),
                 hq=rng.choice((1, 2, 3, 4, 5, 7, 8, 16)), d=rng.choice((64, 128)),
                 page=rng.choice((16, 32, 64, 128)), cache=rng.choice(("bf16", "e4m3")),
                 order=rng.choice(("head", "token")))
        c["hq"] *= c["hkv"]
        window = rng.choice((0, 0, _log(rng, 16, 8192)))
        sinks = rng.choice((0, 1, 4, _log(rng, 1, 128))) if window else 0
        if c["op"] == "rope":
            c.update(tokens=_log(rng, 1, 8192), norm=rng.random() < 0.7, pairs=rng.choice(("half", "even")),
                     rot=16 * rng.randint(0, c["d"] // 16) if rng.random() < 0.4 else c["d"])
            fits = c["tokens"] * (c["hq"] + 2 * c["hkv"]) * c["d"] <= 8192 * 6144
        elif c["op"] == "decode":
            high = _log(rng, 1, 131071)
            c.update(batch=_log(rng, 1, 256), low=rng.choice((1, high)), high=high, window=window, sinks=sinks)
            fits = c["batch"] * high * c["hkv"] * c["d"] * 4 <= _MOST_CACHE
        else:
            high = _log(rng, 1, 8192)
            c.update(batch=_log(rng, 1, 32), qlow=rng.choice((1, high)), qhigh=high,
                     prefix=rng.choice((0, 0, _log(rng, 1, 16000))), window=window, sinks=sinks)
            fits = c["batch"] * c["hq"] * high * (high + c["prefix"]) <= _MOST_SCORES
        sizes = [v for v in c.values() if isinstance(v, int)]
        sizes += [(c["hq"] + 2 * c["hkv"]) * c["d"], c["hq"] * c["d"], c["hkv"] * c["d"]]
        sizes += _lengths(c) if c["op"] != "rope" else []
        if fits and c["hq"] <= 64 and _BARRED not in sizes:
            return c


def _spread(n, low, high):
    """n lengths over [low, high], in no order, the same for every seed."""
    return [low + int((high - low + 1) * math.fmod((i + 1) * 0.6180339887498949, 1.0)) for i in range(n)]


def _lengths(c):
    """New tokens of each sequence ("prompt"), or tokens in its cache ("decode")."""
    return _spread(c["batch"], c.get("qlow", c.get("low")), c.get("qhigh", c.get("high")))


def _seen(length, window, sinks):
    """Keys that the last of `length` tokens sees."""
    return length if not window else min(length, window + min(sinks, max(0, length - window)))


def work(case):
    c = case
    e = 1 if c["cache"] == "e4m3" else 2
    if c["op"] == "rope":
        heads = c["hq"] + 2 * c["hkv"]
        n = c["tokens"] * c["d"]
        # tables: one row of cosines and sines per token; positions and slots: 4 + 8 bytes
        by = n * heads * 2 + n * c["hq"] * 2 + n * 2 * c["hkv"] * e + c["tokens"] * (c["rot"] * 4 + 12)
        return {"bytes": by, "flops": n * (c["hq"] + c["hkv"]) * ((4 if c["norm"] else 0) + 3)}
    if c["op"] == "decode":
        keys = sum(_seen(n, c["window"], c["sinks"]) for n in _lengths(c))
        by = keys * c["hkv"] * c["d"] * 2 * e + 2 * c["batch"] * c["hq"] * c["d"] * 2
        return {"bytes": by, "flops": 4 * keys * c["hq"] * c["d"]}
    new, w, s = _lengths(c), c["window"], c["sinks"]
    seen = sum(_seen(p + 1, w, s) for n in new for p in range(c["prefix"], c["prefix"] + n))
    # of each sequence, the keys that any of its new tokens sees
    keys = sum(min(c["prefix"] + n, n + w - 1 + s) if w else c["prefix"] + n for n in new)
    by = keys * c["hkv"] * c["d"] * 2 * e + 2 * sum(new) * c["hq"] * c["d"] * 2
    return {"bytes": by, "flops": 4 * seen * c["hq"] * c["d"]}


# --------------------------------------------------------------------- inputs
def _cache(c, pages, gen):
    """Keys and values as the cache holds them: [pages, kv heads, page, d], and
    the scale of each kv head for e4m3 codes."""
    shape = (pages, c["page"], c["hkv"], c["d"]) if c["order"] == "token" else (pages, c["hkv"], c["page"], c["d"])
    out = {}
    for name in ("k", "v"):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        if c["cache"] == "e4m3":  # values around 30 of the largest code 448: scale = 1 / 32
            x = (x.mul_(32).clamp_(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
            out[name + "_scale"] = torch.rand(c["hkv"], device="cuda", generator=gen) * 0.02 + 0.02
        out[name] = x.transpose(1, 2) if c["order"] == "token" else x
    return out


def _tables(c, lengths, gen):
    """Each sequence's pages, anywhere in the cache, and how many pages that takes."""
    wide = max(1, max(-(-n // c["page"]) for n in lengths))
    pages = len(lengths) * wide
    return torch.randperm(pages, device="cuda", generator=gen).to(torch.int32).view(len(lengths), wide), pages


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "rope":
        n = c["tokens"]
        pages = -(-n // c["page"]) + 1
        s.update(_cache(c, pages, gen))
        s["qkv"] = torch.empty((n, (c["hq"] + 2 * c["hkv"]) * c["d"]), dtype=torch.bfloat16, device="cuda")
        s["qkv"].normal_(generator=gen).mul_(1.5)
        s["positions"] = torch.randint(0, 8192, (n,), device="cuda", generator=gen, dtype=torch.int32)
        s["slots"] = torch.randperm(pages * c["page"], device="cuda", generator=gen)[:n].contiguous()
        angle = torch.outer(torch.arange(8192, dtype=torch.float64),
                            500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / max(1, c["rot"])))
        s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).float().cuda()
        for name in ("q_weight", "k_weight"):
            w = 1 + 0.2 * torch.randn(c["d"], device="cuda", generator=gen)
            s[name] = w.to(torch.bfloat16) if c["norm"] else None
        s["q"] = torch.empty((n, c["hq"], c["d"]), dtype=torch.bfloat16, device="cuda")
    else:
        new = _lengths(c)
        total = [n + c.get("prefix", 0) for n in new]
        s["page_table"], pages = _tables(c, total, gen)
        s.update(_cache(c, pages, gen))
        s["seq_lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
        rows = c["batch"] if c["op"] == "decode" else sum(new)
        # scores of a few units: some keys matter far more than others
        s["q"] = torch.empty((rows, c["hq"], c["d"]), dtype=torch.bfloat16, device="cuda")
        s["q"].normal_(generator=gen).mul_(2)
        s["out"] = torch.empty_like(s["q"])
        s["most"] = max(total)
        if c["op"] == "prompt":
            cu = [0]
            for n in new:
                cu.append(cu[-1] + n)
            s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            s["most_q"] = max(new)
    if own:  # the handle and the scratch that a serving program keeps
        import semi_structured_sparse_gb300 as sp24
        s["cache"] = sp24.KVCache(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
        if c["op"] == "decode":
            need = sp24.attention_decode_workspace_size(s["cache"], c["hq"])
            s["workspace"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------------------- runs
def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import semi_structured_sparse_gb300 as sp24
        c = s["case"]
        if op == "rope":
            sp24.qk_norm_rope(s["qkv"], c["hq"], s["cache"], s["positions"], s["slots"], s["cos_sin"],
                              s["q_weight"], s["k_weight"], interleaved=c["pairs"] == "even", out=s["q"])
            return {"q": s["q"], "k": _values(s["k"]), "v": _values(s["v"])}
        if op == "decode":
            return sp24.attention_decode(s["q"], s["cache"], s["page_table"], s["seq_lens"], window=c["window"],
                                         sinks=c["sinks"], out=s["out"], workspace=s["workspace"])
        return sp24.attention_prompt(s["q"], s["cu_q"], s["cache"], s["page_table"], s["seq_lens"],
                                     window=c["window"], sinks=c["sinks"], out=s["out"])
    return {"rope": _plain_rope, "decode": _plain_decode, "prompt": _plain_prompt}[op](s)


def _values(x):
    """Codes as the values that they stand for (the same bytes)."""
    return x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x


def _plain_head(x, weight, cos, sin, interleaved, eps=1e-6):
    """x [tokens, heads, d] in 32 bits: normed per head, then rotated."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()
    rot = 2 * cos.shape[-1]
    turn, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
    else:
        a, b = turn[..., :rot // 2], turn[..., rot // 2:]
    a, b = a * cos - b * sin, b * cos + a * sin
    turn = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turn, rest), -1)


def _plain_store(cache, scale, x, slots):
    """x [tokens, kv heads, d] in 32 bits into its slots."""
    if scale is not None:
        x = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    page = cache.shape[2]
    cache[slots // page, :, slots % page] = x.to(cache.dtype)


def _plain_rope(s):
    c = s["case"]
    x = s["qkv"].view(c["tokens"], -1, c["d"]).float()
    q, k, v = x.split((c["hq"], c["hkv"], c["hkv"]), 1)
    turn = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = turn.chunk(2, -1)
    q = _plain_head(q, s["q_weight"], cos, sin, c["pairs"] == "even")
    k = _plain_head(k, s["k_weight"], cos, sin, c["pairs"] == "even")
    _plain_store(s["k"], s.get("k_scale"), k, s["slots"])
    _plain_store(s["v"], s.get("v_scale"), v, s["slots"])
    return {"q": q.to(torch.bfloat16), "k": _values(s["k"]), "v": _values(s["v"])}


def _plain_gather(cache, scale, table, most):
    """[sequences, kv heads, most, d] in 32 bits."""
    x = cache[table.long()].transpose(1, 2).flatten(2, 3)[:, :, :most]
    return x.float() if scale is None else x.view(torch.float8_e4m3fn).float() * scale[:, None, None]


def _plain_mask(at, length, keys, window, sinks):
    """Whether the query at position `at` [...] sees each key, for `length` keys in the cache."""
    j = torch.arange(keys, device="cuda")
    see = (j <= at[..., None]) & (j < length[..., None])
    return see & ((j > at[..., None] - window) | (j < sinks)) if window else see


def _plain_attend(q, k, v, see):
    """q [b, hkv, rows, d], k and v [b, hkv, keys, d], see [b, 1, rows, keys]; rows that see nothing give zero."""
    score = (q @ k.transpose(-1, -2) * (1 / math.sqrt(q.shape[-1]))).masked_fill_(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.masked_fill(top == -math.inf, 0)).exp_()
    total = p.sum(-1, keepdim=True)
    return p @ v / total.masked_fill(total == 0, 1)


def _plain_decode(s):
    c = s["case"]
    k = _plain_gather(s["k"], s.get("k_scale"), s["page_table"], s["most"])
    v = _plain_gather(s["v"], s.get("v_scale"), s["page_table"], s["most"])
    n = s["seq_lens"].long()
    see = _plain_mask(n - 1, n, s["most"], c["window"], c["sinks"])[:, None, None]
    q = s["q"].float().view(c["batch"], c["hkv"], -1, c["d"])
    return _plain_attend(q, k, v, see).reshape(s["q"].shape).to(torch.bfloat16)


def _plain_prompt(s):
    c, q, cu = s["case"], s["q"], s["cu_q"].long()
    most_q, group = s["most_q"], c["hq"] // c["hkv"]
    k = _plain_gather(s["k"], s.get("k_scale"), s["page_table"], s["most"])
    v = _plain_gather(s["v"], s.get("v_scale"), s["page_table"], s["most"])
    n, new = s["seq_lens"].long(), cu[1:] - cu[:-1]
    row = torch.arange(most_q, device="cuda")
    padded = q[(cu[:-1, None] + row).clamp(max=q.shape[0] - 1)].float()  # [b, most_q, hq, d]
    padded = padded.view(c["batch"], most_q, c["hkv"], group, c["d"]).permute(0, 2, 3, 1, 4).flatten(2, 3)
    at = (n - new)[:, None] + row
    see = _plain_mask(at, n[:, None].expand_as(at), s["most"], c["window"], c["sinks"])
    see = see[:, None, None].expand(-1, 1, group, -1, -1).flatten(2, 3)
    y = _plain_attend(padded, k, v, see).view(c["batch"], c["hkv"], group, most_q, c["d"])
    y = y.permute(0, 3, 1, 2, 4).reshape(c["batch"], most_q, c["hq"], c["d"])
    t = torch.arange(q.shape[0], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    return y[b, t - cu[b]].to(torch.bfloat16)


# ---------------------------------------------------------------------- exact
def exact(case, seed):
    """The outputs in 64 bits, one head of one sequence at a time."""
    s = prepare(case, seed)
    c = s["case"]
    wide = {}
    for name in ("k", "v"):
        x = _values(s[name])
        wide[name] = x.double() if x.dtype == torch.float8_e4m3fn and c["op"] == "rope" else x
    if c["op"] == "rope":
        out = {"q": torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), "k": wide["k"].double(),
               "v": wide["v"].double()}
        half = c["rot"] // 2
        pos = s["positions"].long()
        cos, sin = s["cos_sin"][pos, :half].double(), s["cos_sin"][pos, half:].double()
        first = torch.arange(half, device="cuda") * (2 if c["pairs"] == "even" else 1)
        second = first + (1 if c["pairs"] == "even" else half)
        for h in range(c["hq"] + 2 * c["hkv"]):
            x = s["qkv"][:, h * c["d"]:(h + 1) * c["d"]].double()
            kind = "q" if h < c["hq"] else "k" if h < c["hq"] + c["hkv"] else "v"
            if kind != "v":
                w = s[kind + "_weight"]
                if w is not None:
                    x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt() * w.double()
                y = x.clone()
                y[:, first] = x[:, first] * cos - x[:, second] * sin
                y[:, second] = x[:, first] * sin + x[:, second] * cos
                x = y
            if kind == "q":
                out["q"][:, h] = x
            else:
                g = (h - c["hq"]) % c["hkv"]
                if kind + "_scale" in s:
                    x = (x / s[kind + "_scale"][g].double()).clamp(-448, 448)
                out[kind][s["slots"] // c["page"], g, s["slots"] % c["page"]] = x
        return out
    new = [1] * c["batch"] if c["op"] == "decode" else _lengths(c)
    total, group = s["seq_lens"].tolist(), c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for b in range(c["batch"]):
        n, m = total[b], new[b]
        pages = s["page_table"][b, :-(-n // c["page"])].long()
        j = torch.arange(n, device="cuda")
        at = torch.arange(n - m, n, device="cuda")
        hide = j[None] > at[:, None]
        if c["window"]:
            hide |= (j[None] <= at[:, None] - c["window"]) & (j[None] >= c["sinks"])
        for g in range(c["hkv"]):
            k, v = ((_values(s[x])[:, g].view(torch.uint8) if c["cache"] == "e4m3" else s[x][:, g])[pages]
                    for x in ("k", "v"))
            if c["cache"] == "e4m3":
                k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
            k, v = (x.reshape(-1, c["d"])[:n].double() for x in (k, v))
            if c["cache"] == "e4m3":
                k, v = k * s["k_scale"][g].double(), v * s["v_scale"][g].double()
            for h in range(g * group, (g + 1) * group):
                x = s["q"][start:start + m, h].double() @ k.T / math.sqrt(c["d"])
                out[start:start + m, h] = torch.softmax(x.masked_fill_(hide, -math.inf), -1) @ v
        start += m
    return out
