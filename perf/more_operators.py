"""The operators between a layer's q/k/v product and its output product, as they are measured: their cases, their plain
forms in elementary torch operations, and the calls a user makes of them.

  rope        rotary positions: pairs in halves or side by side, part of the head, frequencies scaled for long contexts
  write       new keys (rotated) and values quantized into a paged int8 cache, then read back by their slots
  read        a stored prefix read back from the cache as values
  attention   a chunk of new tokens (one, or many) of each sequence over its pages of the cache, causal

Shapes are those of the 7B layer (28 query heads on 4 key/value heads of 128) and of the 128-expert MoE layer's attention
(32 on 4 of 128) that this repository is measured on elsewhere, and generic ones beside them (heads of 64 and 256, other groups).
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BASE = 1000000.0          # base of the rotary frequencies
ORIGINAL = 32768          # positions that the unscaled frequencies cover


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decoded token: its query heads, before attention (the smallest call)
        {"name": "rope_token", "op": "rope", "T": 1, "H": 28, "D": 128, "rot": 128, "layout": "half", "scaling": "none",
         "far": 32768, "type": "bf16", "out": "bf16"},
        # the query heads of an 8K-token prefill chunk far into a scaled context
        {"name": "rope_prefill8k", "op": "rope", "T": 8192, "H": 28, "D": 128, "rot": 128, "layout": "half",
         "scaling": "yarn", "far": 1000000, "type": "bf16", "out": "bf16"},
        # one new token from each of 64 sequences; a quarter of the head rotated, pairs side by side
        {"name": "write_batch64", "op": "write", "T": 64, "H": 4, "D": 128, "rot": 32, "layout": "interleaved",
         "scaling": "none", "far": 32768, "page": 16, "type": "f16"},
        # the keys and values of an 8K-token prefill
        {"name": "write_prefill8k", "op": "write", "T": 8192, "H": 4, "D": 128, "rot": 128, "layout": "half",
         "scaling": "bands", "far": 131072, "page": 64, "type": "bf16"},
        # a few pages of wide heads read back, odd count
        {"name": "read_201", "op": "read", "T": 201, "H": 8, "D": 256, "page": 32, "type": "bf16"},
        # a stored 32K prefix read back as values
        {"name": "read_prefix32k", "op": "read", "T": 32768, "H": 4, "D": 128, "page": 64, "type": "f16"},
        # one sequence decoding at a short context: latency
        {"name": "attention_token", "op": "attention", "seqs": 1, "new": 1, "context": 2011, "Hq": 28, "Hkv": 4, "D": 128,
         "page": 16, "window": 0, "ragged": False, "type": "bf16"},
        # 64 sequences of different lengths decoded together
        {"name": "attention_batch64", "op": "attention", "seqs": 64, "new": 1, "context": 16384, "Hq": 28, "Hkv": 4,
         "D": 128, "page": 64, "window": 0, "ragged": True, "type": "bf16"},
        # one sequence decoding deep into a long context: the cache is the traffic, and one row of queries per head
        {"name": "attention_token_256k", "op": "attention", "seqs": 1, "new": 1, "context": 262144, "Hq": 32, "Hkv": 4,
         "D": 128, "page": 128, "window": 0, "ragged": False, "type": "f16"},
        # a ragged chunk of prompt after a stored prefix
        {"name": "attention_chunk509", "op": "attention", "seqs": 1, "new": 509, "context": 8192, "Hq": 32, "Hkv": 4,
         "D": 128, "page": 16, "window": 0, "ragged": False, "type": "bf16"},
        # a serving step: decoding sequences and prompt chunks of all lengths in one batch, heads of 64, a sliding window
        {"name": "attention_mixed24", "op": "attention", "seqs": 24, "new": 700, "context": 6000, "Hq": 32, "Hkv": 8,
         "D": 64, "page": 32, "window": 4096, "ragged": True, "type": "f16"},
        # the largest: an 8K prompt from its first token
        {"name": "attention_prefill8k", "op": "attention", "seqs": 1, "new": 8192, "context": 8192, "Hq": 28, "Hkv": 4,
         "D": 128, "page": 64, "window": 0, "ragged": False, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attention", "attention", "attention"])
    while True:
        D = rng.choice([64, 128, 128, 256])
        if op == "rope":
            c = {"op": op, "T": _log(rng, 1, 8192), "H": rng.choice([1, 4, 8, 14, 28, 32, 40]), "D": D,
                 "rot": rng.choice([D, D, D // 2, D // 4]), "layout": rng.choice(["half", "interleaved"]),
                 "scaling": rng.choice(["none", "linear", "bands", "yarn"]), "far": _log(rng, 1000, 1000000),
                 "type": rng.choice(["f32", "bf16", "f16"])}
            c["out"] = rng.choice([c["type"], c["type"], "bf16"])
            ok = c["T"] * c["H"] * D * (SIZE[c["type"]] + SIZE[c["out"]]) <= 8192 * 28 * 128 * 4
        elif op == "write":
            c = {"op": op, "T": _log(rng, 1, 8192), "H": rng.choice([1, 2, 4, 8]), "D": D,
                 "rot": rng.choice([D, D, D // 2, D // 4]), "layout": rng.choice(["half", "interleaved"]),
                 "scaling": rng.choice(["none", "linear", "bands", "yarn"]), "far": _log(rng, 1000, 1000000),
                 "page": rng.choice([16, 32, 64, 128]), "type": rng.choice(["bf16", "f16"])}
            ok = c["T"] * c["H"] * D <= 8192 * 4 * 128
        elif op == "read":
            c = {"op": op, "T": _log(rng, 1, 32768), "H": rng.choice([1, 2, 4, 8]), "D": D,
                 "page": rng.choice([16, 32, 64, 128]), "type": rng.choice(["f32", "bf16", "f16"])}
            ok = c["T"] * c["H"] * D <= 32768 * 4 * 128
        else:
            Hkv = rng.choice([1, 2, 4, 8])
            new = 1 if rng.random() < 0.4 else _log(rng, 2, 8192)
            c = {"op": op, "seqs": _log(rng, 1, 64), "new": new, "context": max(new, _log(rng, 16, 262144)),
                 "Hq": Hkv * rng.choice([1, 2, 4, 7, 8]), "Hkv": Hkv, "D": D, "page": rng.choice([16, 32, 64, 128]),
                 "window": rng.choice([0, 0, 0, _log(rng, 16, 8192)]), "ragged": rng.random() < 0.5,
                 "type": rng.choice(["bf16", "f16"])}
            ok = (c["seqs"] * c["context"] * Hkv * D <= 262144 * 4 * 128 * 2
                  and c["seqs"] * new * c["context"] * c["Hq"] * D <= 8192 * 8192 * 28 * 128)
        if ok:
            return c


def _lengths(case):
    """New tokens and total length of each sequence, from the case alone. Ragged batches hold decoding sequences (one new
    token) beside chunks of any length, and contexts from an eighth of the longest up."""
    if not case["ragged"]:
        return [case["new"]] * case["seqs"], [case["context"]] * case["seqs"]
    rng = random.Random(f"{case['seqs']} {case['new']} {case['context']} {case['Hq']} {case['page']}")
    new = [1 if rng.random() < 0.5 else rng.randint(1, case["new"]) for _ in range(case["seqs"])]
    return new, [max(n, rng.randint(max(1, case["context"] // 8), case["context"])) for n in new]


# ---------------------------------------------------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _heads(g, T, H, D, t):
    """Normal heads whose channels differ in size, with a few large ones, as keys and queries have."""
    x = torch.randn((T, H, D), generator=g, device=DEV)
    size = torch.exp(0.4 * torch.randn((H, D), generator=g, device=DEV))
    return (x * size * torch.where(torch.rand((H, D), generator=g, device=DEV) < 0.01, 4.0, 1.0)).to(t)


def frequencies(rot, scaling):
    """Angle per position of each pair, in 64 bits on the host, and the factor on the rotated values.
    linear: positions 8 times closer. bands: long waves 8 times slower, short ones as they were, a ramp between.
    yarn: the same idea with the ramp over whole turns within the original length, and a factor on the values."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = BASE ** (-2.0 * i / rot)
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return f / 8.0, 1.0
    turns = ORIGINAL * f / (2 * math.pi)
    if scaling == "bands":
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return f / 8.0 * (1 - keep) + f * keep, 1.0

    def pair(n):                      # the pair that makes n turns within the original length
        return rot * math.log(ORIGINAL / (n * 2 * math.pi)) / (2 * math.log(BASE))
    lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
    keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return f / 8.0 * (1 - keep) + f * keep, 0.1 * math.log(8.0) + 1.0


def _positions(g, T, far):
    """A run of consecutive positions that ends before `far`."""
    start = int(torch.randint(0, max(far - T, 1), (1,), generator=g, device=DEV))
    return torch.arange(start, start + T, dtype=torch.int32, device=DEV)


def _slots(g, T, page):
    """Slots of T tokens in order, on pages in no order; about one page in eight belongs to others."""
    need = -(-T // page)
    pages = torch.randperm(need + need // 8 + 1, generator=g, device=DEV)[:need]
    t = torch.arange(T, device=DEV)
    return (pages[t // page] * page + t % page).to(torch.int32), need + need // 8 + 1


def _filled(st, k, v, slots, n_pages, page):
    """The cache with k and v written into it."""
    T, H, D = k.shape
    if own:
        import block_quantized_int8_q8_amd as mmq
        st["cache"] = mmq.kv_cache(n_pages, page, H, D, device=DEV)
        if T:
            mmq.kv_write(k, v, st["cache"], slots)
    else:
        st["cache"] = _plain_cache(n_pages * page, H, D)
        _store(st["cache"], slots, k.float(), v.float())


def prepare(case, seed):
    g = _gen(seed)
    op, t = case["op"], TYPES[case["type"]]
    st = {"op": op, "type": t}
    if op in ("rope", "write"):
        st["layout"] = case["layout"]
        freqs, st["mscale"] = frequencies(case["rot"], case["scaling"])
        st["freqs"] = freqs.to(DEV)
        st["positions"] = _positions(g, case["T"], case["far"])
    if op == "rope":
        st["x"] = _heads(g, case["T"], case["H"], case["D"], t)
        st["out"] = TYPES[case["out"]]
    elif op == "write":
        # keys and values side by side, as the product that makes them leaves them
        kv = _heads(g, case["T"], 2 * case["H"], case["D"], t)
        st["k"], st["v"] = kv[:, :case["H"]], kv[:, case["H"]:]
        st["slots"], n_pages = _slots(g, case["T"], case["page"])
        _filled(st, st["k"][:0], st["v"][:0], st["slots"][:0], n_pages, case["page"])
    elif op == "read":
        k, v = (_heads(g, case["T"], case["H"], case["D"], t) for _ in range(2))
        st["slots"], n_pages = _slots(g, case["T"], case["page"])
        st["D"] = case["D"]
        _filled(st, k, v, st["slots"], n_pages, case["page"])
    else:
        H, D, page = case["Hkv"], case["D"], case["page"]
        new, lens = _lengths(case)
        total = sum(-(-n // page) * page for n in lens)          # every sequence begins a page of its own
        k, v = (_heads(g, total, H, D, t) for _ in range(2))
        slots, n_pages = _slots(g, total, page)
        _filled(st, k, v, slots, n_pages, page)
        table = torch.zeros((len(lens), max(-(-n // page) for n in lens)), dtype=torch.int32)
        at, first = 0, (slots[::page] // page).cpu()
        for b, n in enumerate(lens):
            p = -(-n // page)
            table[b, :p] = first[at:at + p]
            at += p
        st["table"] = table.to(DEV)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["offsets"] = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32).to(DEV)
        st["q"] = _heads(g, sum(new), case["Hq"], D, t)
        st["new"], st["host_lens"] = new, lens                   # the program that made the batch knows them too
        st["window"], st["page"], st["scale"] = case["window"], page, 1.0 / math.sqrt(D)
    return st


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------
def _rotate(x, positions, freqs, layout, mscale):
    """Angles, sines and products in 64 bits: positions near a million leave 32 bits no digits of the angle."""
    rot = 2 * freqs.numel()
    phi = positions.double()[:, None] * freqs
    cos, sin = (torch.cos(phi) * mscale)[:, None], (torch.sin(phi) * mscale)[:, None]
    y = x.double()
    if layout == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], -1)
    a, b = y[..., 0:rot:2], y[..., 1:rot:2]
    r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, y[..., rot:]], -1)


def _quantize(x):
    """d = amax / 127, code = x * (1 / d) rounded half away from zero, of each row of the last axis."""
    d = x.abs().amax(-1)
    d = d / torch.full_like(d, 127.0)          # a tensor: by a number, torch multiplies with its reciprocal
    inv = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    inv = torch.where(torch.isinf(inv), torch.zeros_like(inv), inv)
    v = x * inv[..., None]
    t = torch.trunc(v)
    return (t + torch.sign(v) * ((v - t).abs() >= 0.5)).clamp(-127, 127).to(torch.int8), d


def _plain_cache(slots, H, D):
    return {n: torch.zeros((slots, H, D) if n in "kv" else (slots, H), dtype=torch.int8 if n in "kv" else torch.float32,
                           device=DEV) for n in ("k", "ks", "v", "vs")}


def _store(cache, slots, k, v):
    at = slots.long()
    cache["k"][at], cache["ks"][at] = _quantize(k)
    cache["v"][at], cache["vs"][at] = _quantize(v)


def _load(cache, slots):
    at = slots.long()
    return (cache["k"][at].float() * cache["ks"][at][..., None], cache["v"][at].float() * cache["vs"][at][..., None])


def _attention_plain(st):
    q, out, i = st["q"], torch.empty_like(st["q"]), 0
    Hq = q.shape[1]
    for b, (n, length) in enumerate(zip(st["new"], st["host_lens"])):
        t = torch.arange(length, device=DEV)
        at = st["table"][b].long()[t // st["page"]] * st["page"] + t % st["page"]
        k, v = _load(st["cache"], at)                                        # [length, Hkv, D]
        pos = torch.arange(length - n, length, device=DEV)[:, None]
        hidden = t[None, :] > pos
        if st["window"]:
            hidden |= t[None, :] <= pos - st["window"]
        group = Hq // k.shape[1]
        for h in range(Hq):
            s = torch.matmul(q[i:i + n, h].float(), k[:, h // group].t()) * st["scale"]
            s.masked_fill_(hidden, float("-inf"))
            s = torch.exp(s - s.amax(1, keepdim=True))
            out[i:i + n, h] = torch.matmul(s, v[:, h // group]) / s.sum(1, keepdim=True)
        i += n
    return out


def run(st):
    op = st["op"]
    if own:
        import block_quantized_int8_q8_amd as mmq
        layout = {"half": mmq.ROPE_HALF, "interleaved": mmq.ROPE_INTERLEAVED}.get(st.get("layout"))
        if op == "rope":
            return mmq.rope(st["x"], st["positions"], st["freqs"], layout=layout, mscale=st["mscale"], dtype=st["out"])
        if op == "write":
            mmq.kv_write(st["k"], st["v"], st["cache"], st["slots"], positions=st["positions"], freqs=st["freqs"],
                         layout=layout, mscale=st["mscale"])
            return mmq.kv_read(st["cache"], st["slots"], st["k"].shape[2], dtype=st["type"])
        if op == "read":
            return mmq.kv_read(st["cache"], st["slots"], st["D"], dtype=st["type"])
        return mmq.attention_i8(st["q"], st["cache"], st["table"], st["lens"], st["offsets"], max_q=max(st["new"]),
                                scale=st["scale"], window=st["window"])
    if op == "rope":
        return _rotate(st["x"], st["positions"], st["freqs"], st["layout"], st["mscale"]).to(st["out"])
    if op == "write":
        _store(st["cache"], st["slots"], _rotate(st["k"], st["positions"], st["freqs"], st["layout"], st["mscale"]).float(),
               st["v"].float())
    if op in ("write", "read"):
        return tuple(x.to(st["type"]) for x in _load(st["cache"], st["slots"]))
    return _attention_plain(st)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without, and what it comes to in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def work(case):
    op, b = case["op"], SIZE[case["type"]]
    if op == "rope":
        n = case["T"] * case["H"] * case["D"]
        return {"bytes": n * (b + SIZE[case["out"]]) + 4 * case["T"] + 4 * case["rot"],
                "flops": 3 * case["T"] * case["H"] * case["rot"]}
    if op in ("write", "read"):
        rows = 2 * case["T"] * case["H"]                                     # of keys and of values
        values, stored = rows * case["D"] * b, rows * (case["D"] + 4)
        if op == "read":
            return {"bytes": values + stored + 4 * case["T"], "flops": rows * case["D"]}
        # the values in, the codes written, read again, and the values out
        return {"bytes": 2 * values + 2 * stored + 12 * case["T"] + 4 * case["rot"], "flops": 8 * rows * case["D"]}
    D, w = case["D"], case["window"]
    keys = pairs = 0
    new, lens = _lengths(case)
    for n, length in zip(new, lens):
        first = length - n                                                   # position of the first new token
        keys += length - (max(0, first - w + 1) if w else 0)
        pairs += sum(min(p + 1, w) if w else p + 1 for p in range(first, length))
    return {"bytes": 2 * sum(new) * case["Hq"] * D * b + keys * case["Hkv"] * 2 * (D + 4) + 4 * sum(-(-n // case["page"]) for n in lens),
            "flops": 4 * D * case["Hq"] * pairs}


def _exact_rows(x):
    """What the codes of rows stand for: scale, reciprocal and scaled value are fp32 numbers by the operator's definition;
    each is formed here in 64 bits and rounded to fp32 once."""
    x = x.float().double()
    d = (x.abs().amax(-1, keepdim=True) / 127).float().double()
    y = (x * (1 / d).float().double()).float().double()
    return torch.where(y < 0, torch.ceil(y - 0.5), torch.floor(y + 0.5)).clamp(-127, 127) * d


def _exact_rotation(st, x):
    """The rotation as a product of complex numbers."""
    rot = 2 * st["freqs"].numel()
    angle = st["positions"].double()[:, None, None] * st["freqs"]
    turn = torch.polar(torch.full_like(angle, st["mscale"]), angle)
    y = x.double().clone()
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if st["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    z = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rope":
        return _exact_rotation(st, st["x"])
    if case["op"] == "write":
        return _exact_rows(_exact_rotation(st, st["k"])), _exact_rows(st["v"])
    cache = st["cache"]
    K, V = (cache[n].double() * cache[n + "s"].double()[..., None] for n in "kv")
    if case["op"] == "read":
        at = st["slots"].long()
        return K[at], V[at]
    K, V = (x.view(-1, st["page"], *x.shape[1:]) for x in (K, V))
    parts, i = [], 0
    group = case["Hq"] // case["Hkv"]
    for b, (n, length) in enumerate(zip(st["new"], st["host_lens"])):
        pages = st["table"][b, :-(-length // st["page"])].long()
        k, v = (x[pages].flatten(0, 1)[:length].transpose(0, 1).contiguous() for x in (K, V))      # [Hkv, length, D]
        q = st["q"][i:i + n].double().transpose(0, 1)                                              # [Hq, n, D]
        seen = torch.ones((n, length), dtype=torch.bool, device=DEV).tril(length - n)
        if st["window"]:
            seen = seen.triu(length - n - st["window"] + 1)
        o = torch.empty((n, case["Hq"], case["D"]), dtype=torch.float64, device=DEV)
        for h in range(case["Hq"]):
            s = torch.where(seen, q[h] @ k[h // group].mT / math.sqrt(case["D"]), -math.inf)
            o[:, h] = torch.exp(s - torch.logsumexp(s, 1, keepdim=True)) @ v[h // group]
        parts.append(o)
        i += n
    return torch.cat(parts)
