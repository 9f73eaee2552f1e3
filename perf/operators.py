"""The per-token / per-channel int8 operators, as they are measured: their cases, their plain forms in elementary
torch operations, and the calls a user makes of them.

  quantize   rows of activations (or a weight's channels) -> int8 codes with one scale per row
  silu_mul   silu(gate) * up, quantized per row: what stands between an FFN's two products
  gemm       int8 x int8 with a scale per token and per output channel, with or without a bias
  grouped    the same product grouped by expert, ragged groups, rows gathered from the tokens

Shapes are those of the 7B projections (hidden 3584, kv 512, FFN 18944) and of the 128-expert MoE layer (hidden 2048,
expert FFN 768, 8 experts per token) that this repository is measured on elsewhere, and generic ones between.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def pad16(k):
    return -(-k // 16) * 16


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decoded token's hidden state, before the q/k/v products: the smallest call
        {"name": "quantize_token", "op": "quantize", "M": 1, "K": 3584, "type": "bf16"},
        # the widest activations of a 2K-token prefill (the input of the down projection)
        {"name": "quantize_prefill_ffn", "op": "quantize", "M": 2048, "K": 18944, "type": "bf16"},
        # one token's eight expert hidden rows, between the two expert products
        {"name": "silu_mul_token_experts", "op": "silu_mul", "M": 8, "K": 768, "type": "f16"},
        # the dense FFN of a 2K-token prefill, gate and up side by side in one matrix
        {"name": "silu_mul_prefill_ffn", "op": "silu_mul", "M": 2048, "K": 18944, "type": "bf16"},
        # one decoded token through a square projection: the weights are the traffic
        {"name": "gemm_token_o", "op": "gemm", "M": 1, "N": 3584, "K": 3584, "type": "bf16", "bias": False},
        # thirteen sequences decoded together through the up projection, fp32 out
        {"name": "gemm_batch13_up", "op": "gemm", "M": 13, "N": 18944, "K": 3584, "type": "f32", "bias": False},
        # a ragged chunk of 509 prompt tokens through q, k and v in one matrix, with the projections' bias
        {"name": "gemm_chunk509_qkv", "op": "gemm", "M": 509, "N": 4608, "K": 3584, "type": "f16", "bias": True},
        # a 2K-token prefill through the long-K down projection
        {"name": "gemm_prefill_down", "op": "gemm", "M": 2048, "N": 3584, "K": 18944, "type": "bf16", "bias": False},
        # the largest call: 8K tokens through the gate projection
        {"name": "gemm_prefill8k_gate", "op": "gemm", "M": 8192, "N": 18944, "K": 3584, "type": "bf16", "bias": False},
        # one decoded token at its eight experts' fused gate and up
        {"name": "grouped_token_gate_up", "op": "grouped", "T": 1, "topk": 8, "E": 128, "N": 1536, "K": 2048,
         "gather": True, "skew": 0.0, "type": "bf16"},
        # a 2K-token prefill's fused gate and up: each token's row is read by its eight experts
        {"name": "grouped_prefill_gate_up", "op": "grouped", "T": 2048, "topk": 8, "E": 128, "N": 1536, "K": 2048,
         "gather": True, "skew": 0.0, "type": "bf16"},
        # the down product of a 1501-token chunk whose routing is skewed: groups from a few rows to thousands
        {"name": "grouped_chunk1501_down", "op": "grouped", "T": 1501, "topk": 8, "E": 128, "N": 2048, "K": 768,
         "gather": False, "skew": 1.0, "type": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "silu_mul", "gemm", "gemm", "grouped", "grouped"])
    while True:
        if op in ("quantize", "silu_mul"):
            c = {"op": op, "M": _log(rng, 1, 8192), "K": _log(rng, 32, 18944), "type": rng.choice(["f32", "bf16", "f16"])}
            ok = c["M"] * c["K"] * SIZE[c["type"]] <= 2048 * 18944 * 2
        elif op == "gemm":
            c = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 18944), "K": pad16(_log(rng, 128, 18944)),
                 "type": rng.choice(["f32", "bf16", "f16"]), "bias": rng.random() < 0.3}
            ok = c["M"] * c["N"] * c["K"] <= 2048 * 18944 * 3584
        else:
            c = {"op": op, "T": _log(rng, 1, 4096), "topk": rng.choice([1, 2, 4, 6, 8]), "E": _log(rng, 8, 128),
                 "N": _log(rng, 256, 4096), "K": pad16(_log(rng, 256, 4096)), "gather": rng.random() < 0.5,
                 "skew": round(rng.uniform(0.0, 1.2), 2), "type": rng.choice(["f32", "bf16", "f16"])}
            ok = (c["E"] * c["N"] * c["K"] <= 128 * 1536 * 2048
                  and c["T"] * c["topk"] * c["N"] * c["K"] <= 16384 * 1536 * 2048)
        if ok:
            return c


# ---------------------------------------------------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _activations(g, M, K):
    """Normal activations whose channels differ in size, with a few large ones, as hidden states have."""
    x = torch.randn((M, K), generator=g, device=DEV)
    x *= torch.exp(0.4 * torch.randn((K,), generator=g, device=DEV))
    return x * torch.where(torch.rand((K,), generator=g, device=DEV) < 0.002, 8.0, 1.0)


def _codes(x):
    """int8 codes and fp32 scale of each row."""
    s = x.abs().amax(-1) / 127.0
    return torch.round(x / s[..., None]).clamp_(-127, 127).to(torch.int8), s


def _padded(x):
    k = x.shape[-1]
    return x if k % 16 == 0 else torch.nn.functional.pad(x, (0, pad16(k) - k))


def _routing(g, case):
    """Each token's topk distinct experts, and the routed rows sorted by expert."""
    T, E, topk = case["T"], case["E"], min(case["topk"], case["E"])
    weight = -case["skew"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device=DEV).clamp_(1e-20, 1 - 1e-7)))
    ids = (weight + noise).topk(topk, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return (order // topk).to(torch.int32), offsets, int(counts.max())


def prepare(case, seed):
    g = _gen(seed)
    op, t = case["op"], TYPES[case["type"]]
    st = {"op": op, "type": t}
    if op == "quantize":
        st["x"] = _activations(g, case["M"], case["K"]).to(t)
    elif op == "silu_mul":
        gu = torch.randn((case["M"], 2 * case["K"]), generator=g, device=DEV).to(t)
        st["gate"], st["up"] = gu[:, :case["K"]], gu[:, case["K"]:]
    elif op == "gemm":
        st["xq"], st["xs"] = _codes(_activations(g, case["M"], case["K"]))
        st["wq"], st["ws"] = _codes(0.02 * torch.randn((case["N"], case["K"]), generator=g, device=DEV))
        st["bias"] = torch.randn((case["N"],), generator=g, device=DEV) if case["bias"] else None
    else:
        E, N, K = case["E"], case["N"], case["K"]
        rows, st["offsets"], st["most"] = _routing(g, case)
        st["rows"] = rows if case["gather"] else None
        M = case["T"] if case["gather"] else rows.numel()
        st["xq"], st["xs"] = _codes(_activations(g, M, K))
        st["wq"], st["ws"] = _codes(0.02 * torch.randn((E, N, K), generator=g, device=DEV))
    return st


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------
def _values(q, s, dtype):
    """The values that codes and scales stand for."""
    out = torch.empty(q.shape, dtype=dtype, device=q.device)
    return torch.mul(q, s[:, None], out=out)


def _quantize_plain(x):
    """d = amax / 127, code = x * (1 / d) rounded half away from zero; columns padded with zeros to 16."""
    d = x.abs().amax(1)
    d = d / torch.full_like(d, 127.0)          # a tensor: by a number, torch multiplies with its reciprocal
    inv = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    inv = torch.where(torch.isinf(inv), torch.zeros_like(inv), inv)
    v = x * inv[:, None]
    t = torch.trunc(v)
    q = (t + torch.sign(v) * ((v - t).abs() >= 0.5)).clamp(-127, 127)
    return _padded(q).to(torch.int8), d


def _silu_mul_plain(gate, up):
    g = gate.float()
    return g / (1.0 + torch.exp(-g)) * up.float()


def _gemm_plain(st):
    acc = torch.matmul(st["xq"].float(), st["wq"].float().t())     # integers: exact as long as they stay below 2^24
    out = acc * st["xs"][:, None] * st["ws"][None, :]
    if st["bias"] is not None:
        out = out + st["bias"][None, :]
    return out.to(st["type"])


def _slots(st):
    """The expert of every routed row, and the row's place within its group."""
    off = st["offsets"].long()
    R = st["rows"].numel() if st["rows"] is not None else st["xq"].shape[0]
    r = torch.arange(R, device=DEV)
    e = torch.searchsorted(off[1:].contiguous(), r, right=True)
    return e, r - off[e]


def _grouped_plain(st):
    """Groups padded to the largest and multiplied as a batch."""
    E, N, K = st["wq"].shape
    e, place = _slots(st)
    src = st["rows"].long() if st["rows"] is not None else torch.arange(e.numel(), device=DEV)
    x = torch.zeros((E, st["most"], K), device=DEV)
    x[e, place] = st["xq"][src].float()
    acc = torch.bmm(st["wq"].float(), x.transpose(1, 2).contiguous())                  # [E, N, most]
    out = acc.transpose(1, 2)[e, place] * st["xs"][src][:, None] * st["ws"][e]
    return out.to(st["type"])


def run(st):
    op = st["op"]
    if own:
        import block_quantized_int8_q8_amd as mmq
        if op == "quantize":
            q, s = mmq.quantize_i8(st["x"])
            return _values(q, s, torch.float32), s
        if op == "silu_mul":
            q, s = mmq.silu_mul_quantize_i8(st["gate"], st["up"])
            return _values(q, s, torch.bfloat16), s
        if op == "gemm":
            return mmq.gemm_i8(st["xq"], st["xs"], st["wq"], st["ws"], bias=st["bias"], dtype=st["type"])
        return mmq.grouped_gemm_i8(st["xq"], st["xs"], st["wq"], st["ws"], st["offsets"], rows=st["rows"],
                                   dtype=st["type"])
    if op == "quantize":
        q, s = _quantize_plain(st["x"].float())
        return _values(q, s, torch.float32), s
    if op == "silu_mul":
        q, s = _quantize_plain(_silu_mul_plain(st["gate"], st["up"]))
        # codes next to a border move by a step with the last bit of exp: 16-bit values, which a step does not hide in
        return _values(q, s, torch.bfloat16), s
    if op == "gemm":
        return _gemm_plain(st)
    return _grouped_plain(st)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without, and what it comes to in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def work(case):
    op, b = case["op"], SIZE[case["type"]]
    if op == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": n * b + case["M"] * pad16(case["K"]) + 4 * case["M"], "flops": 4 * n}
    if op == "silu_mul":
        n = case["M"] * case["K"]
        return {"bytes": 2 * n * b + case["M"] * pad16(case["K"]) + 4 * case["M"], "flops": 9 * n}
    N, K = case["N"], case["K"]
    if op == "gemm":
        M = case["M"]
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * b + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    E, topk = case["E"], min(case["topk"], case["E"])
    R = case["T"] * topk
    M = case["T"] if case["gather"] else R
    used = min(E, R)            # at most so many experts have rows
    return {"bytes": M * K + 4 * M + used * (N * K + 4 * N) + R * N * b + 4 * (E + 1) + (4 * R if case["gather"] else 0),
            "flops": 2 * R * N * K}


def _exact_codes(v, width):
    """The codes and scales of rows given in 64 bits. The scale, its reciprocal and the scaled value are fp32 numbers by
    the operator's definition; each is formed here in 64 bits and rounded to fp32 once."""
    d = (v.abs().amax(1) / 127).float().double()
    inv = (1 / d).float().double()
    y = (v * inv[:, None]).float().double()
    q = torch.where(y < 0, torch.ceil(y - 0.5), torch.floor(y + 0.5)).clamp(-127, 127)
    q = torch.nn.functional.pad(q, (0, width - q.shape[1]))
    return q * d[:, None], d


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_codes(st["x"].double(), pad16(case["K"]))
    if case["op"] == "silu_mul":
        g, u = st["gate"].double(), st["up"].double()
        return _exact_codes(g * torch.sigmoid(g) * u, pad16(case["K"]))
    if case["op"] == "gemm":
        y = torch.matmul(st["xq"].double() * st["xs"].double()[:, None], (st["wq"].double() * st["ws"].double()[:, None]).t())
        return y if st["bias"] is None else y + st["bias"].double()
    off = st["offsets"].tolist()
    x = st["xq"].double() * st["xs"].double()[:, None]
    if st["rows"] is not None:
        x = x[st["rows"].long()]
    parts = [torch.matmul(x[a:b], (st["wq"][e].double() * st["ws"][e].double()[:, None]).t())
             for e, (a, b) in enumerate(zip(off, off[1:])) if b > a]
    return torch.cat(parts)
