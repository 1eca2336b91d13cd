"""Cases of the operators between a layer's fused q/k/v projection and its
output projection: the new tokens' heads normalised, rotated and quantized into
a paged INT8 key/value cache, the cache read back, and the attention of the new
tokens over it.

``own`` False computes each operator in elementary torch operations, True
calls the library (``w4a16_linear_layers_gb300.qlin``).
"""
import math

import torch

own = False

DEV = "cuda"
D = 128             # of a head, and of a quantization group
BLOCK = 16          # tokens of one block of the cache
BLOCK_BYTES = 4224  # K codes, V codes, K scales, V scales of a block


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token of one sequence enters the cache: latency counts
        {"name": "write_1x1", "op": "write", "B": 1, "T": 1, "Hq": 32, "Hkv": 8, "L": 2048, "page": 16, "R": 128,
         "axes": 1, "norm": True, "ragged": False},
        # twelve drafted blocks of eight
        {"name": "write_12x8", "op": "write", "B": 12, "T": 8, "Hq": 32, "Hkv": 8, "L": 8192, "page": 16, "R": 128,
         "axes": 1, "norm": True, "ragged": False},
        # three ragged prompts with images: positions of three axes, no norm
        {"name": "write_3x515_axes", "op": "write", "B": 3, "T": 515, "Hq": 28, "Hkv": 4, "L": 515, "page": 64, "R": 128,
         "axes": 3, "norm": False, "ragged": True},
        # a long prompt, half of each head rotated
        {"name": "write_1x8192", "op": "write", "B": 1, "T": 8192, "Hq": 32, "Hkv": 8, "L": 8192, "page": 16, "R": 64,
         "axes": 1, "norm": True, "ragged": False},
        # a short sequence's cache taken out
        {"name": "read_1x515", "op": "read", "B": 1, "L": 515, "Hkv": 8, "page": 16, "ragged": False},
        # the caches of twelve sequences for a pass over all their tokens
        {"name": "read_12x8192", "op": "read", "B": 12, "L": 8192, "Hkv": 8, "page": 64, "ragged": True},
        # one token after a short prompt: latency counts
        {"name": "attn_1x1_515", "op": "attn", "B": 1, "T": 1, "Hq": 32, "Hkv": 8, "L": 515, "page": 16, "causal": True,
         "window": 0, "softcap": 0.0, "ragged": False},
        # three tokens each of five short sequences, an odd number of heads, capped scores
        {"name": "attn_5x3_1000_cap", "op": "attn", "B": 5, "T": 3, "Hq": 30, "Hkv": 6, "L": 1000, "page": 48,
         "causal": True, "window": 0, "softcap": 30.0, "ragged": True},
        # twelve drafted blocks, whose tokens see each other and a window behind them
        {"name": "attn_12x8_w2048", "op": "attn", "B": 12, "T": 8, "Hq": 32, "Hkv": 8, "L": 8192, "page": 16,
         "causal": False, "window": 2048, "softcap": 0.0, "ragged": True},
        # twelve drafted blocks verified against the whole context
        {"name": "attn_12x8_8192", "op": "attn", "B": 12, "T": 8, "Hq": 32, "Hkv": 8, "L": 8192, "page": 16,
         "causal": True, "window": 0, "softcap": 0.0, "ragged": True},
        # a serving batch of ninety-six sequences
        {"name": "attn_96x1_4096", "op": "attn", "B": 96, "T": 1, "Hq": 32, "Hkv": 8, "L": 4096, "page": 16,
         "causal": True, "window": 0, "softcap": 0.0, "ragged": True},
        # one sequence with a very long context
        {"name": "attn_1x1_131072", "op": "attn", "B": 1, "T": 1, "Hq": 32, "Hkv": 8, "L": 131072, "page": 64,
         "causal": True, "window": 0, "softcap": 0.0, "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# no drawn case costs more than its operator's largest listed one
_MOST = {"write": 230_000_000, "read": 600_000_000, "attn": 830_000_000}


def _heads(rng):
    Hkv = rng.choice([1, 2, 4, 5, 8])
    return Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]), Hkv


def draw(rng):
    op = rng.choice(["write", "read", "attn"])
    Hq, Hkv = _heads(rng)
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "write":
        T = _log(rng, 1, 8192)
        c = {"op": op, "B": _log(rng, 1, 96), "T": T, "Hq": Hq, "Hkv": Hkv, "L": T + rng.choice([0, _log(rng, 1, 16384)]),
             "page": page, "R": rng.choice([0, 32, 64, 96, 128]), "axes": rng.choice([1, 1, 2, 3]),
             "norm": rng.random() < 0.6, "ragged": rng.random() < 0.5}
    elif op == "read":
        c = {"op": op, "B": _log(rng, 1, 96), "L": _log(rng, 1, 32768), "Hkv": Hkv, "page": page,
             "ragged": rng.random() < 0.5}
    else:
        T = rng.choice([1, 1, 2, 3, 5, 8, 8, 16])
        c = {"op": op, "B": _log(rng, 1, 128), "T": T, "Hq": Hq, "Hkv": Hkv, "L": T - 1 + _log(rng, 1, 131072), "page": page,
             "causal": rng.random() < 0.6, "window": rng.choice([0, 0, 1, 100, 2048]),
             "softcap": rng.choice([0.0, 0.0, 20.0, 50.0]), "ragged": rng.random() < 0.6}
    while work(c)["bytes"] > _MOST[op] or c["B"] * c["L"] * c["Hkv"] > 3_500_000:
        if c["B"] > 1:
            c["B"] = max(1, c["B"] * 3 // 4)
        else:
            if "T" in c and op == "write":
                c["T"] = max(1, c["T"] * 3 // 4)
            c["L"] = max(c.get("T", 1), c["L"] * 3 // 4)
    return c


def _lens(c):
    """Tokens of each sequence, the new ones included, as the program that made the batch knows them."""
    L, low = c["L"], c.get("T", 1)
    if not c["ragged"]:
        return [L] * c["B"]
    # from half of the longest up, in no order; the first has all
    return [max(low, L - (b * 7919 % c["B"]) * (L // 2) // c["B"]) for b in range(c["B"])]


def _news(c):
    """New tokens of each sequence: ragged prompts are their whole sequence, short ones of a batch all new."""
    T = c["T"]
    if c["op"] == "write" and c["ragged"] and T > 1:
        return [T - (b * 31 % 5) * T // 8 for b in range(c["B"])]
    return [T] * c["B"]


def _seen(c, b_len):
    """Tokens of a sequence that some new token sees."""
    w = c["window"]
    return b_len if w == 0 else min(b_len, c["T"] + w - 1)


def work(case):
    c = case
    if c["op"] == "write":
        rows = sum(_news(c))
        # q, k, v in, q out, codes and scales written and read back, k and v out
        return {"bytes": rows * ((c["Hq"] + 2 * c["Hkv"]) * 2 * D + c["Hq"] * 2 * D + c["Hkv"] * 2 * (2 * (D + 4) + 2 * D)),
                "flops": rows * (c["Hq"] + 2 * c["Hkv"]) * D * 10}
    if c["op"] == "read":
        n = sum(_lens(c)) * c["Hkv"] * 2
        return {"bytes": n * (D + 4) + c["B"] * c["L"] * c["Hkv"] * 2 * 2 * D, "flops": n * D}
    n = sum(_seen(c, n) for n in _lens(c))
    rows = c["B"] * c["T"] * c["Hq"]
    return {"bytes": n * c["Hkv"] * 2 * (D + 4) + rows * 4 * D, "flops": 4 * D * n * c["T"] * c["Hq"]}


# ------------------------------------------------------------------ inputs

def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _places():
    """Offset in a block of component d of token r: its 32-byte quarters are permuted by (r / 4) % 4."""
    r = torch.arange(BLOCK, device=DEV)[:, None]
    d = torch.arange(D, device=DEV)[None, :]
    return r * D + (((d >> 5) ^ ((r >> 2) & 3)) << 5) + (d & 31)


def _cache(c, lens, g, fill):
    """(cache, block table): pages in random order, a few of them unused; with
    fill, keys and values as normal vectors leave them, their sizes unequal."""
    per = [-(-n // c["page"]) for n in lens]
    most, pages = max(per), sum(per) + 3
    blocks = c["page"] // BLOCK
    cache = torch.full((pages, c["Hkv"], blocks, BLOCK_BYTES), 128, dtype=torch.uint8, device=DEV)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((c["B"], most), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    if fill:
        flat = cache.view(-1, BLOCK_BYTES)
        codes = 2 * BLOCK * D
        for i in range(0, flat.shape[0], 65536):
            part = flat[i:i + 65536]
            n = part.shape[0]
            x = torch.randn((n, codes), generator=g, device=DEV).mul_(45.0).round_().clamp_(-127, 127)
            part[:, :codes] = x.add_(128.0).to(torch.uint8)
            s = torch.exp(0.4 * torch.randn((n, 2 * BLOCK), generator=g, device=DEV)) / 45.0
            part[:, codes:] = s.view(torch.uint8)
    return cache, table


def _table(P, R):
    """cos and sin of position times frequency, from 64-bit angles."""
    freq = 1e6 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)
    angle = torch.arange(P, dtype=torch.float64, device=DEV)[:, None] * freq[None, :]
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    c = dict(case)
    lens = _lens(c)
    g = _gen(seed, {"write": 1, "read": 2, "attn": 3}[c["op"]])
    s = {"case": c, "lens": lens, "total": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    s["cache"], s["table"] = _cache(c, lens, g, c["op"] != "write")
    if c["op"] == "read":
        return s
    M = c["B"] * c["T"]
    if c["op"] == "attn":
        # scores of a standard deviation of 2: few tokens of many matter
        s["q"] = (2.0 * torch.randn((M, c["Hq"] * D), generator=g, device=DEV)).to(torch.bfloat16)
        return s
    heads = c["Hq"] + 2 * c["Hkv"]
    x = torch.randn((M, heads * D), generator=g, device=DEV)
    # channels of unequal size, as a projection's output has them
    x *= torch.exp(0.5 * torch.randn((heads * D,), generator=g, device=DEV))
    s["qkv"] = x.to(torch.bfloat16)
    del x
    s["news"] = _news(c)
    s["new"] = torch.tensor(s["news"], dtype=torch.int32, device=DEV)
    s["start"] = s["total"] - s["new"]
    s["q"] = torch.zeros((M, c["Hq"] * D), dtype=torch.bfloat16, device=DEV)
    s["rules"] = {}
    if c["norm"]:
        s["rules"] = {k: (1.0 + 0.1 * torch.randn((D,), generator=g, device=DEV)).to(torch.bfloat16)
                      for k in ("q_gamma", "k_gamma")}
        s["rules"]["eps"] = 1e-6
    if c["R"]:
        P = c["L"] + 8
        s["rules"]["cos_sin"] = _table(P, c["R"])
        if c["axes"] > 1:
            # time, height and width of an image's tokens
            s["rules"]["positions"] = torch.randint(0, P, (c["axes"], M), generator=g, device=DEV).to(torch.int32)
            s["rules"]["axes"] = (torch.arange(c["R"] // 2, device=DEV) * c["axes"] // (c["R"] // 2)).to(torch.uint8)
    return s


# --------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if op == "write":
        return _own_write(state) if own else _plain_write(state)
    if op == "read":
        return _own_read(state) if own else _plain_read(state)
    return _own_attn(state) if own else _plain_attn(state)


def _own_write(s):
    from w4a16_linear_layers_gb300 import qlin

    c = s["case"]
    q = qlin.kv_write_i8(s["qkv"], s["cache"], s["table"], s["total"], c["Hq"], new_len=s["new"], **s["rules"], q=s["q"])
    k, v = qlin.kv_read_bf16(s["cache"], s["table"], s["total"], c["T"], start=s["start"])
    return {"q": q, "k": k, "v": v}


def _own_read(s):
    from w4a16_linear_layers_gb300 import qlin

    k, v = qlin.kv_read_bf16(s["cache"], s["table"], s["total"], s["case"]["L"])
    return {"k": k, "v": v}


def _own_attn(s):
    from w4a16_linear_layers_gb300 import qlin

    c = s["case"]
    return qlin.paged_attn_i8(s["q"], s["cache"], s["table"], s["total"], causal=c["causal"], window=c["window"],
                              softcap=c["softcap"])


# ------------------------------------------------------------ plain forms

def _token_blocks(s, b, first, last):
    """(index of the cache's block, place in it) of a sequence's tokens, for each head: [n, Hkv], [n]."""
    c = s["case"]
    t = torch.arange(first, last, device=DEV)
    page = s["table"][b, t // c["page"]].long()
    h = torch.arange(c["Hkv"], device=DEV)
    blocks = c["page"] // BLOCK
    return (page[:, None] * c["Hkv"] + h[None, :]) * blocks + (t % c["page"] // BLOCK)[:, None], t % BLOCK


def _take(s, b, first, last):
    """Codes [2, n, Hkv, 128] and scales [2, n, Hkv] of a sequence's tokens."""
    flat = s["cache"].view(-1, BLOCK_BYTES)
    block, r = _token_blocks(s, b, first, last)
    place = _places()[r]
    codes, scales = [], []
    for i in range(2):
        codes.append(flat[block[:, :, None], i * BLOCK * D + place[:, None, :]].int() - 128)
        byte = 2 * BLOCK * D + i * 4 * BLOCK + 4 * r
        scales.append(torch.stack([flat[block, (byte + j)[:, None]] for j in range(4)], -1).view(torch.float32)[..., 0])
    return codes, scales


def _put(s, b, first, which, codes, scales):
    flat = s["cache"].view(-1, BLOCK_BYTES)
    block, r = _token_blocks(s, b, first, first + codes.shape[0])
    flat[block[:, :, None], which * BLOCK * D + _places()[r][:, None, :]] = (codes + 128).to(torch.uint8)
    byte = 2 * BLOCK * D + which * 4 * BLOCK + 4 * r
    bytes4 = scales.contiguous().view(torch.uint8).view(*scales.shape, 4)
    for j in range(4):
        flat[block, (byte + j)[:, None]] = bytes4[..., j]


def _rotated(s, x, at, rules):
    """x [n, heads, 128] in 64 bits with cos and sin of its rows' positions."""
    c = s["case"]
    if not c["R"]:
        return x
    half = c["R"] // 2
    table = rules["cos_sin"]
    if "positions" in rules:
        pos = rules["positions"][:, at["rows"]].long().clamp(0, table.shape[0] - 1)      # [axes, n]
        pos = pos[rules["axes"].long()]                                                  # [half, n]
        i = torch.arange(half, device=DEV)[:, None]
        cos, sin = table[pos, i].T.double(), table[pos, half + i].T.double()
    else:
        cos, sin = table[at["pos"], :half].double(), table[at["pos"], half:].double()
    cos, sin = cos[:, None, :], sin[:, None, :]
    a, b = x[..., :half], x[..., half:c["R"]]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., c["R"]:]], -1)


def _plain_write(s):
    # 64 bits: a quotient next to a rounding border decides a code
    c, rules = s["case"], s["rules"]
    T, Hq, Hkv = c["T"], c["Hq"], c["Hkv"]
    k_out = torch.zeros((c["B"], T, Hkv, D), dtype=torch.bfloat16, device=DEV)
    v_out = torch.zeros_like(k_out)
    for b in range(c["B"]):
        n, first = s["news"][b], s["lens"][b] - s["news"][b]
        rows = torch.arange(b * T, b * T + n, device=DEV)
        at = {"rows": rows, "pos": torch.arange(first, first + n, device=DEV)}
        x = s["qkv"][b * T:b * T + n].view(n, Hq + 2 * Hkv, D).double()
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        q_size = k_size = 1.0
        if c["norm"]:
            # the norm's factor of a head cancels in its codes
            q_size = 1.0 / torch.sqrt((q * q).mean(-1, keepdim=True) + rules["eps"])
            k_size = 1.0 / torch.sqrt((k * k).mean(-1, keepdim=True) + rules["eps"])
            q, k = q * rules["q_gamma"].double(), k * rules["k_gamma"].double()
        s["q"][b * T:b * T + n] = (_rotated(s, q, at, rules) * q_size).to(torch.bfloat16).view(n, Hq * D)
        k = _rotated(s, k, at, rules)
        for which, (y, size, to) in enumerate(((k, k_size, k_out), (v, 1.0, v_out))):
            top = y.abs().amax(-1, keepdim=True)
            codes = torch.round(127.0 * y / torch.where(top > 0, top, torch.ones_like(top))).int()
            scales = (top * size / 127.0).float()[..., 0]
            _put(s, b, first, which, codes, scales)
            to[b, :n] = (codes.float() * scales[..., None]).to(torch.bfloat16)
    return {"q": s["q"], "k": k_out, "v": v_out}


def _plain_read(s):
    c = s["case"]
    out = [torch.zeros((c["B"], c["L"], c["Hkv"], D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for b, n in enumerate(s["lens"]):
        for first in range(0, n, 8192):
            last = min(n, first + 8192)
            codes, scales = _take(s, b, first, last)
            for i in range(2):
                out[i][b, first:last] = (codes[i].float() * scales[i][..., None]).to(torch.bfloat16)
    return {"k": out[0], "v": out[1]}


def _mask(c, n, first):
    """Which of the tokens first .. n - 1 the new ones see."""
    i = torch.arange(n - c["T"], n, device=DEV)[:, None]
    j = torch.arange(first, n, device=DEV)[None, :]
    ok = j <= i if c["causal"] else j < n
    if c["window"]:
        ok = ok & ((i - j).abs() < c["window"])
    return ok


def _plain_attn(s):
    c = s["case"]
    T, Hq, Hkv = c["T"], c["Hq"], c["Hkv"]
    G = Hq // Hkv
    out = torch.empty_like(s["q"])
    for b, n in enumerate(s["lens"]):
        first = n - _seen(c, n)
        codes, scales = _take(s, b, first, n)
        k = codes[0].float() * scales[0][..., None]
        v = codes[1].float() * scales[1][..., None]
        q = s["q"][b * T:(b + 1) * T].float().view(T, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, T * G, D)
        x = torch.bmm(q, k.permute(1, 2, 0)) / math.sqrt(D)
        if c["softcap"]:
            x = c["softcap"] * torch.tanh(x / c["softcap"])
        ok = _mask(c, n, first).repeat_interleave(G, 0)[None]
        x = torch.where(ok, x, torch.full((), -math.inf, device=DEV))
        p = torch.exp(x - x.amax(-1, keepdim=True))
        o = torch.bmm(p, v.permute(1, 0, 2)) / p.sum(-1, keepdim=True)
        out[b * T:(b + 1) * T] = o.view(Hkv, T, G, D).permute(1, 0, 2, 3).reshape(T, Hq * D).to(torch.bfloat16)
    return out


# ------------------------------------------------- the definitions in 64 bits

def _unpacked(s):
    """Every token of every page in 64 bits: [pages, page, Hkv, 128], keys and values."""
    pages, Hkv, blocks, _ = s["cache"].shape
    where = _places().reshape(-1)
    both = []
    for i in range(2):
        part = s["cache"][..., i * BLOCK * D:(i + 1) * BLOCK * D][..., where]
        codes = part.view(pages, Hkv, blocks * BLOCK, D).transpose(1, 2).to(torch.float64) - 128.0
        lo = 2 * BLOCK * D + 4 * BLOCK * i
        scale = s["cache"][..., lo:lo + 4 * BLOCK].contiguous().view(torch.float32)
        both.append(codes * scale.view(pages, Hkv, blocks * BLOCK, 1).transpose(1, 2).to(torch.float64))
    return both


def _exact_write(s):
    c, r = s["case"], s["rules"]
    B, T, Hq, Hkv, half = c["B"], c["T"], c["Hq"], c["Hkv"], c["R"] // 2
    x = s["qkv"].view(B, T, Hq + 2 * Hkv, D).to(torch.float64)
    t = torch.arange(T, device=DEV)[None, :]
    live = t < s["new"][:, None]
    pos = (s["start"][:, None] + t).clamp(min=0)
    if c["norm"]:
        gain = torch.ones((Hq + 2 * Hkv, D), dtype=torch.float64, device=DEV)
        gain[:Hq], gain[Hq:Hq + Hkv] = r["q_gamma"].to(torch.float64), r["k_gamma"].to(torch.float64)
        size = torch.rsqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / D + r["eps"])
        size[:, :, Hq + Hkv:] = 1.0
        x = x * gain
    else:
        size = torch.ones((B, T, Hq + 2 * Hkv, 1), dtype=torch.float64, device=DEV)
    if half:
        if "positions" in r:
            each = r["positions"].view(-1, B, T)[r["axes"].to(torch.int64)].permute(1, 2, 0).to(torch.int64)
        else:
            each = pos[:, :, None].expand(B, T, half).to(torch.int64)
        each = each.clamp(0, r["cos_sin"].shape[0] - 1)
        pair = torch.arange(half, device=DEV)
        turn = torch.complex(r["cos_sin"][each, pair].to(torch.float64), r["cos_sin"][each, half + pair].to(torch.float64))
        z = torch.complex(x[:, :, :Hq + Hkv, :half].contiguous(), x[:, :, :Hq + Hkv, half:2 * half].contiguous())
        z = z * turn[:, :, None, :]
        x = x.clone()
        x[:, :, :Hq + Hkv, :half], x[:, :, :Hq + Hkv, half:2 * half] = z.real, z.imag
    q = (x[:, :, :Hq] * size[:, :, :Hq]).reshape(B * T, Hq * D)
    kv = x[:, :, Hq:]
    top = torch.linalg.vector_norm(kv, ord=math.inf, dim=-1, keepdim=True)
    step = (top * size[:, :, Hq:] / 127.0)
    kv = torch.round(torch.nan_to_num(kv * 127.0 / top, nan=0.0)) * step
    kv = torch.where(live[:, :, None, None], kv, 0.0)
    q = torch.where(live.reshape(-1, 1), q, 0.0)
    return {"q": q, "k": kv[:, :, :Hkv], "v": kv[:, :, Hkv:]}


def _exact_read(s):
    c = s["case"]
    page = c["page"]
    out = []
    for pool in _unpacked(s):
        rows = pool[s["table"].long()].reshape(c["B"], -1, c["Hkv"], D)
        full = torch.zeros((c["B"], c["L"], c["Hkv"], D), dtype=torch.float64, device=DEV)
        n = min(c["L"], rows.shape[1])
        full[:, :n] = rows[:, :n]
        full[torch.arange(c["L"], device=DEV)[None, :] >= s["total"][:, None]] = 0.0
        out.append(full)
        del rows
    assert page % BLOCK == 0
    return {"k": out[0], "v": out[1]}


def _exact_attn(s):
    c = s["case"]
    T, Hq, Hkv = c["T"], c["Hq"], c["Hkv"]
    out = torch.empty((c["B"], T, Hq, D), dtype=torch.float64, device=DEV)
    keys, values = _unpacked(s)
    q = s["q"].view(c["B"], T, Hq, D).to(torch.float64)
    for b, n in enumerate(s["lens"]):
        pages = s["table"][b, :-(-n // c["page"])].long()
        far = torch.arange(n - T, n, device=DEV)[:, None] - torch.arange(n, device=DEV)[None, :]
        hidden = torch.zeros_like(far, dtype=torch.bool)
        if c["causal"]:
            hidden |= far < 0
        if c["window"]:
            hidden |= (far >= c["window"]) | (far <= -c["window"])
        for h in range(Hkv):
            k = keys[pages, :, h].reshape(-1, D)[:n]
            v = values[pages, :, h].reshape(-1, D)[:n]
            mine = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = torch.einsum("tgd,nd->gtn", q[b, :, mine], k) * D ** -0.5
            if c["softcap"]:
                x = torch.tanh(x / c["softcap"]) * c["softcap"]
            p = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[b, :, mine] = torch.einsum("gtn,nd->tgd", p, v)
    return out.view(c["B"] * T, Hq * D)


def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attn": _exact_attn}[case["op"]](s)
