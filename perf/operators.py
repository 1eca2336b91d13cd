"""Cases of the operators around a per-channel W8A8 linear: the residual
addition fused with RMSNorm and the per-token INT8 quantization, the INT8
product with one scale per token and one per output channel, and the logits
adjusted by penalties, biases and grammar masks.

``own`` False computes each operator in elementary torch operations, True
calls the library (``w4a16_linear_layers_gb300.qlin``).
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token entering a hidden-5120 layer: latency counts
        {"name": "addnorm_c16_1x5120", "op": "addnorm", "codes": "c16", "M": 1, "K": 5120, "y": False},
        # a decode batch of eight drafted tokens, int8 codes for the small-batch linear
        {"name": "addnorm_i8_8x5120", "op": "addnorm", "codes": "i8", "M": 8, "K": 5120, "y": False},
        # a ragged chunk of a prompt at the intermediate width, the norm's bf16 output kept too
        {"name": "addnorm_c16_333x17408_y", "op": "addnorm", "codes": "c16", "M": 333, "K": 17408, "y": True},
        # a long prompt
        {"name": "addnorm_c16_8192x5120", "op": "addnorm", "codes": "c16", "M": 8192, "K": 5120, "y": False},
        # a key/value projection for one token: latency counts
        {"name": "gemm_i8_1x5120x1024", "op": "gemm", "codes": "i8", "M": 1, "K": 5120, "N": 1024},
        # the fused gate/up projection of a drafted block of eight tokens
        {"name": "gemm_i8_8x5120x34816", "op": "gemm", "codes": "i8", "M": 8, "K": 5120, "N": 34816},
        # the vocabulary head for twelve drafted blocks of eight
        {"name": "gemm_c16_96x5120x248320", "op": "gemm", "codes": "c16", "M": 96, "K": 5120, "N": 248320},
        # the down projection of a ragged prompt chunk, int8 codes
        {"name": "gemm_i8_509x17408x5120", "op": "gemm", "codes": "i8", "M": 509, "K": 17408, "N": 5120},
        # the fused gate/up projection of a long prompt
        {"name": "gemm_c16_8192x5120x34816", "op": "gemm", "codes": "c16", "M": 8192, "K": 5120, "N": 34816},
        # one sequence, all rules, logits written in bf16
        {"name": "logits_bf16_1x248320", "op": "logits", "type": "bf16", "M": 1, "V": 248320, "L": 2000, "B": 16,
         "mask": True, "write": True, "argmax": True},
        # a batch of ninety-six sequences with long histories
        {"name": "logits_bf16_96x248320", "op": "logits", "type": "bf16", "M": 96, "V": 248320, "L": 8192, "B": 64,
         "mask": True, "write": True, "argmax": True},
        # fp32 logits of a small vocabulary, greedy tokens only
        {"name": "logits_f32_33x50264_argmax", "op": "logits", "type": "f32", "M": 33, "V": 50264, "L": 515, "B": 0,
         "mask": False, "write": False, "argmax": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# no drawn case costs more than its operator's largest listed one
_MOST = {"addnorm": ("bytes", 335_000_000), "gemm": ("flops", 2_920_000_000_000), "logits": ("bytes", 101_000_000)}
_MOST_BYTES = 1_320_000_000


def _fits(c):
    w = work(c)
    key, most = _MOST[c["op"]]
    return w[key] <= most and w["bytes"] <= _MOST_BYTES


def draw(rng):
    op = rng.choice(["addnorm", "gemm", "logits"])
    if op == "addnorm":
        c = {"op": op, "codes": rng.choice(["i8", "c16"]), "M": _log(rng, 1, 8192), "K": 128 * _log(rng, 1, 256),
             "y": rng.random() < 0.3}
    elif op == "gemm":
        c = {"op": op, "codes": rng.choice(["i8", "c16"]), "M": _log(rng, 1, 8192), "K": 128 * _log(rng, 1, 200),
             "N": 8 * _log(rng, 8, 31040)}
    else:
        c = {"op": op, "type": rng.choice(["bf16", "f32"]), "M": _log(rng, 1, 256), "V": 8 * _log(rng, 125, 32768),
             "L": rng.choice([0, 1, _log(rng, 2, 8192)]), "B": rng.choice([0, 1, _log(rng, 2, 300)]),
             "mask": rng.random() < 0.6, "write": rng.random() < 0.7, "argmax": True}
    wide = "N" if op == "gemm" else None
    while not _fits(c):
        if c["M"] > 1:
            c["M"] = max(1, c["M"] * 3 // 4)
        elif wide:
            c[wide] = c[wide] // 16 * 8
    return c


def work(case):
    c = case
    if c["op"] == "addnorm":
        M, K = c["M"], c["K"]
        code = 1 if c["codes"] == "i8" else 2
        return {"bytes": M * K * (6 + code + (2 if c["y"] else 0)) + 2 * K + 4 * M, "flops": 10 * M * K}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        code = 1 if c["codes"] == "i8" else 2
        return {"bytes": K * N + 4 * N + code * M * K + 4 * M + 2 * M * N, "flops": 2 * M * N * K}
    M, V = c["M"], c["V"]
    e = 2 if c["type"] == "bf16" else 4
    return {"bytes": M * V * e * (2 if c["write"] else 1) + (M * ((V + 31) // 32) * 4 if c["mask"] else 0)
            + M * (4 * c["L"] + 8 * c["B"] + 24), "flops": 4 * M * V}


# ------------------------------------------------------------------ inputs

def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _outliers(g, M, K):
    """Activations as a residual stream has them: normal, a few channels 20 times larger."""
    x = torch.randn((M, K), generator=g, device=DEV)
    hot = torch.randint(0, K, (8,), generator=g, device=DEV)
    x[:, hot] *= 20.0
    return x


def prepare(case, seed):
    c = dict(case)
    if c["op"] == "addnorm":
        M, K = c["M"], c["K"]
        g = _gen(seed, 1)
        return {"case": c,
                "x": torch.randn((M, K), generator=g, device=DEV).to(torch.bfloat16),
                "residual": _outliers(g, M, K).to(torch.bfloat16),
                "gamma": (1.0 + 0.1 * torch.randn((K,), generator=g, device=DEV)).to(torch.bfloat16),
                "eps": 1e-6}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        g = _gen(seed, 2)
        x = torch.randn((M, K), generator=g, device=DEV)
        # channels of unequal size, as the input of a projection has them
        x *= torch.exp(0.8 * torch.randn((K,), generator=g, device=DEV))
        s_a = x.abs().amax(1) / 127.0
        q = torch.round(x / s_a[:, None]).clamp_(-127, 127)
        q = q.to(torch.int8) if c["codes"] == "i8" else q.to(torch.float16)
        # 8-bit GPTQ words: byte i of word (kk, n) is code (4 kk + i, n) + 128
        words = torch.zeros((K // 4, N), dtype=torch.int32, device=DEV)
        for i in range(4):
            w = torch.randn((K // 4, N), generator=g, device=DEV).mul_(32.0).round_().clamp_(-127, 127)
            words |= (w.to(torch.int32) + 128) << (8 * i)
            del w
        s_w = torch.exp(torch.empty((N,), device=DEV).uniform_(math.log(1e-4), math.log(1e-3), generator=g))
        return {"case": c, "q": q, "s_a": s_a, "qweight": words, "s_w": s_w}
    M, V, L, B = c["M"], c["V"], c["L"], c["B"]
    g = _gen(seed, 3)
    s = {"case": c, "logits": (4.0 * torch.randn((M, V), generator=g, device=DEV)).to(_TYPES[c["type"]]), "rules": {}}
    r = s["rules"]
    if L:
        # text repeats its tokens: half from a small set, half from the whole vocabulary
        few = torch.randint(0, V, (M, 64), generator=g, device=DEV)
        tok = torch.randint(0, V, (M, L), generator=g, device=DEV)
        pick = torch.gather(few, 1, torch.randint(0, 64, (M, L), generator=g, device=DEV))
        r["tokens"] = torch.where(torch.rand((M, L), generator=g, device=DEV) < 0.5, pick, tok).to(torch.int32)
        total = torch.randint(L // 2, L + 1, (M,), generator=g, device=DEV)
        r["total_len"] = total.to(torch.int32)
        r["prompt_len"] = (total // 2).to(torch.int32)
        r["repetition"] = 1.0 + 0.5 * torch.rand((M,), generator=g, device=DEV)
        r["presence"] = torch.rand((M,), generator=g, device=DEV)
        r["frequency"] = 0.2 * torch.rand((M,), generator=g, device=DEV)
    if B:
        r["bias_ids"] = torch.randint(-1, V, (M, B), generator=g, device=DEV).to(torch.int32)
        r["bias"] = 5.0 * torch.randn((M, B), generator=g, device=DEV)
    if c["mask"]:
        r["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (M, (V + 31) // 32), generator=g, device=DEV).to(torch.int32)
    return s


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if op == "addnorm":
        return _own_addnorm(state) if own else _plain_addnorm(state)
    if op == "gemm":
        return _own_gemm(state) if own else _plain_gemm(state)
    return _own_logits(state) if own else _plain_logits(state)


def _own_addnorm(state):
    from w4a16_linear_layers_gb300 import qlin

    c = state["case"]
    x = state["x"]
    y = torch.empty_like(x) if c["y"] else None
    if c["codes"] == "i8":
        q, s, h = qlin.add_rmsnorm_act_quant_i8(x, state["residual"], state["gamma"], state["eps"], y=y)
        q = q.float() * s[:, None]
    else:
        q, s, h = qlin.add_rmsnorm_act_quant_c16(x, state["residual"], state["gamma"], state["eps"], y=y)
    return {"q": q, "s": s, "h": h, "y": y} if c["y"] else {"q": q, "s": s, "h": h}


def _own_gemm(state):
    from w4a16_linear_layers_gb300 import qlin

    call = qlin.gemm_w8a8_ch if state["case"]["codes"] == "i8" else qlin.gemm_w8a8_ch_c16
    return call(state["q"], state["s_a"], state["qweight"], state["s_w"])


def _own_logits(state):
    from w4a16_linear_layers_gb300 import qlin

    c = state["case"]
    if not c["write"]:
        return {"token": qlin.adjust_logits_argmax(state["logits"], **state["rules"])}
    out = torch.empty_like(state["logits"])
    token = qlin.adjust_logits_argmax(state["logits"], **state["rules"], out=out)
    return {"logits": out, "token": token}


# ------------------------------------------------------------ plain forms

def _bf16(d):
    """binary64 -> bf16, rounded once: through binary32 rounded to odd."""
    f = d.to(torch.float32)
    back = f.to(torch.float64)
    f = torch.where(back.abs() > d.abs(), torch.nextafter(f, torch.zeros_like(f)), f)
    odd = (f.to(torch.float64) != d).to(torch.int32)
    return (f.view(torch.int32) | odd).view(torch.float32).to(torch.bfloat16)


def _plain_addnorm(state):
    c = state["case"]
    h = (state["x"].float() + state["residual"].float()).to(torch.bfloat16)
    hd = h.double()
    # 64 bits: a norm's output next to a rounding border decides a code
    rstd = 1.0 / torch.sqrt((hd * hd).sum(1, keepdim=True) / c["K"] + state["eps"])
    t = _bf16(hd * rstd)
    z = (state["gamma"].float() * t.float()).to(torch.bfloat16)
    zf = z.float()
    s = zf.abs().amax(1) / torch.full((), 127.0, device=zf.device)
    safe = torch.where(s > 0, s, torch.ones_like(s))
    q = torch.round(zf / safe[:, None]).clamp(-127, 127)
    q = q * s[:, None] if c["codes"] == "i8" else q.to(torch.float16)
    return {"q": q, "s": s, "h": h, "y": z} if c["y"] else {"q": q, "s": s, "h": h}


def _unpack(qweight):
    K4, N = qweight.shape
    return torch.stack([((qweight >> (8 * i)) & 255) - 128 for i in range(4)], 1).reshape(4 * K4, N)


def _plain_gemm(state):
    p = state["q"].float() @ _unpack(state["qweight"]).float()
    return ((p * state["s_w"]) * state["s_a"][:, None]).to(torch.bfloat16)


def _counts(tokens, keep, V):
    """How often each id occurs at the kept places; ids outside [0, V) do not count."""
    M = tokens.shape[0]
    ids = torch.where(keep & (tokens >= 0) & (tokens < V), tokens, V).long()
    n = torch.zeros((M, V + 1), dtype=torch.int32, device=tokens.device)
    return n.scatter_add_(1, ids, torch.ones_like(ids, dtype=torch.int32))[:, :V]


def _plain_logits(state):
    c, r = state["case"], state["rules"]
    x = state["logits"].float()
    M, V = x.shape
    if "tokens" in r:
        at = torch.arange(r["tokens"].shape[1], device=x.device)[None, :]
        made = _counts(r["tokens"], (at >= r["prompt_len"][:, None]) & (at < r["total_len"][:, None]), V)
        seen = _counts(r["tokens"], at < r["total_len"][:, None], V) > 0
        rep = r["repetition"][:, None]
        x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
        x = torch.where(made > 0, x - (r["frequency"][:, None] * made.float() + r["presence"][:, None]), x)
    if "bias_ids" in r:
        # of entries with the same id the last one counts
        B = r["bias_ids"].shape[1]
        ids = torch.where((r["bias_ids"] >= 0) & (r["bias_ids"] < V), r["bias_ids"], V).long()
        slot = torch.full((M, V + 1), -1, dtype=torch.int64, device=x.device)
        slot.scatter_reduce_(1, ids, torch.arange(B, device=x.device).expand(M, B), "amax")
        slot = slot[:, :V]
        x = torch.where(slot >= 0, x + torch.gather(r["bias"], 1, slot.clamp(min=0)), x)
    if "allowed" in r:
        bit = torch.arange(V, device=x.device)
        ok = (r["allowed"][:, bit // 32] >> (bit % 32)) & 1
        x = torch.where(ok != 0, x, torch.full((), -math.inf, device=x.device))
    x = x.to(state["logits"].dtype)
    v = torch.where(torch.isnan(x), torch.full((), -math.inf, device=x.device, dtype=x.dtype), x)
    best = v.amax(1, keepdim=True)
    at = torch.arange(V, device=x.device, dtype=torch.int32)
    token = torch.where(v == best, at, V).amin(1).to(torch.int32)
    token = torch.where(best[:, 0] == -math.inf, -1, token).to(torch.int32)
    return {"logits": x, "token": token} if c["write"] else {"token": token}


# ------------------------------------------------- the definitions in 64 bits

def _round_to_bf16(v):
    """binary64 rounded to 8 significant bits, half to even, on its own bits."""
    u = v.view(torch.int64)
    u = u + ((1 << 44) - 1) + ((u >> 45) & 1)
    return (u & ~((1 << 45) - 1)).view(torch.float64)


def _exact_addnorm(s):
    # h, t, z and the scale are rounded by the operator's definition, and a
    # code is the nearest integer to the binary32 quotient
    c = s["case"]
    h = _round_to_bf16(s["x"].double() + s["residual"].double())
    norm = torch.linalg.vector_norm(h, dim=1, keepdim=True)
    t = _round_to_bf16(h / torch.sqrt(norm * norm / c["K"] + s["eps"]))
    z = _round_to_bf16(t * s["gamma"].double())
    scale = (z.abs().max(1).values / 127.0).float().double()
    q = torch.round(torch.nan_to_num((z / scale[:, None]).float().double(), nan=0.0))
    if c["codes"] == "i8":
        q = q * scale[:, None]
    return {"q": q, "s": scale, "h": h, "y": z} if c["y"] else {"q": q, "s": scale, "h": h}


def _exact_gemm(s):
    K4, N = s["qweight"].shape
    M = s["q"].shape[0]
    q = s["q"].double().reshape(M, K4, 4)
    p = torch.zeros((M, N), dtype=torch.float64, device=DEV)
    for byte in range(4):
        code = torch.bitwise_and(torch.bitwise_right_shift(s["qweight"], 8 * byte), 0xFF).double() - 128.0
        p += torch.matmul(q[:, :, byte], code)
        del code
    return p * torch.outer(s["s_a"].double(), s["s_w"].double())


def _exact_logits(s):
    c, r = s["case"], s["rules"]
    x = s["logits"].double().cpu().clone()
    M, V = x.shape
    for m in range(M):
        row = x[m]
        if "tokens" in r:
            total, prompt = int(r["total_len"][m]), int(r["prompt_len"][m])
            t = r["tokens"][m, :total].cpu().long()
            ids = torch.unique(t)
            rep = float(r["repetition"][m])
            row[ids] = torch.where(row[ids] > 0, row[ids] / rep, row[ids] * rep)
            ids, n = torch.unique(t[prompt:], return_counts=True)
            row[ids] -= n.double() * float(r["frequency"][m]) + float(r["presence"][m])
        if "bias_ids" in r:
            last = dict(zip(r["bias_ids"][m].tolist(), r["bias"][m].tolist()))
            for i, b in last.items():
                if 0 <= i < V:
                    row[i] += b
        if "allowed" in r:
            words = r["allowed"][m].cpu().long() & 0xFFFFFFFF
            bits = (words[:, None] >> torch.arange(32)) & 1
            row[bits.reshape(-1)[:V] == 0] = -math.inf
    return {"logits": x, "token": None}


def exact(case, seed):
    if case["op"] == "logits" and not case["write"]:
        return None
    s = prepare(case, seed)
    return {"addnorm": _exact_addnorm, "gemm": _exact_gemm, "logits": _exact_logits}[case["op"]](s)
