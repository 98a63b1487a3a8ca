"""Cases of the 8-bit projections of a block and of its rotary positions: the product of e4m3
activations and e4m3 weights with a scale for each run or block of 128, the gated feed-forward's first
half (both projections, activation and product, plain or 8-bit output), the quantisation that makes their
operands, and the norms of query and key heads with the rotation in the same pass.

Each case can be run in a plain form (elementary torch operations in 32 bits) or, with ``own`` set,
through genomic_lm_amd.

Operands of a product y = x w^T: x (T, K) e4m3 with fp32 scales (T) or (T, ceil(K / 128)), w (N, K) e4m3 with
fp32 scales (ceil(N / 128), ceil(K / 128)): a code stands for code * scale.
"""
import math
import random

import torch

own = False

FP8_MAX = 448.0
GROUP = 128                  # columns (and rows of a weight) that share a scale
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token in front of a Hyena mixer (in_proj), a scale per token: latency, the weight is read once
        {"name": "linear 1 x 4096 to 12288", "op": "linear", "rows": 1, "k": 4096, "n": 12288, "group": 0,
         "bias": False, "out": "bf16"},
        # one token of each of 16 sequences through the feed-forward's last projection
        {"name": "linear 16 x 11008 to 4096", "op": "linear", "rows": 16, "k": 11008, "n": 4096, "group": GROUP,
         "bias": False, "out": "bf16"},
        # a mixed step of an odd number of tokens, odd widths (rows that are not aligned), fp32 out
        {"name": "linear 333 x 1001 to 1000 fp32", "op": "linear", "rows": 333, "k": 1001, "n": 1000,
         "group": GROUP, "bias": True, "out": "fp32"},
        # a prefill of 8192 tokens in front of a Hyena mixer
        {"name": "linear 8192 x 4096 to 12288", "op": "linear", "rows": 8192, "k": 4096, "n": 12288,
         "group": GROUP, "bias": False, "out": "bf16"},
        # the feed-forward of four decoding sequences, codes for its last projection
        {"name": "gated 4 x 4096 to 11008 fp8", "op": "gated", "rows": 4, "k": 4096, "n": 11008, "group": GROUP,
         "act": "gelu", "out": "fp8"},
        # a chunk of a prompt, inner width that is no multiple of 128
        {"name": "gated 1000 x 4096 to 10928", "op": "gated", "rows": 1000, "k": 4096, "n": 10928, "group": 0,
         "act": "silu", "out": "bf16"},
        # the feed-forward of a prefill of 8192 tokens
        {"name": "gated 8192 x 4096 to 11008 fp8", "op": "gated", "rows": 8192, "k": 4096, "n": 11008,
         "group": GROUP, "act": "gelu", "out": "fp8"},
        # a mixer's output of 16 decoding sequences in front of out_proj: latency
        {"name": "quantize 16 x 4096", "op": "quantize", "rows": 16, "dim": 4096, "block": 1, "group": 0,
         "dtype": "bf16"},
        # the same for a 32768-token prefill
        {"name": "quantize 32768 x 4096", "op": "quantize", "rows": 32768, "dim": 4096, "block": 1, "group": GROUP,
         "dtype": "bf16"},
        # a projection's weight at load time, fp32 checkpoint
        {"name": "quantize weight 11008 x 4096", "op": "quantize", "rows": 11008, "dim": 4096, "block": GROUP,
         "group": GROUP, "dtype": "fp32"},
        # one token of each of 16 sequences, eight query heads for each key head: latency
        {"name": "rope 16 x 32 + 4 heads", "op": "rope", "tokens": 16, "requests": 16, "hq": 32, "hk": 4,
         "dim": 128, "rotary": 128, "norm": True, "interleaved": False, "base": 10000.0, "factor": 32.0,
         "most": 262144, "dtype": "bf16"},
        # ragged prompts of 32768 tokens in all, every head with its own keys
        {"name": "rope 32768 x 32 + 32 heads", "op": "rope", "tokens": 32768, "requests": 5, "hq": 32, "hk": 32,
         "dim": 128, "rotary": 128, "norm": True, "interleaved": False, "base": 10000.0, "factor": 1.0,
         "most": 40000, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """Widths of layers: multiples of 128, of 16, or any."""
    n = _log(rng, lo, hi)
    step = rng.choice((128, 16, 16, 1))
    return max(step, n // step * step)


def draw(rng):
    op = rng.choice(("linear", "gated", "linear", "gated", "quantize", "rope"))
    if op in ("linear", "gated"):
        case = {"op": op, "k": _width(rng, 64, 11008), "n": _width(rng, 64, 12288),
                "group": rng.choice((0, GROUP))}
        most = (4e11 if op == "linear" else 2e11) / (case["k"] * case["n"])
        case["rows"] = _log(rng, 1, int(min(8192, max(1, most))))
        if op == "linear":
            return {**case, "bias": rng.random() < 0.5, "out": rng.choice(("bf16", "bf16", "fp32"))}
        return {**case, "act": rng.choice(("gelu", "gelu_tanh", "silu", "none")),
                "out": rng.choice(("fp8", "fp8", "bf16", "fp32"))}
    if op == "quantize":
        block = rng.choice((1, 1, GROUP))
        dim = _width(rng, 64, 11008)
        return {"op": op, "rows": _log(rng, 1, min(32768, (1 << 27) // dim)), "dim": dim, "block": block,
                "group": GROUP if block > 1 else rng.choice((0, GROUP)), "dtype": rng.choice(("bf16", "fp32"))}
    hk, dim = rng.choice((1, 2, 4, 8, 32)), rng.choice((64, 64, 128, 128, 96, 80))
    tokens = _log(rng, 1, 16384)
    norm = rng.random() < 0.5
    return {"op": op, "tokens": tokens, "requests": min(tokens, _log(rng, 1, 32)),
            "hq": min(32, hk * rng.choice((1, 2, 3, 4, 8))), "hk": hk, "dim": dim,
            "rotary": rng.choice((dim, dim, dim // 2)), "norm": norm, "interleaved": rng.random() < 0.3,
            "base": rng.choice((10000.0, 1e6)), "factor": rng.choice((1.0, 32.0)),
            "most": _log(rng, 20000, 1000000), "dtype": rng.choice(("bf16", "bf16", "fp32"))}


def _ceil(a, b):
    return -(-a // b)


def work(case):
    if case["op"] in ("linear", "gated"):
        t, k, n, two = case["rows"], case["k"], case["n"], 2 if case["op"] == "gated" else 1
        runs = _ceil(k, GROUP)
        scales = 4 * (t * (runs if case["group"] else 1) + two * runs * _ceil(n, GROUP))
        out = t * n * {"bf16": 2, "fp32": 4, "fp8": 1}[case["out"]]
        if case["out"] == "fp8":
            out += 4 * t * _ceil(n, GROUP)
        return {"bytes": t * k + two * n * k + scales + out + (4 * n if case.get("bias") else 0),
                "flops": 2 * two * t * n * k}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "quantize":
        n = case["rows"] * case["dim"]
        runs = _ceil(case["dim"], case["group"]) if case["group"] else 1
        return {"bytes": n * (size + 1) + 4 * _ceil(case["rows"], case["block"]) * runs, "flops": 3 * n}
    heads = case["hq"] + case["hk"]
    n = case["tokens"] * heads * case["dim"]
    return {"bytes": 2 * size * n + 4 * case["tokens"], "flops": (6 if case["norm"] else 3) * n}


# ------------------------------------------------------------------ inputs
def _codes(shape, g):
    """e4m3 codes of normally distributed values that use the format's range."""
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * 112).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def _scales(shape, size, g):
    return size / 112 * torch.exp(0.5 * torch.randn(shape, generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] in ("linear", "gated"):
        t, k, n = case["rows"], case["k"], case["n"]
        runs = _ceil(k, GROUP)
        s["x"] = _codes((t, k), g)
        s["x_scale"] = _scales((t, runs) if case["group"] else (t,), 1.0, g)
        for i in range(2 if case["op"] == "gated" else 1):
            s["w%d" % i] = _codes((n, k), g)
            s["w%d_scale" % i] = _scales((_ceil(n, GROUP), runs), k ** -0.5, g)
        s["bias"] = torch.randn(n, generator=g, device="cuda") if case.get("bias") else None
    elif case["op"] == "quantize":
        # rows of a mixer's output, or of a weight, differ in size
        size = torch.exp(torch.randn((case["rows"], 1), generator=g, device="cuda"))
        x = torch.randn((case["rows"], case["dim"]), generator=g, device="cuda") * size
        s["x"] = x.to(DTYPES[case["dtype"]])
    else:
        hq, hk, d, t, n = case["hq"], case["hk"], case["dim"], case["tokens"], case["requests"]
        # queries, keys and values side by side, as the projection leaves them
        x = torch.randn((t, hq + 2 * hk, d), generator=g, device="cuda")
        x = x.mul_(torch.exp(0.5 * torch.randn((t, 1, 1), generator=g, device="cuda"))).to(DTYPES[case["dtype"]])
        s["q"], s["k"] = x[:, :hq], x[:, hq:hq + hk]
        # requests of random lengths, each at a random place of its sequence
        rng = random.Random(seed)
        cut = sorted(rng.sample(range(1, t), n - 1)) if t > 1 else []
        parts = [(b - a, rng.randrange(max(1, case["most"] - (b - a)))) for a, b in zip([0] + cut, cut + [t])]
        s["positions"] = torch.cat([torch.arange(a, a + m, dtype=torch.int32) for m, a in parts]).cuda()
        i = torch.arange(0, case["rotary"], 2, dtype=torch.float64)
        s["inv_freq"] = (case["base"] ** (-i / case["rotary"]) / case["factor"]).float().cuda()
        if case["norm"]:
            s["q_weight"], s["k_weight"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in "qk")
            s["eps"] = 1e-6
        else:
            s["q_weight"] = s["k_weight"] = s["eps"] = None
    return s


# ------------------------------------------------------------------ plain forms
def _wide(q, scale, rows):
    """What the codes stand for, in 32 bits: a scale for `rows` rows by GROUP columns, or for each row."""
    n, k = q.shape
    if scale.dim() == 1:
        return q.float() * scale[:, None]
    scale = scale.repeat_interleave(rows, 0)[:n] if rows > 1 else scale
    return q.float() * scale.repeat_interleave(GROUP, 1)[:, :k]


def _quantized(y, block, group):
    """Codes and scales of blocks of `block` rows by `group` columns (0: whole rows)."""
    rows, dim = y.shape
    group = group or dim
    down, runs = _ceil(rows, block), _ceil(dim, group)
    z = torch.nn.functional.pad(y, (0, runs * group - dim, 0, down * block - rows))
    z = z.view(down, block, runs, group)
    top = z.abs().amax((1, 3), keepdim=True)
    scale = torch.where(top > 0, top / FP8_MAX, torch.ones_like(top))
    q = (z / scale).view(down * block, runs * group)[:rows, :dim].to(torch.float8_e4m3fn)
    return q, scale.view(down, runs)


def _activated(g, act):
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return g


def _product(s):
    case = s["case"]
    x = _wide(s["x"], s["x_scale"], 1)
    y = torch.matmul(x, _wide(s["w0"], s["w0_scale"], GROUP).t())
    if case["op"] == "linear":
        if s["bias"] is not None:
            y = y + s["bias"]
        return {"y": y.to(DTYPES[case["out"]])}
    h = _activated(y, case["act"]) * torch.matmul(x, _wide(s["w1"], s["w1_scale"], GROUP).t())
    if case["out"] != "fp8":
        return {"h": h.to(DTYPES[case["out"]])}
    q, scale = _quantized(h, 1, GROUP)
    return {"q": q, "scale": scale}


def _quantize(s):
    case = s["case"]
    q, scale = _quantized(s["x"].float(), case["block"], case["group"])
    return {"q": q, "scale": scale if case["group"] else scale.view(-1)}


def _rope(s):
    case = s["case"]
    half = case["rotary"] // 2
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        if case["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s[name + "_weight"]
        r, rest = x[..., :2 * half], x[..., 2 * half:]
        if case["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        out[name] = torch.cat([turned, rest], -1).to(s[name].dtype)
    return out


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    import genomic_lm_amd as G

    case = s["case"]
    if case["op"] == "linear":
        return {"y": G.linear_fp8(s["x"], s["x_scale"], s["w0"], s["w0_scale"], bias=s["bias"],
                                  dtype=DTYPES[case["out"]])}
    if case["op"] == "gated":
        args = (s["x"], s["x_scale"], s["w0"], s["w0_scale"], s["w1"], s["w1_scale"], case["act"])
        if case["out"] != "fp8":
            return {"h": G.gated_linear_fp8(*args, dtype=DTYPES[case["out"]])}
        q, scale = G.gated_linear_fp8(*args, dtype=torch.float8_e4m3fn)
        return {"q": q, "scale": scale}
    if case["op"] == "quantize":
        q, scale = (G.quantize_weight_fp8(s["x"]) if case["block"] > 1
                    else G.quantize_fp8(s["x"], group=case["group"]))
        return {"q": q, "scale": scale}
    q, k = G.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"],
                          eps=s["eps"], interleaved=case["interleaved"])
    return {"q": q, "k": k}


def run(state):
    if own:
        return _own(state)
    return {"linear": _product, "gated": _product, "quantize": _quantize, "rope": _rope}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "quantize":
        x, b = s["x"].to(f), case["block"]
        q, scales = torch.empty_like(x), []
        for i in range(0, x.shape[0], b if b > 1 else x.shape[0]):
            rows = slice(i, i + b) if b > 1 else slice(None)
            line = []
            for part, to in zip(x[rows].split(case["group"] or x.shape[1], 1),
                                q[rows].split(case["group"] or x.shape[1], 1)):
                c = part.abs().max() / FP8_MAX if b > 1 else part.abs().max(1).values / FP8_MAX
                to.copy_(part / (c if b > 1 else c[:, None]))
                line.append(c)
            scales.append(torch.stack(line, -1) if case["group"] else line[0])
        return {"q": q, "scale": torch.stack(scales) if b > 1 else scales[0]}
    if case["op"] == "rope":
        turn = torch.polar(torch.ones((), dtype=f, device="cuda"),
                           s["positions"].to(f)[:, None] * s["inv_freq"].to(f)[None])[:, None]
        out = {}
        for name in "qk":
            x = s[name].to(f)
            if case["norm"]:
                x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt()
                x = x * s[name + "_weight"].to(f)
            n = s["inv_freq"].numel()
            first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if case["interleaved"] else (
                slice(0, n), slice(n, 2 * n))
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            x[..., first], x[..., second] = z.real, z.imag
            out[name] = x
        return out

    def product(w, scale):
        # run by run of K: the codes' products, then the run's scales
        y = torch.zeros((case["rows"], case["n"]), dtype=f, device="cuda")
        for j, a in enumerate(range(0, case["k"], GROUP)):
            z = torch.matmul(s["x"][:, a:a + GROUP].to(f), w[:, a:a + GROUP].to(f).t())
            z *= (s["x_scale"][:, j] if case["group"] else s["x_scale"]).to(f)[:, None]
            y += z * scale[:, j].to(f).repeat_interleave(GROUP)[:case["n"]]
        return y

    y = product(s["w0"], s["w0_scale"])
    if case["op"] == "linear":
        return {"y": y if s["bias"] is None else y + s["bias"].to(f)}
    if case["act"] == "gelu":
        y = y * (1 - 0.5 * torch.erfc(y / math.sqrt(2)))
    elif case["act"] == "gelu_tanh":
        y = y * torch.sigmoid(math.sqrt(8 / math.pi) * (y + 0.044715 * y ** 3))
    elif case["act"] == "silu":
        y = y * torch.sigmoid(y)
    h = y * product(s["w1"], s["w1_scale"])
    if case["out"] != "fp8":
        return {"h": h}
    parts = h.split(GROUP, 1)
    scales = [p.abs().max(1).values / FP8_MAX for p in parts]
    return {"q": torch.cat([p / c[:, None] for p, c in zip(parts, scales)], 1), "scale": torch.stack(scales, 1)}
