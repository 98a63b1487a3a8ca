"""Cases of the serving operators next to the Hyena mixer: the residual addition with its
root-mean-square norm (plain and 8-bit output), the page map built from request lengths, the append
into the 8-bit K/V cache and the attention that reads it.

Each case can be run in a plain form (elementary torch operations in 32 bits) or, with ``own`` set,
through genomic_lm_amd.

Cache layout: K (pages, heads, page tokens, head dim), V (pages, heads, head dim, page tokens), both
e4m3, with one fp32 scale per (page, head) each: a code stands for code * scale.
"""
import math
import random

import torch

own = False

FP8_MAX = 448.0
MIN_SCALE = 2.0 ** -96       # lower bound of a cache block's scale
NORM_GROUP = 128             # columns that share a scale in the norm's grouped output
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of each of 16 sequences in front of in_proj, scales per token: latency
        {"name": "norm fp8 16 x 4096", "op": "norm", "rows": 16, "dim": 4096, "dtype": "bf16",
         "residual": True, "out": "fp8", "group": 0},
        # a 32768-token prefill in front of in_proj, a scale per 128 columns: the largest norm
        {"name": "norm fp8 32768 x 4096", "op": "norm", "rows": 32768, "dim": 4096, "dtype": "bf16",
         "residual": True, "out": "fp8", "group": NORM_GROUP},
        # odd row length and fp32 activations: rows that are not 16-byte aligned
        {"name": "norm fp32 5000 x 1001", "op": "norm", "rows": 5000, "dim": 1001, "dtype": "fp32",
         "residual": True, "out": "plain", "group": 0},
        # the tables of one decode step of 16 sequences: latency
        {"name": "map decode 16", "op": "map", "requests": 16, "kind": "decode", "max_old": 32768,
         "max_new": 1, "page": 64, "lens": 1},
        # a step that mixes decodes with prefill chunks of up to 4096 tokens, small pages
        {"name": "map mixed 512", "op": "map", "requests": 512, "kind": "mixed", "max_old": 32768,
         "max_new": 4096, "page": 16, "lens": 2},
        # one token of each of 128 sequences into the caches of 32 heads
        {"name": "append decode 128", "op": "append", "requests": 128, "kind": "decode", "max_old": 1024,
         "max_new": 1, "page": 64, "hkv": 32, "dim": 128, "dtype": "bf16", "lens": 3},
        # prefill chunks of up to 8192 tokens
        {"name": "append chunks 5", "op": "append", "requests": 5, "kind": "chunk", "max_old": 1000,
         "max_new": 8192, "page": 64, "hkv": 32, "dim": 128, "dtype": "bf16", "lens": 4},
        # a single sequence's token over 1024 cached ones: latency
        {"name": "attn decode 1 x 1k", "op": "attn", "requests": 1, "kind": "decode", "max_old": 1024,
         "max_new": 1, "page": 64, "hq": 32, "hkv": 32, "dim": 128, "dtype": "bf16", "lens": 5},
        # a decode batch with shared K/V heads and ragged lengths
        {"name": "attn decode 64 x 8k", "op": "attn", "requests": 64, "kind": "decode", "max_old": 8192,
         "max_new": 1, "page": 64, "hq": 32, "hkv": 8, "dim": 128, "dtype": "bf16", "lens": 6},
        # one token over a 262144-token context: the split over a long axis
        {"name": "attn decode 1 x 262k", "op": "attn", "requests": 1, "kind": "decode", "max_old": 262144,
         "max_new": 1, "page": 64, "hq": 32, "hkv": 32, "dim": 128, "dtype": "bf16", "lens": 7},
        # a 4096-token prefill chunk at the end of a 32768-token context: matrix cores
        {"name": "attn chunk 4k at 32k", "op": "attn", "requests": 1, "kind": "chunk", "max_old": 28672,
         "max_new": 4096, "page": 64, "hq": 32, "hkv": 32, "dim": 128, "dtype": "bf16", "lens": 8},
        # decodes, chunks and idle requests in one call; fp32, small heads and pages, shared heads
        {"name": "attn mixed fp32 9", "op": "attn", "requests": 9, "kind": "mixed", "max_old": 3000,
         "max_new": 333, "page": 16, "hq": 12, "hkv": 4, "dim": 64, "dtype": "fp32", "lens": 9},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "map", "append", "attn", "attn"))
    lens = rng.randrange(1 << 30)
    if op == "norm":
        dim = _log(rng, 64, 8192)
        out, group = rng.choice((("plain", 0), ("fp8", 0), ("fp8", NORM_GROUP)))
        return {"op": op, "rows": _log(rng, 1, min(32768, 32768 * 4096 // dim)), "dim": dim,
                "dtype": rng.choice(("bf16", "bf16", "fp32")), "residual": rng.random() < 0.7,
                "out": out, "group": group}
    page = rng.choice((16, 32, 64, 128))
    if op == "map":
        return {"op": op, "requests": _log(rng, 1, 512), "kind": rng.choice(("decode", "mixed", "chunk")),
                "max_old": _log(rng, 16, 32768), "max_new": _log(rng, 1, 1024), "page": page, "lens": lens}
    dim = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 4, 8, 32))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    kind = rng.choice(("decode", "chunk") if op == "append" else ("decode", "chunk", "mixed"))
    most = _log(rng, 1, 256)
    if op == "append":
        # at most 32768 tokens of 8192 bytes for a chunk, 64 million cached values
        old = _log(rng, 1, min(4096, max(16, 8192 * 8192 // (most * hkv * dim))))
        new = 1 if kind == "decode" else _log(rng, 2, max(2, min(4096, 4096 * 8192 // (most * hkv * dim))))
        return {"op": op, "requests": most, "kind": kind, "max_old": old, "max_new": new, "page": page,
                "hkv": hkv, "dim": dim, "dtype": dtype, "lens": lens}
    group = rng.choice((1, 1, 3, 4, 8))
    hq = hkv * group
    # bounded over all requests, each as long as the longest: cached values, scores, outputs
    old = _log(rng, 16, max(16, min(65536, (1 << 28) // (most * hkv * dim))))
    new = 1 if kind == "decode" else _log(rng, 2, 2048)
    while new > 1 and (most * hq * new * (old + new) > 1 << 31 or most * (old + new) * hkv * dim > 1 << 29
                       or most * hq * new * dim > 1 << 27):
        new = (new + 1) // 2
    return {"op": op, "requests": most, "kind": kind, "max_old": old, "max_new": new, "page": page,
            "hq": hq, "hkv": hkv, "dim": dim, "dtype": dtype, "lens": lens}


def _lengths(case):
    """Cached and new tokens of each request: a part of the case, not of its inputs."""
    rng = random.Random(case["lens"])
    n, most = case["requests"], case["max_new"]
    old = [rng.randint(1, case["max_old"]) for _ in range(n)]
    old[-1] = case["max_old"]
    if case["kind"] == "decode":
        new = [1] * n
    else:
        new = [rng.randint(1, most) for _ in range(n)]
        new[0] = most
        if case["kind"] == "mixed":
            # one request in eight is a chunk, one is idle, the others decode a token
            new = [x if i % 8 == 0 else 0 if i % 8 == 5 else 1 for i, x in enumerate(new)]
    return old, new


def _ceil(a, b):
    return -(-a // b)


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["dim"]
        size = 2 if case["dtype"] == "bf16" else 4
        reads = size * (2 if case["residual"] else 1)
        writes = (size if case["residual"] else 0) + (1 if case["out"] == "fp8" else size)
        scales = 0
        if case["out"] == "fp8":
            scales = 4 * case["rows"] * (_ceil(case["dim"], case["group"]) if case["group"] else 1)
        return {"bytes": n * (reads + writes) + scales + 4 * case["dim"], "flops": 6 * n}
    old, new = _lengths(case)
    tokens, page = sum(new), case["page"]
    if case["op"] == "map":
        fresh = sum(_ceil(o + n, page) - _ceil(o, page) for o, n in zip(old, new))
        # lengths in and out, the prefix sums; a table entry for each new page and its place in the
        # free list; a position and a slot for each token
        return {"bytes": 16 * len(old) + 8 * fresh + 12 * tokens, "flops": 4 * tokens}
    size = 2 if case["dtype"] == "bf16" else 4
    width = case["hkv"] * case["dim"]
    if case["op"] == "append":
        return {"bytes": tokens * (2 * width * (size + 1) + 8), "flops": 6 * tokens * width}
    read = sum(o + n for o, n in zip(old, new) if n)
    seen = sum(n * o + n * (n + 1) // 2 for o, n in zip(old, new))
    return {"bytes": 2 * width * read + 2 * size * tokens * case["hq"] * case["dim"],
            "flops": 4 * seen * case["hq"] * case["dim"]}


# ------------------------------------------------------------------ inputs
def _tables(case, g, after):
    """Lengths, table and free pages of a step, on the GPU. `after`: the table already holds the
    pages of the new tokens."""
    old, new = _lengths(case)
    page, n = case["page"], case["requests"]
    whole = [_ceil(o + x, page) for o, x in zip(old, new)]
    have = whole if after else [_ceil(o, page) for o in old]
    width = max(whole) + 1
    pages = sum(whole) + 8
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor(have, device="cuda")
    start = torch.cumsum(count, 0) - count
    j = torch.arange(width, device="cuda")
    held = j[None] < count[:, None]
    at = (start[:, None] + j[None]).clamp(max=pages - 1)
    s = {"table": torch.where(held, order[at], -1).to(torch.int32), "pages": pages,
         "free": order[sum(have):].contiguous(), "head": torch.zeros(1, dtype=torch.int32, device="cuda"),
         "old": torch.tensor(old, dtype=torch.int32, device="cuda"),
         "new": torch.tensor(new, dtype=torch.int32, device="cuda"),
         "lens": torch.tensor([o + x for o, x in zip(old, new)], dtype=torch.int32, device="cuda"),
         "tokens": sum(new), "most_new": max(new), "most": max(o + x for o, x in zip(old, new))}
    s["cu"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    s["cu"][1:] = torch.cumsum(s["new"], 0)
    return s


def _codes(shape, g):
    """e4m3 codes of normally distributed values that use the format's range."""
    c = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for i in range(0, shape[0], 512):
        part = torch.randn((min(512, shape[0] - i), *shape[1:]), generator=g, device="cuda")
        c[i:i + 512] = (part * 112).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return c


def _cache(s, case, g, lo, hi):
    """A cache whose blocks have scales 2^lo ... 2^(hi - 1)."""
    n, h, p, d = s["pages"], case["hkv"], case["page"], case["dim"]
    s["k_cache"], s["v_cache"] = _codes((n, h, p, d), g), _codes((n, h, d, p), g)
    for k in ("k_scale", "v_scale"):
        s[k] = torch.exp2(torch.randint(lo, hi, (n, h), generator=g, device="cuda").float())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES.get(case.get("dtype"))
    if case["op"] == "norm":
        shape = (case["rows"], case["dim"])

        def stream(spread):
            # rows of a residual stream differ in size by orders of magnitude
            size = torch.exp(spread * torch.randn((shape[0], 1), generator=g, device="cuda"))
            return (torch.randn(shape, generator=g, device="cuda") * size).to(dtype)

        s = {"x": stream(0.5), "weight": 1 + 0.1 * torch.randn(shape[1], generator=g, device="cuda"),
             "residual": stream(2.0) if case["residual"] else None, "eps": 1e-6}
    elif case["op"] == "map":
        s = _tables(case, g, after=False)
    else:
        s = _tables(case, g, after=True)
        if case["op"] == "append":
            _cache(s, case, g, -9, -5)
            # each token's slot: the page of its position, and its place there
            req = torch.repeat_interleave(torch.arange(case["requests"], device="cuda"), s["new"].long(),
                                          output_size=s["tokens"])
            pos = s["old"].long()[req] + torch.arange(s["tokens"], device="cuda") - s["cu"].long()[req]
            s["slots"] = s["table"].long()[req, pos // case["page"]] * case["page"] + pos % case["page"]
            for k in ("k", "v"):
                x = torch.randn((s["tokens"], case["hkv"], case["dim"]), generator=g, device="cuda")
                x *= torch.exp2(2 * torch.rand((s["tokens"], 1, 1), generator=g, device="cuda") - 1)
                s[k] = x.to(dtype)
        else:
            _cache(s, case, g, -8, -5)
            s["q"] = torch.randn((s["tokens"], case["hq"], case["dim"]), generator=g, device="cuda").to(dtype)
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms
def _norm(s):
    case, x = s["case"], s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    r = {"residual": x.to(s["x"].dtype)} if s["residual"] is not None else {}
    if case["out"] == "plain":
        return {"y": y.to(s["x"].dtype), **r}
    rows, dim = y.shape
    group = case["group"] or dim
    runs = _ceil(dim, group)
    z = torch.nn.functional.pad(y, (0, runs * group - dim)).view(rows, runs, group)
    top = z.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / FP8_MAX, torch.ones_like(top))
    q = (z / scale).view(rows, runs * group)[:, :dim].to(torch.float8_e4m3fn)
    return {"q": q, "scale": scale.view(rows, runs) if case["group"] else scale.view(rows), **r}


def _map(s):
    page, table, free, head = s["case"]["page"], s["table"], s["free"], s["head"].long()
    old, new = s["old"].long(), s["new"].long()
    lens = old + new
    have, want = (old + page - 1) // page, (lens + page - 1) // page
    need = want - have
    end = torch.cumsum(need, 0)
    j = torch.arange(table.shape[1], device="cuda")[None]
    at = head + (end - need)[:, None] + j - have[:, None]
    fresh = (j >= have[:, None]) & (j < want[:, None])
    got = fresh & (at < free.numel())
    table.copy_(torch.where(got, free[at.clamp(0, free.numel() - 1)], table))
    cu = torch.zeros(old.numel() + 1, dtype=torch.int64, device="cuda")
    cu[1:] = torch.cumsum(new, 0)
    t = torch.arange(s["tokens"], device="cuda")
    req = torch.searchsorted(cu[1:], t, right=True)
    pos = old[req] + t - cu[req]
    entry = table[req, pos // page].long()
    slots = torch.where(entry >= 0, entry * page + pos % page, -1)
    status = torch.cat([torch.clamp(head + end[-1:], max=free.numel()), (slots < 0).sum()[None]])
    return {"table": table, "cu": cu.int(), "lens": lens.int(), "positions": pos.int(), "slots": slots,
            "status": status.int()}


def _block_scale(top):
    """The smallest power of two s with top / s <= 448, at least MIN_SCALE."""
    m, e = torch.frexp(top / FP8_MAX)
    s = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))
    return torch.where(top > 0, s, torch.zeros_like(s)).clamp_(min=MIN_SCALE)


def _append(s):
    page, slots, first = s["case"]["page"], s["slots"], s["slots"][s["cu"][:-1].long()]
    at, off, edge, filled = slots // page, slots % page, first // page, first % page
    touched = torch.zeros(s["pages"], dtype=torch.bool, device="cuda").index_fill_(0, at, True)
    fresh = torch.ones_like(touched).index_copy_(0, edge, filled == 0)
    here = torch.arange(page, device="cuda")[None] < filled[:, None]
    for x, cache, scale, kept in ((s["k"], s["k_cache"], s["k_scale"], here[:, None, :, None]),
                                  (s["v"], s["v_cache"], s["v_scale"], here[:, None, None, :])):
        x = x.float()
        top = torch.zeros_like(scale).index_reduce_(0, at, x.abs().amax(-1), "amax")
        want = _block_scale(top)
        after = torch.where(touched[:, None], torch.where(fresh[:, None], want, torch.maximum(scale, want)), scale)
        # a request's first page may hold older tokens: their codes move to the block's new scale
        bits = cache.view(torch.uint8)
        was = bits[edge]
        moved = was.view(torch.float8_e4m3fn).float() * (scale[edge] / after[edge])[..., None, None]
        bits[edge] = torch.where(kept, moved.to(torch.float8_e4m3fn).view(torch.uint8), was)
        code = (x / after[at][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        if cache is s["k_cache"]:
            bits[at, :, off, :] = code
        else:
            bits[at, :, :, off] = code
        scale.copy_(after)
    return {k: s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _attn(s):
    case = s["case"]
    n, page, hq, hkv, dim = case["requests"], case["page"], case["hq"], case["hkv"], case["dim"]
    span = _ceil(s["most"], page)
    length, rows = span * page, s["most_new"]
    table = s["table"][:, :span].long().clamp(min=0)
    lens, cu, new = s["lens"].long(), s["cu"].long(), s["new"].long()
    j = torch.arange(length, device="cuda")
    here = (j[None] < lens[:, None])[:, None]

    def load(cache, scale):
        x = cache.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        return x * scale[table][..., None, None]

    k = load(s["k_cache"], s["k_scale"]).permute(0, 2, 1, 3, 4).reshape(n, hkv, length, dim)
    v = load(s["v_cache"], s["v_scale"]).permute(0, 2, 1, 4, 3).reshape(n, hkv, length, dim)
    v = torch.where(here[..., None], v, 0.0)
    i = torch.arange(rows, device="cuda")
    q = s["q"][(cu[:-1, None] + i[None]).clamp(max=s["tokens"] - 1)].float()
    q = q.view(n, rows, hkv, hq // hkv, dim).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, dim)
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(dim)).view(n, hkv, -1, rows, length)
    pos = (lens - new)[:, None] + i[None]
    seen = (j[None, None] <= pos[:, :, None]) & here
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp_(min=-3e38)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(n, hkv, -1, length), v).view(n, hkv, -1, rows, dim)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n, rows, hq, dim)
    t = torch.arange(s["tokens"], device="cuda")
    req = torch.searchsorted(cu[1:], t, right=True)
    return {"out": o[req, t - cu[req]].to(s["q"].dtype)}


# ------------------------------------------------------------------ the framework's operators
def _own(s):
    import genomic_lm_amd as G

    case = s["case"]
    if case["op"] == "norm":
        if case["out"] == "plain":
            y, r = G.add_rmsnorm(s["x"], s["weight"], s["residual"], eps=s["eps"])
            return {"y": y, "residual": r} if r is not None else {"y": y}
        q, scale, r = G.add_rmsnorm_fp8(s["x"], s["weight"], s["residual"], eps=s["eps"], group=case["group"])
        return {"q": q, "scale": scale, "residual": r} if r is not None else {"q": q, "scale": scale}
    if case["op"] == "map":
        cu, lens, positions, slots, status = G.page_map(s["old"], s["new"], s["table"], s["free"], s["head"],
                                                        case["page"], s["tokens"])
        return {"table": s["table"], "cu": cu, "lens": lens, "positions": positions, "slots": slots,
                "status": status}
    if case["op"] == "append":
        G.kv_append_fp8(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        return {k: s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale")}
    return {"out": G.attn_paged_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                    s["lens"], s["cu"], s["most_new"])}


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm, "map": _map, "append": _append, "attn": _attn}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "map":
        return None
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "norm":
        t = s["x"].to(f) + (s["residual"].to(f) if s["residual"] is not None else 0)
        y = t / (t.pow(2).sum(1, keepdim=True) / t.shape[1] + s["eps"]).sqrt() * s["weight"].to(f)
        r = {"residual": t} if s["residual"] is not None else {}
        if case["out"] == "plain":
            return {"y": y, **r}
        parts = y.split(case["group"] or t.shape[1], dim=1)
        scales = [p.abs().max(1).values / FP8_MAX for p in parts]
        q = torch.cat([p / c[:, None] for p, c in zip(parts, scales)], 1)
        return {"q": q, "scale": torch.stack(scales, 1) if case["group"] else scales[0], **r}
    if case["op"] == "append":
        return _exact_append(case, s)
    return _exact_attn(case, s)


def _exact_append(case, s):
    page, cu = case["page"], s["cu"].tolist()
    out = {"k_cache": s["k_cache"].to(torch.float64), "v_cache": s["v_cache"].to(torch.float64),
           "k_scale": s["k_scale"].to(torch.float64), "v_scale": s["v_scale"].to(torch.float64)}
    for r in range(case["requests"]):
        a, slots = cu[r], s["slots"][cu[r]:cu[r + 1]].tolist()
        while slots:
            p, o = divmod(slots[0], page)
            n = min(page - o, len(slots))
            for x, cache, scale in ((s["k"], out["k_cache"][p], out["k_scale"]),
                                    (s["v"], out["v_cache"][p].transpose(1, 2), out["v_scale"])):
                x = x[a:a + n].to(torch.float64).transpose(0, 1)
                need = torch.exp2(torch.ceil(torch.log2(x.abs().amax((1, 2)) / FP8_MAX))).clamp(min=MIN_SCALE)
                if o:
                    need = torch.maximum(need, scale[p])
                    cache[:, :o] *= (scale[p] / need)[:, None, None]
                cache[:, o:o + n] = x / need[:, None, None]
                scale[p] = need
            a, slots = a + n, slots[n:]
    return out


def _exact_attn(case, s):
    f, group = torch.float64, case["hq"] // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=f, device="cuda")
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    for r in range(case["requests"]):
        a, b, n = cu[r], cu[r + 1], lens[r]
        if a == b:
            continue
        pages = s["table"][r, :_ceil(n, case["page"])].long()
        future = torch.arange(n, device="cuda")[None] > torch.arange(n - (b - a), n, device="cuda")[:, None]
        step = max(1, min(case["hkv"], (1 << 28) // (group * (b - a) * n)))
        for h in range(0, case["hkv"], step):
            k = s["k_cache"][:, h:h + step].view(torch.uint8)[pages].view(torch.float8_e4m3fn).to(f)
            v = s["v_cache"][:, h:h + step].view(torch.uint8)[pages].view(torch.float8_e4m3fn).to(f)
            k = k * s["k_scale"][pages, h:h + step].to(f)[..., None, None]
            v = v * s["v_scale"][pages, h:h + step].to(f)[..., None, None]
            heads = k.shape[1]
            k = k.permute(1, 3, 0, 2).reshape(heads, case["dim"], -1)[..., :n].contiguous()
            v = v.permute(1, 0, 3, 2).reshape(heads, -1, case["dim"])[:, :n].contiguous()
            q = s["q"][a:b, h * group:(h + heads) * group].to(f).view(b - a, heads, group, -1)
            for i in range(group):
                z = torch.matmul(q[:, :, i].transpose(0, 1).contiguous(), k) / math.sqrt(case["dim"])
                w = torch.softmax(z.masked_fill(future[None], float("-inf")), -1)
                out[a:b, h * group + i::group][:, :heads] = torch.matmul(w, v).transpose(0, 1)
    return {"out": out}
