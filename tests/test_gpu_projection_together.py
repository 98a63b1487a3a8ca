"""The 8-bit projections, the quantisation, the rotary positions and the serving operators as a block uses them:
together against 64 bits, captured into a graph, on other streams and from several host threads."""
import threading

import numpy as np
import pytest
import torch

import genomic_lm_amd as G
from genomic_lm_amd import serving
from tests import projection_ref as ref
from tests import serving_ref
from tests.gpu_util import dev, to_f64
from tests.serving_ref import decode

pytestmark = pytest.mark.gpu

BF, F8, U8 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.lib()
    yield


def raw(t):
    return t.contiguous().view(U8).cpu().numpy()


def bits_equal(a, b):
    return torch.equal(a.contiguous().view(-1).view(U8), b.contiguous().view(-1).view(U8))


class Block:
    """An attention block with its MLP: heads of 64, an inner width that is no multiple of 128."""

    def __init__(self, requests, new, dim=256, heads=4, inner=688, page=16, old=40, seed=0):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s, scale=1.0: (torch.randn(s, generator=g) * scale).to(dev())  # noqa: E731
        self.heads, self.dim, self.page, self.inner = heads, dim, page, inner
        weight = lambda *s: G.quantize_weight_fp8(rand(*s, scale=s[1] ** -0.5))  # noqa: E731
        self.w_in, self.w_out, self.w_down = weight(3 * dim, dim), weight(dim, dim), weight(dim, inner)
        self.w_gate, self.w_up = weight(inner, dim), weight(inner, dim)
        self.norms = [1 + rand(dim, scale=0.1) for _ in range(2)]
        self.qw, self.kw = 1 + rand(dim // heads, scale=0.1), 1 + rand(dim // heads, scale=0.1)
        self.inv = G.rotary_inv_freq(dim // heads, factor=32.0)
        self.tokens, self.most = requests * new, new
        per = -(-(old + new) // page)
        i32 = dict(dtype=torch.int32, device=dev())
        self.table = torch.arange(requests * per, **i32).view(requests, per).flip(1).contiguous()
        # the pages that page_map hands out: those past the old tokens', in the requests' order
        self.free = self.table[:, -(-old // page):].flatten().contiguous()
        self.old, self.new = torch.full((requests,), old, **i32), torch.full((requests,), new, **i32)
        self.cache = serving.new_cache(requests * per, heads, page, dim // heads)
        k, v = rand(requests * old, heads, dim // heads), rand(requests * old, heads, dim // heads)
        j = torch.arange(old, device=dev())
        slots = (self.table.long()[:, j // page] * page + j % page).reshape(-1)
        G.kv_append_fp8(k, v, slots, *self.cache)
        self.x, self.res = rand(self.tokens, dim).to(BF), rand(self.tokens, dim).to(BF)
        self.kept = [c.clone() for c in self.cache]

    def reset(self):
        for c, k in zip(self.cache, self.kept):
            c.copy_(k)

    def step(self, x):
        """Every tensor that the block makes."""
        out = {}
        cu, lens, positions, slots, _ = G.page_map(self.old, self.new, self.table, self.free, None, self.page,
                                                   self.tokens)
        out["q0"], out["s0"], out["res"] = G.add_rmsnorm_fp8(x, self.norms[0], self.res, group=128)
        proj = G.linear_fp8(out["q0"], out["s0"], *self.w_in)
        q, k, v = proj.view(-1, 3, self.heads, self.dim // self.heads).unbind(1)
        out["proj"], out["positions"] = proj, positions
        out["q"], out["k"] = G.qk_norm_rope(q, k, positions, self.inv, self.qw, self.kw, eps=1e-6)
        G.kv_append_fp8(out["k"], v, slots, *self.cache)
        out["attn"] = G.attn_paged_fp8(out["q"], *self.cache, self.table, lens, cu, self.most)
        out["q1"], out["s1"] = G.quantize_fp8(out["attn"].view(-1, self.dim), group=128)
        out["x1"] = G.linear_fp8(out["q1"], out["s1"], *self.w_out)
        out["q2"], out["s2"], out["res2"] = G.add_rmsnorm_fp8(out["x1"], self.norms[1], out["res"], group=128)
        out["h"], out["hs"] = G.gated_linear_fp8(out["q2"], out["s2"], *self.w_gate, *self.w_up, act="gelu", dtype=F8)
        out["x2"] = G.linear_fp8(out["h"], out["hs"], *self.w_down)
        return out


@pytest.mark.parametrize("requests,new", [(3, 1), (20, 1), (2, 50), (5, 70)])
def test_block_against_64_bits(requests, new):
    """Each operator against 64 bits on the inputs that the one before it gave.  The tolerances are those of
    the operators' own tests (test_gpu_projection.py) with a bf16 output: 2^-8 of the value and 2^-10 of the
    magnitudes behind a sum, which a turn and a norm stay far below."""
    b = Block(requests, new)
    out = b.step(b.x)
    wide = lambda q, s, rows=1: ref.widen(raw(q), s.cpu().numpy(), rows)  # noqa: E731

    def near(got, want, size):
        e = np.abs(to_f64(got) - want)
        assert (e <= 2.0 ** -10 * size + 2.0 ** -8 * (np.abs(want) + size * 2.0 ** -10)).all(), (e / (size + 1e-30)).max()

    def product(q, s, w):
        x, w = wide(q, s), wide(*w, 128)
        return x @ w.T, np.abs(x) @ np.abs(w).T

    near(out["proj"], *product(out["q0"], out["s0"], b.w_in))
    pos = out["positions"].cpu().numpy()
    assert (pos.reshape(requests, new) == 40 + np.arange(new)).all()
    heads = to_f64(out["proj"]).reshape(-1, 3, b.heads, b.dim // b.heads)
    for name, i, w in (("q", 0, b.qw), ("k", 1, b.kw)):
        near(out[name], *ref.rope(heads[:, i], pos, b.inv.cpu().numpy(), False, 1e-6, to_f64(w)))
    near(out["x1"], *product(out["q1"], out["s1"], b.w_out))
    near(out["x2"], *product(out["h"], out["hs"], b.w_down))
    # the whole block by 64-bit steps from the same codes of the cache: within a few roundings to 8 bits
    T, dh = b.tokens, b.dim // b.heads
    s, y = serving_ref.rmsnorm(to_f64(b.x), to_f64(b.res), to_f64(b.norms[0]), 1e-6)
    p = y @ wide(*b.w_in, 128).T
    p = p.reshape(T, 3, b.heads, dh)
    q, _ = ref.rope(p[:, 0], pos, b.inv.cpu().numpy(), False, 1e-6, to_f64(b.qw))
    kc, vc, ks, vs = b.cache
    lens = np.full(requests, 40 + new)
    attn, _, _ = serving_ref.attention(q, raw(kc), raw(vc), to_f64(ks), to_f64(vs), b.table.cpu().numpy(), lens,
                                       np.arange(requests + 1) * new, dh ** -0.5, b.page)
    x1 = attn.reshape(T, b.dim) @ wide(*b.w_out, 128).T
    s2, y2 = serving_ref.rmsnorm(x1, s, to_f64(b.norms[1]), 1e-6)
    h = ref.act(y2 @ wide(*b.w_gate, 128).T, "gelu") * (y2 @ wide(*b.w_up, 128).T)
    x2 = h @ wide(*b.w_down, 128).T
    far = np.linalg.norm(to_f64(out["x2"]) - x2) / np.linalg.norm(x2)
    # six roundings to e4m3 stand between (norm, cache's queries' own keys and values, attention, norm, h),
    # 2^-4 at most and 2.6 % in the mean each, carried by products that keep relative size
    assert far < 0.12, far


def test_block_in_a_graph():
    """Captured once, replayed with other inputs, eager work between the replays."""
    b = Block(4, 1, seed=1)
    x = b.x.clone()
    for _ in range(3):
        b.reset()
        b.step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    b.reset()
    with torch.cuda.graph(graph):
        held = b.step(x)
    for n in range(4):
        fresh = torch.randn(x.shape, generator=torch.Generator().manual_seed(n)).to(BF).to(dev())
        b.reset()
        want = {k: v.clone() for k, v in b.step(fresh).items()}
        b.reset()
        x.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        for k, v in want.items():
            assert bits_equal(held[k], v), (n, k)


@pytest.mark.parametrize("T", [4, 40, 200, 2100])
def test_products_in_a_graph(T):
    """Each size of kernel captured, replayed and compared with the eager call."""
    K, N = 512, 4000
    g = torch.Generator().manual_seed(T)
    w, ws = G.quantize_weight_fp8(torch.randn((N, K), generator=g).to(dev()))
    u, us = G.quantize_weight_fp8(torch.randn((N, K), generator=g).to(dev()))
    x = torch.randn((T, K), generator=g).to(BF).to(dev())

    def run():
        q, s = G.quantize_fp8(x, group=128)
        return (G.linear_fp8(q, s, w, ws), G.linear_fp8(q, s, w, ws, dtype=torch.float32),
                *G.gated_linear_fp8(q, s, w, ws, u, us, dtype=F8), G.gated_linear_fp8(q, s, w, ws, u, us, "silu"))

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for n in range(3):
        x.copy_(torch.randn((T, K), generator=g).to(BF).to(dev()))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, run()):
            assert bits_equal(a, b)


def test_streams_and_threads():
    """The current stream is the one that runs, and calls from several threads do not meet."""
    K, N = 384, 1000
    g = torch.Generator().manual_seed(5)
    w, ws = G.quantize_weight_fp8(torch.randn((N, K), generator=g).to(dev()))
    xs = [torch.randn((T, K), generator=g).to(dev()) for T in (5, 60, 300, 5, 60, 300)]
    want = [G.linear_fp8(*G.quantize_fp8(x, group=128), w, ws) for x in xs]
    torch.cuda.synchronize()
    got = [None] * len(xs)

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(5):
                got[i] = G.linear_fp8(*G.quantize_fp8(xs[i], group=128), w, ws)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert bits_equal(a, b)


def test_padded_step():
    """A step of fixed size: page_map gives the tokens past the last request position -1; their rows of the
    queries and keys stay, and the others are as in a step of their own size."""
    heads, dh, R = 3, 64, 2
    i32 = dict(dtype=torch.int32, device=dev())
    table, free = torch.zeros((R, 4), **i32), torch.arange(8, **i32)
    _, _, positions, _, _ = G.page_map(torch.tensor([3, 7], **i32), torch.tensor([2, 3], **i32), table, free, None,
                                       16, 9)
    assert positions.tolist() == [3, 4, 7, 8, 9, -1, -1, -1, -1]
    x = torch.randn((9, heads, dh), device=dev())
    before = x.clone()
    inv = G.rotary_inv_freq(dh)
    want, _ = G.qk_norm_rope(x[:5].clone(), None, positions[:5], inv, eps=1e-6)
    G.qk_norm_rope(x, None, positions, inv, eps=1e-6, q_out=x)
    assert bits_equal(x[:5], want) and bits_equal(x[5:], before[5:])
