"""The serving operators against plain 64-bit implementations (serving_ref.py).

Tolerances, stated before any run:
* norm: fp32 arithmetic.  A sum of D squares over at most 32 terms per lane and a
  tree of 10 carries at most 42 roundings, halved by the square root; the sum s,
  the quotient, eps and the products add 8: below 32 * 2^-24 = 2^-19 of
  (|x| + |r|) * inv * |w|.  Outputs add half a unit in the last place, at most
  2^-p of the value for p significant bits: 2^-8 in bf16, 2^-24 in fp32.
* norm, 8 bits: the same plus the code's own rounding, 2^-4 of the value or
  half a subnormal step (2^-10 of the scale).
* append, page map: exact.
* attention: with A = sum_j p_j |v_j|, each weight p_j may be off by the score's error --
  DH products and their sum in fp32, (DH + 8) 2^-24 of the largest
  sum |q||k| scale, twice (numerator and denominator) -- by the exponential
  (2^-21) and, for bf16 activations, by its rounding to bf16 (2^-8); sums over n
  tokens add n 2^-24; the output is rounded once (2^-8 or 2^-24 of the value)."""
import numpy as np
import pytest
import torch

import genomic_lm_amd as G
from genomic_lm_amd import serving
from tests import serving_ref as ref
from tests.gpu_util import dev, log, to_f64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.lib()
    yield


def tensor(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(dev())


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def bits_equal(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------------ norm
def check_norm(x, r, w, eps, y, ro, dtype, q=None, scale=None, group=0):
    X = to_f64(x).reshape(-1, x.shape[-1])
    R = None if r is None else to_f64(r).reshape(X.shape)
    W = None if w is None else to_f64(w)
    s, want = ref.rmsnorm(X, R, W, eps)
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    size = np.abs(X) + (0 if R is None else np.abs(R))
    _, gain = ref.rmsnorm(X, R, W, eps)
    rel = np.divide(np.abs(gain), np.abs(s), out=np.zeros_like(s), where=s != 0)      # |inv * w|
    tol = 2.0 ** -19 * size * rel
    if ro is not None:
        e = np.abs(to_f64(ro).reshape(s.shape) - s)
        assert (e <= half * np.abs(s) + 2.0 ** -24 * size + 2.0 ** -140).all(), e.max()
    if q is None:
        e = np.abs(to_f64(y).reshape(want.shape) - want)
        assert (e <= tol + half * np.abs(want) * (1 + 2.0 ** -8) + 2.0 ** -140).all(), e.max()
        return
    D = X.shape[1]
    c = ref.decode(codes(q).reshape(X.shape))
    sc = to_f64(scale).reshape(X.shape[0], -1)
    step = group or D
    assert sc.shape[1] == -(-D // step)
    for i in range(sc.shape[1]):
        run = slice(i * step, min((i + 1) * step, D))
        top = np.abs(want[:, run]).max(1)
        t = tol[:, run].max(1)
        assert (np.abs(sc[:, i] - np.where(top > 0, top / 448, 1.0)) <= (t + 2.0 ** -22 * top) / 448).all()
        e = np.abs(c[:, run] * sc[:, i:i + 1] - want[:, run])
        lim = tol[:, run] * 1.1 + 2.0 ** -4 * np.abs(want[:, run]) * (1 + 2.0 ** -8) + 2.0 ** -10 * sc[:, i:i + 1]
        assert (e <= lim).all(), (e / lim).max()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [1, 7, 64, 129, 512, 520, 1001, 1920, 2049, 4096, 5000, 8192, 8200, 32768])
def test_norm(D, dtype):
    rng = np.random.default_rng(D)
    for T, res in ((1, False), (5, True)):
        x = tensor(rng.standard_normal((T, D)) * np.exp(rng.standard_normal((T, 1))), dtype)
        r = tensor(rng.standard_normal((T, D)) * 8, dtype) if res else None
        w = tensor(1 + 0.1 * rng.standard_normal(D)) if res else None
        y, ro = G.add_rmsnorm(x, w, r, eps=1e-5)
        check_norm(x, r, w, 1e-5, y, ro, dtype)
        for group in (0, 128):
            q, sc, ro8 = G.add_rmsnorm_fp8(x, w, r, eps=1e-5, group=group)
            check_norm(x, r, w, 1e-5, None, ro8, dtype, q, sc, group)
            if res:
                assert bits_equal(ro8, ro)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_strides_and_in_place(dtype):
    rng = np.random.default_rng(3)
    wide = tensor(rng.standard_normal((3, 6, 3 * 200 + 1)), dtype)
    x = wide[:, :, 201:401]                       # rows at a stride, odd alignment, three axes
    r = tensor(rng.standard_normal((1, 1, 200)), dtype).expand(3, 6, 200)[:, :, :]
    r = r.reshape(18, 200)[:1].expand(18, 200)    # one row repeated (stride 0)
    x2 = x.reshape(18, 200)
    base, ro = G.add_rmsnorm(x2, None, r)
    check_norm(x2, r, None, 1e-6, base, ro, dtype)
    y, none = G.add_rmsnorm(x, None)
    assert none is None
    check_norm(x, None, None, 1e-6, y, None, dtype)
    # residual_out in the residual, y in x
    xa, ra = x2.clone(), r.contiguous()
    y, ro2 = G.add_rmsnorm(xa, None, ra, out=xa, residual_out=ra)
    assert y is xa and ro2 is ra and bits_equal(xa, base) and bits_equal(ra, ro)
    # residual_out in x, written into a strided view: its surroundings stay
    buf = torch.full((18, 256), 7.0, dtype=dtype, device=dev())
    buf[:, 16:216] = x2
    y, _ = G.add_rmsnorm(buf[:, 16:216], None, r, residual_out=buf[:, 16:216])
    assert bits_equal(y, base) and bits_equal(buf[:, 16:216], ro)
    assert (buf[:, :16] == 7).all() and (buf[:, 216:] == 7).all()
    with pytest.raises(ValueError):
        G.add_rmsnorm(x2.t())
    with pytest.raises(ValueError):
        G.add_rmsnorm(x2, None, residual_out=x2)


def test_norm_extremes():
    """Rows of zeros, of 1e30, of tiny values; a NaN and an infinity stay in their rows."""
    D = 1500
    rng = np.random.default_rng(4)
    x = rng.standard_normal((7, D))
    x[1] = 0.0
    x[2] *= 1e30
    x[3] *= 1e-30
    x = tensor(x)
    x[5, 70] = float("nan")
    x[6, 80] = float("inf")
    rows = [0, 1, 2, 3, 4]
    for eps in (1e-6, 0.0):
        keep = rows if eps else [0, 2, 4]          # without eps a row of zeros is 0 / 0
        y, _ = G.add_rmsnorm(x, None, eps=eps)
        check_norm(x[keep], None, None, eps, y[keep], None, F32)
        assert y[5].isnan().all() and y[6, 80].isnan()
        q, sc, _ = G.add_rmsnorm_fp8(x, None, eps=eps, group=128)
        check_norm(x[keep], None, None, eps, None, None, F32, q[keep], sc[keep], 128)
        assert (codes(q)[5] & 0x7F == 0x7F).all() and codes(q)[6, 80] & 0x7F == 0x7F
        if eps:
            assert (codes(q)[1] == 0).all() and (sc[1] == 1).all()
    # values that reach 448 times a scale below fp32's normal range
    w = torch.full((D,), 1e-38, device=dev())
    q, sc, _ = G.add_rmsnorm_fp8(x[:1], w, eps=1e-6)
    assert int((codes(q) & 0x7F).max()) == 0x7E and sc.item() > 0


def test_norm_empty_and_many_rows():
    x = torch.empty((0, 64), dtype=BF, device=dev())
    y, _ = G.add_rmsnorm(x)
    q, sc, _ = G.add_rmsnorm_fp8(x, group=128)
    assert y.shape == (0, 64) and q.shape == (0, 64) and sc.shape == (0, 1)
    # more rows than one launch takes, at the shortest row
    T = (1 << 21) + 3
    x = torch.arange(T, device=dev()).remainder(7).sub(3).to(BF)[:, None].expand(T, 8).contiguous()
    y, _ = G.add_rmsnorm(x, eps=0.25)
    want = (x.double() / torch.sqrt(x.double() ** 2 + 0.25))
    assert ((y.double() - want).abs() <= 2.0 ** -8).all()


# ------------------------------------------------------------------ page map
def run_map(old, new, table, free, head, P, T, **kw):
    t = tensor(table, I32)
    h = None if head is None else tensor(np.array([head]), I32)
    out = G.page_map(tensor(np.array(old), I32), tensor(np.array(new), I32), t,
                     tensor(np.array(free, dtype=np.int64), I32), h, P, T, **kw)
    want_table = table.copy()
    want = ref.page_map(old, new, want_table, free, head or 0, P, T)
    assert (t.cpu().numpy() == want_table).all()
    for got, w, name in zip(out, want, ("cu", "lens", "positions", "slots", "status")):
        assert (got.cpu().numpy() == w).all(), name
    return out


@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("R", [1, 2, 63, 257, 700])
def test_page_map(R, P):
    rng = np.random.default_rng(R * P)
    old = rng.integers(0, 900, R)
    new = np.where(rng.random(R) < 0.2, rng.integers(0, 700, R), rng.integers(0, 2, R))
    old[0], new[-1] = 0, 1
    have = -(-old // P)
    width = int((-(-(old + new) // P)).max()) + 1
    pool = rng.permutation(int(have.sum() + (-(-(old + new) // P) - have).sum() + 5))
    table = np.full((R, width), -1)
    at = 0
    for r in range(R):
        table[r, :have[r]] = pool[at:at + have[r]]
        at += have[r]
    free = pool[at:]
    for head, T in ((0, int(new.sum())), (None, int(new.sum()) + 37), (3, max(int(new.sum()) - 2, 0))):
        run_map(old, new, table, free, head, P, T)
    # the free list runs out, and the table does
    run_map(old, new, table, free[:2], 0, P, int(new.sum()))
    run_map(old, new, table, free[:0], 0, P, int(new.sum()))
    run_map(old, new, table[:, :max(width - 2, 1)].copy(), free, 1, P, int(new.sum()))


def test_page_map_edges():
    # no request, no token, negative lengths, a head past the list's end
    run_map([], [], np.zeros((0, 4), dtype=np.int64), [1, 2], 0, 16, 3)
    run_map([5], [0], np.array([[3, -1]]), [1], 0, 16, 0)
    run_map([-4, 16], [-1, 1], np.array([[-1, -1], [9, -1]]), [2, 8], 0, 16, 2)
    run_map([0], [40], np.full((1, 4), -1), [2, 8], 7, 16, 40)
    # lengths whose sum passes 2^31: no slot is found beyond the table
    big = 2 ** 31 - 1
    t = torch.full((2, 2), -1, dtype=I32, device=dev())
    cu, lens, pos, slots, status = G.page_map(
        tensor(np.array([big, 0]), I32), tensor(np.array([big, 20]), I32), t,
        tensor(np.array([6, 7]), I32), None, 16, 40)
    assert lens.tolist() == [big, 20] and pos.tolist()[:20] == list(range(20))
    assert slots.tolist() == [96 + i for i in range(16)] + [112 + i for i in range(4)] + [-1] * 20
    with pytest.raises(G.HyenaError):
        run_map([1], [1], np.array([[0]]), [1], 0, 24, 1)


# ------------------------------------------------------------------ append
def host_cache(c):
    return [codes(c[0]).copy(), codes(c[1]).copy(), c[2].double().cpu().numpy(), c[3].double().cpu().numpy()]


def random_cache(N, H, P, DH, seed, old=True):
    """A cache of finite random codes and power-of-two scales."""
    rng = np.random.default_rng(seed)

    def some(shape):
        c = rng.integers(0, 256, shape, dtype=np.uint8)
        return np.where(c & 0x7F == 0x7F, np.uint8(0x30), c)

    k = torch.from_numpy(some((N, H, P, DH))).to(dev()).view(torch.float8_e4m3fn)
    v = torch.from_numpy(some((N, H, DH, P))).to(dev()).view(torch.float8_e4m3fn)
    sc = [tensor(2.0 ** rng.integers(-10, -6, (N, H))) for _ in range(2)]
    return [k, v, *sc]


def check_append(cache, want):
    got = host_cache(cache)
    for g, w, name in zip(got, want, ("k_cache", "v_cache", "k_scale", "v_scale")):
        if g.dtype == np.uint8:
            nan = (g & 0x7F == 0x7F) & (w & 0x7F == 0x7F)
            assert ((g == w) | nan).all(), (name, int(((g != w) & ~nan).sum()))
        else:
            assert (g == w).all(), name


def runs(spec, P):
    """Slots of (page, first place, tokens) runs."""
    return np.concatenate([np.arange(n) + p * P + o for p, o, n in spec]) if spec else np.zeros(0, int)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P,DH,H", [(16, 64, 3), (64, 128, 2), (32, 128, 1), (256, 64, 2), (256, 128, 1)])
def test_append(P, DH, H, dtype):
    rng = np.random.default_rng(P + DH)
    spec = [(3, 0, 1), (5, 7, 1), (0, 0, P), (2, P - 1, 1), (6, 5, min(P - 5, 70)), (9, 1, 3), (7, 0, 9),
            (8, 2, 4), (10, P // 2, P - P // 2), (11, 0, 5)]
    for slots in (runs(spec, P), runs(spec[:1], P), runs(spec[::-1], P)):
        T = len(slots)
        big = np.exp2(rng.integers(-6, 5, (T, 1, 1)))
        k, v = (tensor(rng.standard_normal((T, H, DH)) * big, dtype) for _ in range(2))
        cache = random_cache(13, H, P, DH, P)
        want = host_cache(cache)
        ref.append(to_f64(k), to_f64(v), slots, *want, P)
        G.kv_append_fp8(k, v, tensor(slots, torch.int64), *cache)
        check_append(cache, want)


def test_append_long_call():
    """More tokens than the short calls' limit: runs that cross the workgroups' token groups."""
    P, H, DH, T = 64, 2, 64, 4500
    rng = np.random.default_rng(1)
    spec, left, page = [], T, 0
    while left:
        o = int(rng.integers(0, P)) if rng.random() < 0.3 else 0
        n = min(left, int(rng.integers(1, P - o + 1)) if rng.random() < 0.5 else P - o)
        spec.append((page, o, n))
        page, left = page + 1, left - n
    slots = runs(spec, P)
    k, v = (tensor(rng.standard_normal((T, H, DH)) * 4, BF) for _ in range(2))
    cache = random_cache(page, H, P, DH, 2)
    want = host_cache(cache)
    ref.append(to_f64(k), to_f64(v), slots, *want, P)
    G.kv_append_fp8(k, v, tensor(slots, torch.int64), *cache)
    check_append(cache, want)


def test_append_strides_and_holes():
    """K and V inside one fused projection; tokens without a slot and slots out of the cache."""
    P, H, DH, N = 16, 2, 64, 4
    rng = np.random.default_rng(5)
    slots = np.array([16, 17, -1, 18, 64, 1 << 40, 3 * 16 + 15, -7, 0])
    T = len(slots)
    wide = tensor(rng.standard_normal((T, 3 * H * DH + 1)), BF)
    k = wide[:, 1:1 + H * DH].unflatten(1, (H, DH))
    v = wide[:, 2 * H * DH:3 * H * DH].unflatten(1, (H, DH))
    cache = random_cache(N, H, P, DH, 6)
    want = host_cache(cache)
    ref.append(to_f64(k), to_f64(v), slots, *want, P)
    G.kv_append_fp8(k, v, tensor(slots, torch.int64), *cache)
    check_append(cache, want)
    # one head's rows for all heads (stride 0), and a call without tokens
    one = k[:, :1].expand(T, H, DH)
    ref.append(to_f64(one), to_f64(v), slots, *want, P)
    G.kv_append_fp8(one, v, tensor(slots, torch.int64), *cache)
    check_append(cache, want)
    G.kv_append_fp8(k[:0], v[:0], tensor(slots[:0], torch.int64), *cache)
    check_append(cache, want)


@pytest.mark.parametrize("n", [1, 40])
def test_append_non_finite_and_zero(n):
    P, H, DH = 64, 2, 128
    rng = np.random.default_rng(7)
    slots = runs([(1, 3, n), (2, 0, n)], P)
    k, v = (tensor(rng.standard_normal((2 * n, H, DH)), F32) for _ in range(2))
    k[0, 0, 5] = float("nan")
    v[n - 1, 1, 9] = float("-inf")
    k[n, 1, 0] = float("inf")
    k[n:, 0] = 0.0
    v[n:, 0] = 1e-35
    cache = random_cache(3, H, P, DH, 8)
    want = host_cache(cache)
    ref.append(to_f64(k), to_f64(v), slots, *want, P)
    G.kv_append_fp8(k, v, tensor(slots, torch.int64), *cache)
    check_append(cache, want)


# ------------------------------------------------------------------ attention
def attn_case(old, new, Hq, Hkv, DH, P, dtype, seed=0, width=None):
    """Cache, tables and queries of requests with old cached and new tokens.  Places past the
    lengths and unused pages hold NaN codes and NaN scales."""
    rng = np.random.default_rng(seed)
    R = len(old)
    lens = np.array(old) + np.array(new)
    need = -(-lens // P)
    N = int(need.sum()) + 3
    width = max(int(need.max()) if R else 0, 1) + 1 if width is None else width
    order = rng.permutation(N)
    table = rng.integers(-5, N + 5, (R, width))           # unused entries: anything
    kc = np.full((N, Hkv, P, DH), 0x7F, np.uint8)
    vc = np.full((N, Hkv, DH, P), 0xFF, np.uint8)
    sc = np.full((2, N, Hkv), np.nan)
    at = 0
    for r in range(R):
        for j in range(int(need[r])):
            p = order[at]
            at += 1
            table[r, j] = p
            m = min(P, lens[r] - j * P)
            kc[p, :, :m] = ref.encode(np.clip(rng.standard_normal((Hkv, m, DH)) * 100, -448, 448))
            vc[p, :, :, :m] = ref.encode(np.clip(rng.standard_normal((Hkv, DH, m)) * 100, -448, 448))
            sc[:, p] = 2.0 ** rng.integers(-8, -5, (2, Hkv))
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    q = rng.standard_normal((T, Hq, DH))
    f8 = torch.float8_e4m3fn
    return {"q": tensor(q, dtype), "k": torch.from_numpy(kc).to(dev()).view(f8),
            "v": torch.from_numpy(vc).to(dev()).view(f8), "ks": tensor(sc[0]), "vs": tensor(sc[1]),
            "table": tensor(table, I32), "lens": tensor(lens, I32), "cu": tensor(cu, I32), "P": P,
            "max_q": max(list(new) + [0]), "DH": DH, "dtype": dtype}


def attend(c, **kw):
    return G.attn_paged_fp8(c["q"], c["k"], c["v"], c["ks"], c["vs"], c["table"], c["lens"], c["cu"],
                            c["max_q"], **kw)


def check_attn(c, out, scale=None, max_q=None, label=""):
    scale = c["DH"] ** -0.5 if scale is None else scale
    want, mag, reach = ref.attention(to_f64(c["q"]), codes(c["k"]), codes(c["v"]), to_f64(c["ks"]),
                                     to_f64(c["vs"]), c["table"].cpu().numpy(), c["lens"].cpu().numpy(),
                                     c["cu"].cpu().numpy(), scale, c["P"], max_q)
    bf = c["dtype"] == BF
    n = int(c["lens"].max()) if c["lens"].numel() else 0
    weight = 2 * (c["DH"] + 8) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + n * 2.0 ** -24
    lim = mag * (weight + (2.0 ** -8 if bf else 2.0 ** -22)) + (2.0 ** -8 if bf else 2.0 ** -24) * np.abs(want) * 1.01
    got = to_f64(out)
    seen = ~np.isnan(want)
    e = np.abs(got - want)[seen]
    if e.size:
        log(f"  {label} worst error / bound {np.max(e / np.maximum(lim[seen], 1e-300)):.3f}")
    assert np.isfinite(got[seen]).all() and (e <= lim[seen] + 1e-30).all()
    return seen


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P,DH,Hq,Hkv", [(16, 64, 6, 2), (64, 128, 4, 4), (32, 128, 8, 1), (256, 64, 3, 3),
                                         (128, 128, 40, 2)])
def test_attn_ragged(P, DH, Hq, Hkv, dtype):
    """Single tokens, chunks, idle requests, lengths around the page and tile edges."""
    old = [0, 5, 63, 64, 200, 15, 0, 300, 0, 700, 127, 1]
    new = [1, 1, 1, 1, 0, 17, 33, 70, 0, 1, 2, 130]
    c = attn_case(old, new, Hq, Hkv, DH, P, dtype, seed=P + DH)
    out = attend(c)
    assert check_attn(c, out, label=f"P={P} DH={DH} Hq={Hq}/{Hkv} {dtype}").all()
    assert bits_equal(out, attend(c))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_split(dtype):
    """Long sequences over few heads: pieces that are joined, beside a short one."""
    c = attn_case([5000, 3, 2111], [1, 1, 3], 4, 1, 128, 64, dtype, seed=9)
    check_attn(c, attend(c), label="split")
    # the same with a workspace full of NaN from an earlier use, and one request alone
    need = G.attn_paged_workspace_size(3, 5, 3, c["table"].shape[1], 64, 4, 1, 128)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev())
    out = torch.full_like(c["q"], float("nan"))
    assert attend(c, workspace=ws, out=out) is out
    check_attn(c, out, label="split, dirty workspace")
    one = attn_case([4097], [1], 2, 2, 64, 16, dtype, seed=10)
    check_attn(one, attend(one), label="one long request")


def test_attn_chunk_long():
    """A chunk over a long context: many units whose pieces are joined."""
    c = attn_case([1500], [300], 4, 2, 128, 64, BF, seed=11)
    check_attn(c, attend(c), label="chunk")


def test_attn_rows_without_tokens():
    """Fewer cached tokens than queries, no cached tokens, pages out of range, a table that is
    too short: rows that see nothing are 0, hidden tokens do not count."""
    for dtype in (BF, F32):
        c = attn_case([0, 40, 90, 64], [5, 3, 1, 2], 4, 2, 64, 16, dtype, seed=12)
        c["lens"][0] = 2                       # queries 0 .. 2 stand before the first token
        c["lens"][1] = 0
        c["table"][2, 1] = -1                  # a page in the middle is gone
        c["table"][2, 3] = 10 ** 6
        out = attend(c)
        check_attn(c, out, label="holes")
        assert (out[:3] == 0).all() and (out[5:8] == 0).all()
        c["table"][3] = -1
        out = attend(c)
        check_attn(c, out)
        assert (out[9:] == 0).all()
    # lens past the table's end are cut to it
    c = attn_case([30], [2], 2, 1, 64, 16, BF, seed=13, width=2)
    c["lens"][0] = 1000
    check_attn(c, attend(c), label="cut")


def test_attn_padding_and_max_q():
    """Query rows past cu[R], and rows past max_q, are left alone."""
    c = attn_case([40, 9], [4, 1], 4, 2, 64, 16, BF, seed=14)
    c["q"] = torch.cat([c["q"], c["q"][:3]])
    out = torch.full_like(c["q"], 9.0)
    attend(c, out=out)
    seen = check_attn(c, out, label="padding")
    assert not seen[5:].any() and (out[5:] == 9).all()
    c["max_q"] = 2
    out = torch.full_like(c["q"], 9.0)
    attend(c, out=out)
    seen = check_attn(c, out, max_q=2)
    assert (out[torch.from_numpy(~seen).to(dev())] == 9).all()


def test_attn_strides_scale_and_values():
    """Queries inside a fused projection; another scale; large scores; a NaN key reaches the
    queries that see it and no others."""
    c = attn_case([30, 100], [6, 1], 4, 2, 128, 16, BF, seed=15)
    T = c["q"].shape[0]
    wide = torch.randn((T, 3, 4, 131), device=dev()).to(BF)
    wide[:, 1, :, 3:] = c["q"]
    c["q"] = wide[:, 1, :, 3:]
    check_attn(c, attend(c), label="strided")
    check_attn(c, attend(c, scale=2.0), scale=2.0, label="scale 2")
    check_attn(c, attend(c, scale=-0.5), scale=-0.5, label="scale -0.5")
    check_attn(c, attend(c, scale=0.0), scale=0.0, label="scale 0")
    base = attend(c)
    p, o = divmod(33, 16)                       # the token of query 3 of request 0
    c["k"].view(torch.uint8)[int(c["table"][0, p]), 1, o, 7] = 0x7F
    out = attend(c)
    assert out[3:6, 2:].isnan().all()
    assert bits_equal(out[:3], base[:3]) and bits_equal(out[:, :2], base[:, :2]) and bits_equal(out[6:], base[6:])


def test_attn_offsets_past_32_bits():
    """Pages whose bytes lie past 2^32 in both caches."""
    P, H, DH = 256, 8, 128
    N = (1 << 32) // (P * H * DH) + 40
    small = attn_case([1000], [1], H, H, DH, P, BF, seed=16)
    f8 = torch.float8_e4m3fn
    big = dict(small)
    big["k"] = torch.zeros((N, H, P, DH), dtype=torch.uint8, device=dev()).view(f8)
    big["v"] = torch.zeros((N, H, DH, P), dtype=torch.uint8, device=dev()).view(f8)
    big["ks"], big["vs"] = torch.zeros((N, H), device=dev()), torch.zeros((N, H), device=dev())
    n = small["k"].shape[0]
    for k in ("k", "v"):
        big[k].view(torch.uint8)[-n:] = small[k].view(torch.uint8)
    for k in ("ks", "vs"):
        big[k][-n:] = small[k]
    big["table"] = small["table"] + (N - n)
    assert bits_equal(attend(big), attend(small))
    # the append at the same place
    k = torch.randn((3, H, DH), device=dev()).to(BF)
    slots = tensor((N - 1) * P + np.arange(3), torch.int64)
    G.kv_append_fp8(k, k, slots, big["k"], big["v"], big["ks"], big["vs"])
    back = big["k"][-1, :, :3].float() * big["ks"][-1][:, None, None]
    assert ((back.transpose(0, 1) - k.float()).abs() <= 2.0 ** -4 * k.float().abs() + 2.0 ** -10 * big["ks"][-1][None, :, None]).all()
    assert torch.equal(big["v"][-1, :, :, :3].float(), big["k"][-1, :, :3].float().transpose(1, 2))


# ------------------------------------------------------------------ together
def step(tables, cache, qkv, H, DH, P):
    """One serving step of a layer: map, append, attend."""
    old, new, table, free, head, T, max_q = tables
    cu, lens, _, slots, status = G.page_map(old, new, table, free, head, P, T)
    q, k, v = (qkv[:, i] for i in range(3))
    G.kv_append_fp8(k, v, slots, *cache)
    return G.attn_paged_fp8(q, *cache, table, lens, cu, max_q), lens, status


@pytest.mark.parametrize("P", [16, 64])
def test_chunks_and_tokens_agree(P):
    """A sequence in one chunk, and in pieces down to single tokens, over growing block scales."""
    H, DH, L = 2, 64, 150
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn((L, 3, H, DH), generator=g) * torch.exp2(torch.linspace(-3, 3, L))[:, None, None, None]
    qkv[:, 0] = torch.randn((L, H, DH), generator=g)
    qkv = qkv.to(dev()).to(F32)
    outs = []
    for sizes in ([L], [70, 1, 1, 40, 1, 37], [100] + [1] * 50):
        cache = serving.new_cache(16, H, P, DH)
        table = torch.full((1, -(-L // P)), -1, dtype=I32, device=dev())
        free = torch.randperm(16, generator=g).to(I32).to(dev())
        lens, head, at, got = torch.zeros(1, dtype=I32, device=dev()), torch.zeros(1, dtype=I32, device=dev()), 0, []
        for n in sizes:
            o, lens, status = step((lens, torch.full((1,), n, dtype=I32, device=dev()), table, free, head, n, n),
                                   cache, qkv[at:at + n], H, DH, P)
            head, at = status[:1].clone(), at + n
            assert status[1].item() == 0
            got.append(o)
        outs.append(torch.cat(got))
    x = qkv.double()
    s = torch.einsum("ihd,jhd->hij", x[:, 0], x[:, 1]) / DH ** 0.5
    s.masked_fill_(torch.ones(L, L, dtype=torch.bool, device=dev()).triu(1), float("-inf"))
    want = torch.einsum("hij,jhd->ihd", s.softmax(-1), x[:, 2])
    for o in outs:
        # 8-bit keys and values: a few per cent of the rows' size
        e = (o.double() - want).norm(dim=-1) / want.norm(dim=-1)
        assert e.max() < 0.5 and e.mean() < 0.1, (e.max(), e.mean())


def test_graph_and_stream():
    """A decode step captured once and replayed with other lengths and inputs, and the operators on
    a stream of their own, against eager results."""
    H, DH, P, R, D = 4, 64, 16, 3, 4 * 64
    g = torch.Generator().manual_seed(2)
    cache = serving.new_cache(64, H, P, DH)
    table = torch.full((R, 12), -1, dtype=I32, device=dev())
    free = torch.randperm(64, generator=g).to(I32).to(dev())
    lens = torch.zeros(R, dtype=I32, device=dev())
    head = torch.zeros(1, dtype=I32, device=dev())
    one = torch.ones(R, dtype=I32, device=dev())
    x = torch.randn((R, 3 * D), generator=g).to(dev()).to(BF)
    res = torch.randn((R, 3 * D), generator=g).to(dev()).to(BF)
    ws = torch.empty(G.attn_paged_workspace_size(R, R, 1, 12, P, H, H, DH) or 16, dtype=torch.uint8, device=dev())
    bufs = {}

    def program(st):
        y, ro = G.add_rmsnorm(st["x"], None, st["res"], out=st.get("y"), residual_out=st.get("ro"))
        q8, sc, _ = G.add_rmsnorm_fp8(y, None, group=128, q=st.get("q8"), scale=st.get("sc"))
        cu, ln, pos, slots, status = G.page_map(st["lens"], one, st["table"], free, st["head"], P, R,
                                                *(st.get(k) for k in ("cu", "ln", "pos", "slots", "status")))
        qkv = y.view(R, 3, H, DH)
        G.kv_append_fp8(qkv[:, 1], qkv[:, 2], slots, *st["cache"])
        out = G.attn_paged_fp8(qkv[:, 0], *st["cache"], st["table"], ln, cu, 1, out=st.get("out"), workspace=ws)
        st["lens"].copy_(ln)
        st["head"].copy_(status[:1])
        return {"y": y, "ro": ro, "q8": q8, "sc": sc, "cu": cu, "ln": ln, "pos": pos, "slots": slots,
                "status": status, "out": out}

    def fresh():
        return {"x": x.clone(), "res": res.clone(), "lens": lens.clone(), "head": head.clone(),
                "table": table.clone(), "cache": [t.clone() for t in cache]}

    eager, want = fresh(), []
    for i in range(20):
        eager["x"].mul_(1.25 if i % 2 else 0.7)
        want.append({k: v.clone() for k, v in program(eager).items()})
    st = fresh()
    st.update({k: torch.empty_like(v) for k, v in want[0].items()})
    warm = {k: (v if not isinstance(v, torch.Tensor) else v.clone()) for k, v in st.items()}
    warm["cache"] = [t.clone() for t in cache]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        program(warm)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert bits_equal(warm["lens"], one)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        program(st)
    for i in range(20):
        st["x"].mul_(1.25 if i % 2 else 0.7)
        for k in ("y", "out"):
            st[k].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for k in want[i]:
            assert bits_equal(st[k], want[i][k]), (i, k)


# ------------------------------------------------------------------ paths that small cases do not reach
@pytest.mark.parametrize("P", [16, 64])
def test_append_gaps_inside_long_runs(P):
    """Tokens without a slot between the tokens of one page, in runs of the workgroup's size.  Each
    page's first token has its largest values, so the scale does not depend on how a run is cut."""
    H, DH, N = 2, 128, 12
    rng = np.random.default_rng(21)
    slots = []
    for page in (4, 1, 9):
        here = list(page * P + np.arange(P))
        for at in sorted(rng.choice(np.arange(2, P), 5, replace=False))[::-1]:
            here[at:at] = [-1] * int(rng.integers(1, 4))
        slots += here + [-1] * 3
    for pad in (0, 4300):                           # short calls, and the long ones' token groups
        s = np.array([-1] * pad + slots)
        T = len(s)
        k, v = (rng.uniform(-1, 1, (T, H, DH)) for _ in range(2))
        first = [i for i in range(T) if s[i] >= 0 and s[i] % P == 0]
        k[first], v[first] = 3.0, -3.0
        k, v = tensor(k, BF), tensor(v, BF)
        cache = random_cache(N, H, P, DH, 22)
        want = host_cache(cache)
        ref.append(to_f64(k), to_f64(v), s, *want, P)
        G.kv_append_fp8(k, v, tensor(s, torch.int64), *cache)
        check_append(cache, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R", [70, 300])
def test_attn_many_requests(R, dtype):
    """More requests than a wave has lanes: decodes, chunks, idle ones and empty ones together."""
    rng = np.random.default_rng(R)
    old = rng.integers(0, 60, R)
    new = np.where(rng.random(R) < 0.1, rng.integers(2, 40, R), rng.integers(0, 2, R))
    old[R // 2], new[R // 2] = 900, 1
    old[-1], new[-1] = 150, 30
    c = attn_case(old.tolist(), new.tolist(), 4, 2, 64, 16, dtype, seed=R)
    c["lens"][3] = 0
    check_attn(c, attend(c), label=f"{R} requests")


@pytest.mark.parametrize("P,width", [(16, 16), (64, 4), (128, 1)])
def test_attn_short_tables(P, width):
    """Tables of at most four tiles: a unit per wave, no workspace."""
    c = attn_case([P * width - 3, 0, 5, 100], [3, 1, 2, 1], 6, 2, 128, P, BF, seed=30, width=width)
    assert G.attn_paged_workspace_size(4, 7, 3, width, P, 6, 2, 128) == 0
    check_attn(c, attend(c), label="short tables")


def exact_attention(c, rows):
    """torch in 64 bits on the device, for one request: out of the queries `rows`, and the sums of
    the absolute terms."""
    P, n = c["P"], int(c["lens"][0])
    pages = c["table"][0, :-(-n // P)].long()
    f = torch.float64
    k = (c["k"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).to(f) * c["ks"][pages].to(f)[..., None, None])
    v = (c["v"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).to(f) * c["vs"][pages].to(f)[..., None, None])
    k = k.permute(1, 0, 2, 3).flatten(1, 2)[:, :n]
    v = v.permute(1, 0, 3, 2).flatten(1, 2)[:, :n]
    q = c["q"].to(f)
    T, Hq, DH = q.shape
    group = Hq // k.shape[0]
    outs, mags = [], []
    for h in range(Hq):
        s = (q[rows, h] @ k[h // group].t().contiguous()) * DH ** -0.5
        pos = torch.arange(n - T, n, device=s.device)[rows]
        s.masked_fill_(torch.arange(n, device=s.device)[None] > pos[:, None], float("-inf"))
        w = s.softmax(-1)
        outs.append(w @ v[h // group])
        mags.append(w @ v[h // group].abs())
    return torch.stack(outs, 1), torch.stack(mags, 1)


def long_case(n, T, Hq, Hkv, DH, P, dtype, seed):
    """One request of n cached tokens, made on the device, with one scale for all blocks: the same
    tokens for every page size."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = (torch.randn((n, Hkv, DH), generator=g, device=dev()) * 100).clamp(-448, 448)
    v = (torch.randn((n, Hkv, DH), generator=g, device=dev()) * 100).clamp(-448, 448)
    q = torch.randn((T, Hq, DH), generator=g, device=dev()).to(dtype)
    pages = -(-n // P)
    pad = torch.full((pages * P - n, Hkv, DH), float("nan"), device=dev())
    f8 = torch.float8_e4m3fn
    k = torch.cat([k, pad]).to(f8).view(torch.uint8).view(pages, P, Hkv, DH).permute(0, 2, 1, 3).contiguous()
    v = torch.cat([v, pad]).to(f8).view(torch.uint8).view(pages, P, Hkv, DH).permute(0, 2, 3, 1).contiguous()
    order = torch.randperm(pages, generator=g, device=dev())
    one = torch.full((pages, Hkv), 2.0 ** -6, device=dev())
    return {"q": q, "k": k[order].view(f8), "v": v[order].view(f8), "ks": one, "vs": one,
            "table": torch.argsort(order).to(I32)[None], "lens": torch.tensor([n], dtype=I32, device=dev()),
            "cu": torch.tensor([0, T], dtype=I32, device=dev()), "P": P, "max_q": T, "DH": DH, "dtype": dtype}


@pytest.mark.parametrize("DH,Hq,Hkv,n,T", [(128, 8, 2, 20000, 2048), (64, 8, 4, 9001, 1500), (128, 2, 2, 40000, 3)])
def test_attn_long_pieces(DH, Hq, Hkv, n, T):
    """Pieces longer than the tables are looked ahead for; the result does not depend on the page
    size, bit for bit."""
    outs = {}
    for P in (16, 32, 64, 256):
        c = long_case(n, T, Hq, Hkv, DH, P, BF, 40)
        outs[P] = attend(c)
        if P == 16:
            rows = torch.cat([torch.arange(0, T, max(1, T // 200)), torch.tensor([T - 1])]).to(dev())
            want, mag = exact_attention(c, rows)
            # as check_attn, with the scores' error bounded by the largest |q||k| of 448 * 2^-6 * 5 * DH
            reach = 7 * 5 * DH * DH ** -0.5
            lim = mag * (2 * (DH + 8) * 2.0 ** -24 * reach + 2.0 ** -21 + n * 2.0 ** -24 + 2.0 ** -8) + 2.0 ** -8 * want.abs() * 1.01
            e = (outs[P][rows].double() - want).abs()
            log(f"  long DH={DH} n={n} T={T}: worst error / bound {(e / lim).max().item():.3f}")
            assert (e <= lim).all()
    for P in (32, 64, 256):
        assert bits_equal(outs[P], outs[16]), P


def test_graph_of_a_mixed_step():
    """Chunks and decodes in one captured call, both kernels with their joins, replayed with other
    queries and lengths between."""
    c = attn_case([3000, 40, 2500, 7], [1, 200, 2, 1], 8, 2, 128, 64, BF, seed=50)
    need = G.attn_paged_workspace_size(4, c["q"].shape[0], 200, c["table"].shape[1], 64, 8, 2, 128)
    ws = torch.empty(need, dtype=torch.uint8, device=dev())
    out = torch.empty_like(c["q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        attend(c, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attend(c, out=out, workspace=ws)
    lens = c["lens"].clone()
    for i in range(4):
        c["q"].mul_(0.9)
        c["lens"].copy_(lens - 5 * i)
        want = attend(c)
        out.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert bits_equal(out, want), i
        check_attn(c, out, label=f"replay {i}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P,DH,Hq,Hkv,most", [(64, 128, 32, 1, 1), (16, 128, 8, 1, 4), (128, 64, 10, 1, 3), (32, 64, 34, 2, 1),
                                              (64, 128, 6, 2, 10), (256, 64, 64, 2, 1), (64, 64, 8, 1, 5)])
def test_attn_some_columns(P, DH, Hq, Hkv, most, dtype):
    """Single tokens under many shared heads and a few tokens under some: 16 to 40 columns, requests
    of one tile, of no token and of many pieces."""
    old = [0, 5, 63, 64, 2000, 15, 0, 129, 640, 31]
    new = [1, most, 1, most, most, 0, 1, 1, most, max(1, most - 1)]
    c = attn_case(old, new, Hq, Hkv, DH, P, dtype, seed=P + Hq)
    c["lens"][8] = 0
    out = attend(c)
    check_attn(c, out, label=f"P={P} DH={DH} Hq={Hq}/{Hkv} x{most} {dtype}")
    assert bits_equal(out, attend(c))
    one = attn_case([6000], [most], Hq, Hkv, DH, P, dtype, seed=P)
    check_attn(one, attend(one), label="  one request")
    short = attn_case([100, 0, 7], [most, 1, most], Hq, Hkv, DH, 64, dtype, seed=P, width=3)
    check_attn(short, attend(short), label="  short tables")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [1, 5, 8, 60, 64, 65, 72, 128, 130, 192, 255, 256, 257])
def test_norm_short_rows(D, dtype):
    """Rows that share a wave: counts that leave it part empty, and rows whose squares leave fp32, of
    zeros and of NaN beside ordinary ones, which keep their bits."""
    rng = np.random.default_rng(D)
    w = tensor(1 + 0.1 * rng.standard_normal(D))
    for T in (3, 31, 77, 1000):
        x = tensor(rng.standard_normal((T, D)) * np.exp(rng.standard_normal((T, 1))), dtype)
        r = tensor(rng.standard_normal((T, D)) * 8, dtype)
        y, ro = G.add_rmsnorm(x, w, r)
        check_norm(x, r, w, 1e-6, y, ro, dtype)
        eights = {g: G.add_rmsnorm_fp8(x, w, r, group=g) for g in (0, 128)}
        for g, (q, sc, ro8) in eights.items():
            check_norm(x, r, w, 1e-6, None, ro8, dtype, q, sc, g)
        odd = x.clone()
        odd[1::5] = 1e30
        odd[2::7] = float("nan")
        same = torch.ones(T, dtype=torch.bool, device=dev())
        same[1::5] = same[2::7] = False
        y2, _ = G.add_rmsnorm(odd, w, r)
        assert bits_equal(y2[same], y[same]) and y2[2::7].isnan().all()
        huge = odd.clone()
        huge[2::7] = 0
        zero = r.clone()
        zero[2::7] = 0
        y3, ro3 = G.add_rmsnorm(huge, w, zero)
        check_norm(huge, zero, w, 1e-6, y3, ro3, dtype)
        for g, (q, sc, _) in eights.items():
            q2, sc2, _ = G.add_rmsnorm_fp8(huge, w, zero, group=g)
            assert bits_equal(q2.view(torch.uint8)[same], q.view(torch.uint8)[same]) and bits_equal(sc2[same], sc[same])
            assert (q2.view(torch.uint8)[2::7] & 0x7F == 0).all() and (sc2[2::7] == 1).all()
