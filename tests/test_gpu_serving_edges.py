"""The serving operators at the edges of what they accept, against 64-bit formulas.

Tolerances are stated with each test, before its first run."""
import os
import sys

import numpy as np
import pytest
import torch

import genomic_lm_amd as G
from tests import serving_ref as ref
from tests.gpu_util import dev, log, to_f64
from tests.test_gpu_serving import (BF, F32, I32, attend, attn_case, check_norm, codes, host_cache, random_cache,
                                    tensor)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.lib()
    yield


# ------------------------------------------------------------------ the weights of bf16 attention
# (old, new, query heads, K/V heads): requests for the kernel of few columns, and of many
COLUMNS = {"few": ([700, 130], [1, 2], 4, 2), "many": ([700, 130], [70, 33], 4, 2)}


def set_codes(t, a):
    t.view(torch.uint8).copy_(torch.from_numpy(np.ascontiguousarray(a)))


@pytest.mark.parametrize("kind", ["sharp", "flat"])
@pytest.mark.parametrize("DH,P", [(64, 16), (128, 64)])
@pytest.mark.parametrize("columns", list(COLUMNS))
def test_attn_equal_values(columns, DH, P, kind):
    """Where all values of a dimension are equal, their average is that value whatever the weights:
    the result has no rounding of its own (e4m3 values times a power of two are bf16 values), so
    weights that keep 11 bits, off by 2^-11 of their sum at most, must give it back exactly (the
    nearest bf16 values lie 2^-8 of it away, the halfway points 2^-9).  sharp: scores far apart, few
    tokens carry a row.  flat: one token above all others, which have one weight that is
    anything but a power of two, so their rounding has one sign."""
    old, new, Hq, Hkv = COLUMNS[columns]
    c = attn_case(old, new, Hq, Hkv, DH, P, BF, seed=DH)
    rng = np.random.default_rng(DH)
    row = ref.encode(rng.uniform(0.5, 2.0, (Hkv, DH, 1)))
    v = np.where(codes(c["v"]) == 0xFF, np.uint8(0xFF), row[None])
    set_codes(c["v"], v)
    c["vs"].fill_(2.0 ** -3)
    scale = 1.0
    if kind == "flat":
        k = codes(c["k"]).copy()
        k[k != 0x7F] = 0
        for r in range(2):
            k[int(c["table"][r, 0]), :, 0, 0] = 0x38        # 1.0 in the first token
        set_codes(c["k"], k)
        c["ks"].fill_(1.0)
        c["q"] = tensor(rng.uniform(0.2, 2.5, to_f64(c["q"]).shape), BF)
    out = to_f64(attend(c, scale=scale))
    want = ref.decode(row)[:, :, 0] * 2.0 ** -3
    want = np.repeat(want, Hq // Hkv, 0)[None]
    e = np.abs(out - want) / want
    log(f"  {columns} {kind} DH={DH}: {np.mean(e > 0):.4f} of the outputs off, at most {e.max():.2e}")
    assert (out == want).all()


@pytest.mark.parametrize("DH,P", [(64, 16), (128, 64), (128, 128)])
@pytest.mark.parametrize("columns", list(COLUMNS))
def test_attn_weights_keep_11_bits(columns, DH, P):
    """As test_gpu_serving's attention tolerance, with 2^-11 for the weights' rounding in the place of
    2^-8, and 2^-32 of the largest weight times its value scale for each small one (times codes
    of up to 448)."""
    old, new, Hq, Hkv = COLUMNS[columns]
    for scale in (DH ** -0.5, 0.6):
        c = attn_case(old, new, Hq, Hkv, DH, P, BF, seed=P)
        want, mag, reach = ref.attention(to_f64(c["q"]), codes(c["k"]), codes(c["v"]), to_f64(c["ks"]),
                                         to_f64(c["vs"]), c["table"].cpu().numpy(), c["lens"].cpu().numpy(),
                                         c["cu"].cpu().numpy(), scale, P)
        n = int(c["lens"].max())
        weight = 2 * (DH + 8) * 2.0 ** -24 * reach[..., None] + 2.0 ** -21 + n * 2.0 ** -24
        floor = n * 2.0 ** -32 * 448 * float(np.nanmax(to_f64(c["vs"])))
        lim = mag * (weight + 2.0 ** -11) + floor + 2.0 ** -8 * np.abs(want) * 1.01
        e = np.abs(to_f64(attend(c, scale=scale)) - want)
        log(f"  {columns} DH={DH} P={P}: worst error / bound {(e / lim).max():.3f}, "
            f"rms {np.sqrt(np.mean(e ** 2) / np.mean(want ** 2)):.2e}")
        assert (e <= lim).all()


@pytest.mark.parametrize("columns", list(COLUMNS))
def test_attn_small_weights_add_up(columns):
    """One token of value 0 in front, all others 2^-22 to 2^-20 of its weight: they alone make the result.
    Such a weight keeps 2^-32 of the largest, so at least 2^-10 of itself; 2^-11 for the largest,
    2^-8 of the value for the output's rounding, 2^-16 for scores, exponentials and sums."""
    old, new, Hq, Hkv = COLUMNS[columns]
    c = attn_case(old, new, Hq, Hkv, 64, 64, BF, seed=3)
    k, v = codes(c["k"]).copy(), codes(c["v"]).copy()
    k[k != 0x7F] = 0
    v[v != 0xFF] = 0x38
    for r in range(2):
        p = int(c["table"][r, 0])
        k[p, :, 0, 0] = 0x38
        v[p, :, :, 0] = 0
    set_codes(c["k"], k)
    set_codes(c["v"], v)
    c["ks"].fill_(1.0)
    c["vs"].fill_(1.0)
    rng = np.random.default_rng(4)
    c["q"] = tensor(rng.uniform(20 * np.log(2), 21.9 * np.log(2), to_f64(c["q"]).shape), BF)
    out = to_f64(attend(c, scale=1.0))
    cu, lens = c["cu"].cpu().numpy(), c["lens"].cpu().numpy()
    q0 = to_f64(c["q"])[:, :, 0]
    others = np.concatenate([lens[r] - (cu[r + 1] - cu[r]) + np.arange(cu[r + 1] - cu[r]) for r in range(2)])
    w = np.exp(-q0) * others[:, None]
    want = (w / (1 + w))[..., None]
    e = np.abs(out - want) / want
    log(f"  {columns}: {e.max():.2e}")
    assert (e <= 2.0 ** -10 + 2.0 ** -11 + 2.0 ** -8 + 2.0 ** -16).all()


# ------------------------------------------------------------------ lengths and positions
@pytest.mark.parametrize("Hq", [1, 40])
def test_attn_longest_table(Hq):
    """A table as long as one may be (all but 1024 of 2^31 tokens), the same page everywhere: the average
    over it is the average over one page, for one column and for as many as share tiles.  The
    sums are long: a lane adds up to 2^18 terms in fp32, each 2^-24 off at most, in the numerator and
    in the divisor."""
    P, DH = 64, 64
    width = (2 ** 31 - 1 - 1024) // P
    one = attn_case([P - 1], [1], Hq, 1, DH, P, BF, seed=5)
    p = int(one["table"][0, 0])
    want, mag, _ = ref.attention(to_f64(one["q"]), codes(one["k"]), codes(one["v"]), to_f64(one["ks"]),
                                 to_f64(one["vs"]), np.array([[p]]), [P], [0, 1], DH ** -0.5, P)
    c = dict(one)
    c["table"] = torch.full((1, width), p, dtype=I32, device=dev())
    c["lens"] = tensor(np.array([width * P]), I32)
    log(f"  {width * P} tokens, {Hq} columns")
    e = np.abs(to_f64(attend(c)) - want)
    lim = mag * (2 * 2.0 ** -6 + 2.0 ** -11) + 2.0 ** -8 * np.abs(want) * 1.01
    log(f"  worst error / bound {(e / lim).max():.3f}")
    assert (e <= lim).all()


@pytest.mark.parametrize("most", [1, 40])
def test_attn_offsets_that_descend(most):
    """Query offsets that go back below 0 give no request queries: nothing is written."""
    low = -2 ** 31
    for cu in ([3, low], [4, low, 0], [5] + [low] * 70, [1, -1], [2 ** 31 - 1, low]):
        R = len(cu) - 1
        c = attn_case([300] * R, [1] * R, 4, 2, 64, 64, BF, seed=6)
        c["q"] = c["q"][:1].expand(5, 4, 64).contiguous()
        c["cu"] = torch.tensor(cu, dtype=I32, device=dev())
        c["max_q"] = most
        if R > 1:
            c["cu"][2:] = 0                            # (a request of one's own would write its rows)
        log(f"  {cu[:4]}, up to {most} queries")
        out = torch.full_like(c["q"], 9.0)
        attend(c, out=out)
        assert (out == 9).all()


def by_formula(c, T, scale):
    """out (T, Hq, DH) and its bound, row by row from the definition: query i of request r at position
    lens[r] - (cu[r + 1] - cu[r]) + i sees the tokens up to there whose page the table holds.  For
    requests that have a query within the table."""
    q, kc, vc = to_f64(c["q"]), codes(c["k"]), codes(c["v"])
    ks, vs = to_f64(c["ks"]), to_f64(c["vs"])
    cu, lens, table, P = c["cu"].tolist(), c["lens"].tolist(), c["table"].tolist(), c["P"]
    Hq, G = q.shape[1], q.shape[1] // kc.shape[1]
    out, lim = np.zeros(q.shape), np.zeros(q.shape)
    for r in range(len(lens)):
        for t in range(cu[r], min(cu[r + 1], T)):
            pos = lens[r] - (cu[r + 1] - cu[r]) + t - cu[r]
            see = [(table[r][j // P], j % P) for j in range(pos + 1)
                   if j // P < len(table[r]) and 0 <= table[r][j // P] < len(kc)]
            if not see:
                continue
            p, o = np.array(see).T
            for h in range(Hq):
                K = ref.decode(kc[p, h // G, o]) * ks[p, h // G][:, None]
                V = ref.decode(vc[p, h // G, :, o]) * vs[p, h // G][:, None]
                s = K @ q[t, h] * scale
                w = np.exp(s - s.max())
                w /= w.sum()
                out[t, h] = w @ V
                reach = (np.abs(K) @ np.abs(q[t, h])).max() * abs(scale)
                rel = 2 * (q.shape[2] + 8) * 2.0 ** -24 * reach + 2.0 ** -21 + len(see) * 2.0 ** -24
                half, weight = (2.0 ** -8, 2.0 ** -11) if c["dtype"] == BF else (2.0 ** -24, 2.0 ** -22)
                floor = len(see) * 2.0 ** -32 * 448 * vs[p].max() if c["dtype"] == BF else 0.0
                lim[t, h] = w @ np.abs(V) * (rel + weight) + floor + half * np.abs(out[t, h]) * 1.01
    return out, lim


def check_formula(c, T, label):
    q = c["q"]
    want, lim = by_formula(c, T, c["DH"] ** -0.5)
    c = dict(c, q=q[:T].contiguous())
    out = to_f64(attend(c))
    e = np.abs(out - want[:T])
    log(f"  {label} {c['dtype']}: worst error / bound {(e / np.maximum(lim[:T], 1e-300)).max():.3f}")
    assert np.isfinite(out).all() and (e <= lim[:T] + 1e-30).all()


# (old, new, T): the last request that has rows is cut by T
CUT = {"few": ([90, 200, 30], [2, 4, 3], 4), "many": ([90, 200, 30], [20, 60, 5], 47),
       "one": ([100], [90], 50), "requests": ([40] * 70, [1] * 60 + [30] * 10, 75)}


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", list(CUT))
def test_attn_fewer_rows_than_queries(kind, dtype):
    """T below cu[R], as after a page map with a fixed T: the queries that have rows keep their
    positions, and the tokens of the others, which got places but were never appended, are not read
    (their places hold NaN codes).  Tolerance: as the attention's with 11-bit weights."""
    old, new, T = CUT[kind]
    for P, DH, Hq, Hkv in ((16, 64, 4, 2), (64, 128, 2, 1)):
        c = attn_case(old, new, Hq, Hkv, DH, P, dtype, seed=7)
        k, v = codes(c["k"]).copy(), codes(c["v"]).copy()
        cu, table = c["cu"].tolist(), c["table"].tolist()
        for r in range(len(old)):
            for t in range(max(cu[r], T), cu[r + 1]):
                page, at = divmod(old[r] + t - cu[r], P)
                k[table[r][page], :, at] = 0x7F
                v[table[r][page], :, :, at] = 0x7F
        set_codes(c["k"], k)
        set_codes(c["v"], v)
        check_formula(c, T, f"{kind} P={P}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new", [2, 7, 40])
def test_attn_chunk_past_the_table(new, dtype):
    """A chunk that begins in its table and ends past it: its tokens in the table are seen where they
    stand, the others are not there."""
    for P, DH, Hq, Hkv, width in ((16, 64, 4, 2, 3), (64, 128, 2, 1, 2), (64, 64, 4, 1, 8)):
        cap = P * width
        c = attn_case([cap - 1, 5, cap - max(new // 2, 1)], [new, 1, new], Hq, Hkv, DH, P, dtype, seed=8)
        c["table"] = c["table"][:, :width].contiguous()
        check_formula(c, c["q"].shape[0], f"{new} new, table of {cap}")


# ------------------------------------------------------------------ norm
def check_norms(x, r, w, eps, dtype):
    """All three outputs, with the tolerances of test_gpu_serving."""
    y, ro = G.add_rmsnorm(x, w, r, eps=eps)
    check_norm(x, r, w, eps, y, ro, dtype)
    for group in (0, 128):
        q, sc, ro = G.add_rmsnorm_fp8(x, w, r, eps=eps, group=group)
        check_norm(x, r, w, eps, None, ro, dtype, q, sc, group)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [8, 64, 200, 512, 1000, 2048, 4096, 8192, 32768])
def test_norm_largest_rows(D, dtype):
    """Finite rows up to the type's largest value, with and without a residual, and an eps that counts
    beside them; an infinity by the formula: NaN in its column, 0 in the others."""
    rng = np.random.default_rng(D)
    sign = rng.choice([-1.0, 1.0], (6, D))
    size = np.array([1e18, 1e19, 1e36, 1e37, 1e38, 3.3e38])[:, None]
    x = tensor(sign * size * rng.uniform(0.25, 1.0, (6, D)), dtype)
    w = tensor(1 + 0.1 * rng.standard_normal(D))
    for eps in (1e-6, 3e38):
        check_norms(x, None, w, eps, dtype)
        check_norms(x[:5], x[:5].roll(1, 1), w, eps, dtype)
    check_norms(tensor(rng.standard_normal((3, D)), dtype), None, None, 3.4e38, dtype)
    x = tensor(rng.standard_normal((3, D)), dtype)
    x[1, D // 2] = float("inf")
    y, _ = G.add_rmsnorm(x, w)
    want = torch.zeros(D, device=dev())
    want[D // 2] = float("nan")
    assert torch.equal(y[1].isnan(), want.isnan()) and (y[1].nan_to_num() == 0).all()
    assert torch.isfinite(y[[0, 2]].float()).all()
    q, sc, _ = G.add_rmsnorm_fp8(x, w, group=128)
    c = codes(q)[1] & 0x7F
    assert c[D // 2] == 0x7F and (np.delete(c, D // 2) == 0).all() and (sc[1] == 1).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [1, 8, 64, 200, 512, 1000, 2048, 4096, 8192, 32768])
def test_norm_smallest_rows(D, dtype):
    """Rows whose squares fall out of fp32's range, down to its smallest values, with no eps or one
    that does not cover them, beside rows that are not small; and with one that does."""
    rng = np.random.default_rng(D)
    sign = rng.choice([-1.0, 1.0], (9, D))
    size = np.array([1.0, 1e-12, 1e-17, 1e-19, 1e-23, 1e-30, 1e-37, 1e-40, 2.0 ** -133])[:, None]
    x = tensor(sign * size * rng.uniform(0.6, 1.0, (9, D)), dtype)
    assert (x != 0).all()
    w = tensor(1 + 0.1 * rng.standard_normal(D))
    for eps in (0.0, 1e-45, 1e-38, 1e-30):
        eps = float(np.float32(eps))
        check_norms(x, None, w, eps, dtype)
        check_norms(x, x.clone(), None, eps, dtype)
    check_norms(x[:6], None, w, 1e-6, dtype)


@pytest.mark.parametrize("D", [64, 256, 1001])
def test_norm_codes_of_subnormal_values(D):
    """Weights that make y a number below fp32's normal range, down to its smallest: codes are numbers,
    and code * scale is y within e4m3's rounding (2^-4 of the value, half a subnormal step: 2^-10 of the
    scale) and fp32's there (2^-149, twice: y and the scale times 448)."""
    rng = np.random.default_rng(D)
    x = tensor(rng.standard_normal((4, D)), F32)
    for size in (1.4e-45, 1e-44, 1e-43, 3e-43, 9e-43, 4e-42, 1e-40, 1e-38):
        w = tensor(size * rng.uniform(0.5, 2.0, D))
        _, want = ref.rmsnorm(to_f64(x), None, to_f64(w), 1e-6)
        for group in (0, 128):
            q, sc, _ = G.add_rmsnorm_fp8(x, w, eps=1e-6, group=group)
            c, s = ref.decode(codes(q)), np.repeat(to_f64(sc).reshape(4, -1), group or D, 1)[:, :D]
            assert np.isfinite(c).all() and (s >= 2.0 ** -140).all(), size
            e = np.abs(c * s - want)
            lim = 2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -8) + 2.0 ** -10 * s + 2 * 2.0 ** -149
            assert (e <= lim).all(), (size, (e / lim).max())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_rows_of_single_axes(dtype):
    """Rows at one stride under axes of size one: the last token of each sequence, in and out."""
    x = torch.randn((3, 7, 40), device=dev()).to(dtype)
    want, _ = G.add_rmsnorm(x[:, -1].contiguous())
    whole = torch.full_like(x, 9.0)
    for a, b in ((x[:, -1:], whole[:, 2:3]), (x[:, -1:, None], whole[:, 3:4, None]), (x[None, :, None, -1], None)):
        y, _ = G.add_rmsnorm(a, out=b)
        assert y.shape == a.shape and torch.equal(y.reshape(3, 40), want)
    assert (whole[:, [0, 1, 4, 5, 6]] == 9).all()
    y, _ = G.add_rmsnorm(x[1:2, 3:4, 5:30])
    assert torch.equal(y, G.add_rmsnorm(x[1:2, 3:4, 5:30].contiguous())[0])
    with pytest.raises(ValueError):
        G.add_rmsnorm(x[:, 1:3])


# ------------------------------------------------------------------ append
def append_by_page(k, v, slots, kc, vc, ks, vs, P):
    """The header's formulas page by page, over all tokens of the call that a page takes, wherever they
    stand in it and in whatever order; codes and scales are changed in place."""
    pages = {}
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < len(kc) * P:
            pages.setdefault(s // P, []).append((t, s % P))
    for page, tokens in pages.items():
        t, o = np.array(tokens).T
        low = o.min()
        for h in range(k.shape[1]):
            a, b = k[t, h], v[t, h]
            for x, c, sc in ((a, kc[page, h], ks), (b, vc[page, h].T, vs)):
                scale = ref.block_scale(np.abs(x).max())
                if low > 0:
                    scale = max(scale, sc[page, h])
                    c[:low] = ref.encode(ref.decode(c[:low]) * (sc[page, h] / scale))
                sc[page, h] = scale
                c[o] = ref.encode(x / scale)


def check_pages(slots, N, H, P, DH, dtype, seed, big=()):
    """big: tokens whose values are larger than all others'."""
    rng = np.random.default_rng(seed)
    T = len(slots)
    k, v = (rng.uniform(-1, 1, (T, H, DH)) for _ in range(2))
    for t in big:
        k[t], v[t] = k[t] * 40, v[t] * 90
    k, v = tensor(k, dtype), tensor(v, dtype)
    cache = random_cache(N, H, P, DH, seed)
    for sc in cache[2:]:
        sc[: N // 2] = float("nan")                # of pages never written: not read by a fresh block
    want = host_cache(cache)
    append_by_page(to_f64(k), to_f64(v), slots, *want, P)
    G.kv_append_fp8(k, v, tensor(slots, torch.int64), *cache)
    used = np.unique(slots[(slots >= 0) & (slots < N * P)] // P)
    for name, g, w in zip(("k_cache", "v_cache", "k_scale", "v_scale"), host_cache(cache), want):
        for page in used:
            assert (g[page] == w[page]).all(), (name, int(page), int((g[page] != w[page]).sum()))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [0, 4300])
@pytest.mark.parametrize("P,DH", [(16, 64), (64, 128), (256, 64)])
def test_append_places_in_any_order(P, DH, pad, dtype):
    """A page's places from the last to the first, shuffled, and with place 0 in the middle, in fresh
    pages (whose scales hold NaN) and in pages with older tokens, in runs of a wave's and of the
    workgroup's size.  Exact."""
    rng = np.random.default_rng(P + pad)
    N = 16
    old = N // 2                                   # pages from here on have a scale
    n = min(P, 70)
    here = [np.array([1, 0]), np.array([2, 0, 1]), np.arange(4)[::-1], rng.permutation(n), np.arange(n)[::-1],
            np.concatenate([np.arange(5, n), np.arange(5)])]
    late = [np.array([P - 1, P - 2]), 3 + rng.permutation(4), P - 1 - np.arange(min(P - 5, 66)),
            5 + rng.permutation(P - 5)[:60]]
    slots = np.concatenate([np.full(pad, -1)] + [i * P + o for i, o in enumerate(here)] +
                           [(old + i) * P + o for i, o in enumerate(late)]).astype(np.int64)
    big = rng.choice(np.arange(pad, len(slots)), 12, replace=False)
    check_pages(slots, N, 2, P, DH, dtype, P, big)


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("gap", [1, 3, 32, 61, 62])
def test_append_largest_value_after_a_gap(gap, long):
    """Up to 62 tokens without a slot between two of one page, at every position against the 64 tokens
    that are looked at together: one scale for all of the page's tokens, taken from the last of them, in
    fresh pages and behind older tokens.  Exact."""
    H, DH, P, N = 1, 64, 64, 40
    rng = np.random.default_rng(gap)
    none = [-1, -7, N * P, 1 << 40]
    slots, big, fresh, held = [-1] * (4200 if long else 0), [], iter(range(N // 2)), iter(range(N // 2, N))
    for i in range(36):
        page, o = (next(fresh), 0) if i % 2 else (next(held), int(rng.integers(1, 20)))
        before, after = (1, 1) if i < 12 else (int(rng.integers(1, 22)), int(rng.integers(1, 22)))
        for at in range(before + after):
            if at == before or (i >= 24 and at and rng.random() < 0.2):
                slots += [none[int(x)] for x in rng.integers(0, 4, gap if at == before else 2)]
            slots.append(page * P + o + at)
        big.append(len(slots) - 1)
        slots += [-1] * int(rng.integers(0, 9))
    check_pages(np.array(slots, dtype=np.int64), N, H, P, DH, BF, gap, big)


# ------------------------------------------------------------------ page map
@pytest.mark.parametrize("R", [1, 5, 300])
def test_page_map_after_a_shortage(R):
    """Steps that go on after the free list ran out: status counts every new token whose slot is -1, those
    in a part-filled page that the earlier step did not get among them.  Exact."""
    rng = np.random.default_rng(R)
    P, width = 16, 8
    i32 = lambda a: tensor(np.array(a), I32)  # noqa: E731
    table = torch.full((R, width), -1, dtype=I32, device=dev())
    lens = torch.zeros(R, dtype=I32, device=dev())
    free, head = i32(rng.permutation(3 * R)), i32([0])
    lost = 0
    for step in range(14):
        new = rng.integers(0, 25 if step < 4 else 4, R)
        new[0] = 9
        T = int(new.sum())
        cu, after, pos, slots, status = G.page_map(lens, i32(new), table, free, head, P, T)
        want = np.full(T, -1)
        t = 0
        rows = table.cpu().numpy()
        for r in range(R):
            for p in range(int(lens[r]), int(after[r])):
                if p // P < width and rows[r, p // P] >= 0:
                    want[t] = rows[r, p // P] * P + p % P
                t += 1
        assert (slots.cpu().numpy() == want).all(), step
        assert status.tolist() == [min(3 * R, int(status[0])), int((want < 0).sum())], step
        lost += int(status[1])
        lens, head = after, status[:1].clone()
    assert lost > 0


# ------------------------------------------------------------------ example
@pytest.mark.parametrize("args", [["--prompts", "1", "1", "--steps", "3", "--page", "64"],
                                  ["--prompts", "40", "9", "--steps", "24", "--page", "64"],
                                  ["--prompts", "29", "9", "--steps", "2", "--page", "16"]])
def test_example_places_every_token(args, monkeypatch):
    """The serving example at lengths that end with a page, and with prompts shorter than one: no step
    leaves a token without a page."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    monkeypatch.syspath_prepend(os.path.join(root, "examples"))
    import striped_serving
    seen, page_map = [], G.page_map

    def watched(*a):
        out = page_map(*a)
        seen.append(out[4])
        return out

    monkeypatch.setattr(striped_serving.G, "page_map", watched)
    far, finite = striped_serving.main(["--dim", "256", "--heads", "4", "--chunk", "48", *args])
    assert finite and max(far) < 0.05, far
    assert seen and not torch.stack(seen)[:, 1].any()
