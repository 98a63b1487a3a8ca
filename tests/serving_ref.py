"""Plain 64-bit implementations of the serving operators, for their tests.

Written from the formulas in include/hyena.h with numpy loops; they share no
code with the kernels.  e4m3 codes are read through a table built from the
format's definition and rounded by nearest-value search (ties to the even
code)."""
from __future__ import annotations

import numpy as np

FP8_MAX = 448.0
MIN_SCALE = 2.0 ** -96


def _table():
    """Values of the 128 non-negative codes: 4 exponent bits (bias 7), 3 mantissa bits."""
    v = np.empty(128)
    for c in range(128):
        e, m = c >> 3, c & 7
        v[c] = np.nan if c == 127 else (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return v


POS = _table()
VALUES = np.concatenate([POS, -POS])          # code -> value (0x80: -0)


def decode(codes):
    return VALUES[np.asarray(codes, dtype=np.uint8)]


def encode(x):
    """Nearest e4m3 code of each x, |x| <= 464; ties to the even code; NaN -> a NaN code."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    grid = POS[:127]
    hi = np.clip(np.searchsorted(grid, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - grid[lo], grid[hi] - a
    near = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    near = np.where(a >= grid[126], 126, near)
    code = near.astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def rmsnorm(x, r, w, eps):
    s = x + (0.0 if r is None else r)
    top = np.maximum(np.max(np.abs(s), axis=-1, keepdims=True), 1e-300)
    with np.errstate(invalid="ignore", over="ignore"):
        z = s / top
        y = z / np.sqrt(np.mean(z * z, axis=-1, keepdims=True) + eps / top / top)
    return s, y if w is None else y * w


def page_map(old, new, table, free, head, P, T):
    """The step's tables by walking the requests; table is changed."""
    R, width = table.shape
    cu, lens, pos, slots = [0], [], [], []
    at, lost = head, 0
    for r in range(R):
        o, n = max(int(old[r]), 0), max(int(new[r]), 0)
        have, want = min(-(-o // P), width), min(-(-(o + n) // P), width)
        for j in range(have, want):
            if at < len(free):
                table[r, j] = free[at]
            at += 1
        got = min(max(len(free) - (at - (want - have)), 0), want - have)
        lost += max(0, o + n - max(o, (have + got) * P))
        for i in range(n):
            p = o + i
            j = p // P
            ok = j < have + got and table[r, j] >= 0
            pos.append(p)
            slots.append(int(table[r, j]) * P + p % P if ok else -1)
        cu.append(cu[-1] + n)
        lens.append(o + n)
    pad = T - len(pos)
    pos, slots = pos[:T] + [-1] * max(pad, 0), slots[:T] + [-1] * max(pad, 0)
    return (np.array(cu), np.array(lens, dtype=np.int64), np.array(pos, dtype=np.int64),
            np.array(slots, dtype=np.int64), np.array([max(min(at, len(free)), head), lost]))


def block_scale(top):
    """The smallest power of two s with top / s <= 448, by search over exponents."""
    if top <= 0:
        return MIN_SCALE
    e = int(np.floor(np.log2(top))) - 12
    while top / 2.0 ** e > FP8_MAX:
        e += 1
    return max(2.0 ** e, MIN_SCALE)


def append(k, v, slots, kc, vc, ks, vs, P):
    """Codes (uint8) and scales changed in place; k, v (T, H, DH) in 64 bits."""
    T, H, DH = k.shape
    N = kc.shape[0]
    t = 0
    while t < T:
        s = int(slots[t])
        if s < 0 or s >= N * P:
            t += 1
            continue
        page, o = divmod(s, P)
        n = 1
        while o + n < P and t + n < T and slots[t + n] == s + n:
            n += 1
        for h in range(H):
            a, b = k[t:t + n, h], v[t:t + n, h]
            poison = ~(np.isfinite(a).all(-1) & np.isfinite(b).all(-1))
            for x, c, sc in ((a, kc[page, h], ks), (b, vc[page, h].T, vs)):
                fin = np.abs(x[np.isfinite(x)])
                scale = block_scale(fin.max() if fin.size else 0.0)
                if o:
                    if scale > sc[page, h]:
                        c[:o] = encode(decode(c[:o]) * (sc[page, h] / scale))
                    else:
                        scale = sc[page, h]
                sc[page, h] = scale
                code = encode(np.where(np.isfinite(x), x, 0.0) / scale)
                if sc is ks:
                    code[poison] = 0x7F
                c[o:o + n] = code
        t += n


def attention(q, kc, vc, ks, vs, table, lens, cu, scale, P, max_q=None):
    """(out, bound): bound[t, h, d] = sum_j p_j |v_j|, the scale of the weights' rounding, and
    the largest sum |q||k| scale over the seen tokens per row.  Unwritten rows are NaN."""
    T, Hq, DH = q.shape
    N, Hkv = kc.shape[:2]
    G = Hq // Hkv
    out = np.full(q.shape, np.nan)
    mag = np.zeros(q.shape)
    reach = np.zeros((T, Hq))
    width = table.shape[1]
    for r in range(len(lens)):
        c0, c1 = max(int(cu[r]), 0), min(int(cu[r + 1]), T)
        nq = c1 - c0 if max_q is None else min(c1 - c0, max_q)
        n = min(max(int(lens[r]), 0), width * P)
        for h in range(Hkv):
            j = np.arange(n)
            pages = table[r, j // P].astype(np.int64)
            ok = (pages >= 0) & (pages < N)
            pages = np.where(ok, pages, 0)
            K = decode(kc[pages, h, j % P]) * ks[pages, h][:, None]
            V = decode(vc[pages, h, :, j % P]) * vs[pages, h][:, None]
            for i in range(nq):
                pos = n - nq + i if max_q is None else n - (c1 - c0) + i
                see = ok & (np.arange(n) <= pos)
                for g in range(G):
                    qq = q[c0 + i, h * G + g]
                    if not see.any():
                        out[c0 + i, h * G + g] = 0.0
                        continue
                    s = K[see] @ qq * scale
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[c0 + i, h * G + g] = w @ V[see]
                    mag[c0 + i, h * G + g] = w @ np.abs(V[see])
                    reach[c0 + i, h * G + g] = (np.abs(K[see]) @ np.abs(qq)).max() * abs(scale)
    return out, mag, reach
