"""The 8-bit projections, the quantisation of their operands and the rotary positions against plain
64-bit implementations (projection_ref.py).

Tolerances, stated before any run:
* product: with A = sum |x| |w| (scales included) behind an element.  A product of two codes has 8 bits.
  The sum of a run's 128 may round at every addition, toward zero too: 128 * 2^-23 of the
  run's magnitudes; the two scales' product, its product with the sum and the sums over the b runs (and over up
  to 16 waves' parts) (b + 20) * 2^-24: (b + 276) 2^-24 A.  The output adds half a unit in the last place, at
  most 2^-p of the value for p significant bits: 2^-8 in bf16, 2^-24 in fp32.  With a bf16 output the matrix
  unit adds the codes' products in groups of eight columns, each product cut below 2^-13 of the group's largest
  (2^16 + 2^2 in one group gives 2^16): eight cuts a group, 2^-10 of its largest product, 2^-10 A in all.
* gated: h = act(g) u with errors dg, du as above; no activation is steeper than 1.13.  The gelu's argument
  g / sqrt 2 is off by 2^-23 of itself, which moves erfc by (g^2 + 2) 2^-23 of its value where g < 0, the
  exponentials' arguments z by 4 * 2^-24 |z|, with 16 * 2^-24 for the functions and the products:
  |u| 1.13 dg + |act(g)| du + (16 + 2 g^2 + 4 |z|) 2^-24 |h| + dg du.
* codes: their scale has the error of the largest |h| of its run and 2^-22, a code half a step: 2^-4 of
  the value or 2^-10 of the scale.
* quantisation: scale 2^-23 of itself (one division); codes as above, z = x * (1 / scale) two roundings.
* rotation: the fraction of a turn is rounded to 2^-26 turns at most (it is below half a turn),
  2 pi 2^-26 < 2^-23 of angle, sine and cosine 2 units in the last place: below 2^-21 of |a| + |b|; a norm
  of up to 256 columns adds 2^-19 (64 terms per lane and a tree of 6, halved by the root, and 8 more)."""
import math

import numpy as np
import pytest
import torch

import genomic_lm_amd as G
from tests import projection_ref as ref
from tests.gpu_util import dev, to_f64
from tests.serving_ref import decode

pytestmark = pytest.mark.gpu

BF, F32, F8, U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.lib()
    yield


def put(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(dev())


def raw(t):
    return t.contiguous().view(U8).cpu().numpy()


def bits_equal(a, b):
    if a.shape != b.shape or not a.numel():
        return a.shape == b.shape
    return torch.equal(a.contiguous().view(-1).view(U8), b.contiguous().view(-1).view(U8))


def codes(rng, *shape):
    """Any finite code."""
    c = rng.integers(0, 256, shape).astype(np.uint8)
    return np.where(c & 0x7F == 0x7F, np.uint8(0x3A), c)


def f32(a):
    return np.asarray(a, dtype=np.float32)


def operands(rng, T, K, N, group, weights=1):
    runs = -(-K // 128)
    x = codes(rng, T, K)
    xs = f32(np.exp(rng.normal(size=(T, runs) if group else (T,))))
    ws = [(codes(rng, N, K), f32(np.exp(rng.normal(size=(-(-N // 128), runs))) / 64)) for _ in range(weights)]
    return x, xs, ws


def to_gpu(x, xs, ws):
    return (put(x, U8), put(xs), *(put(a, t) for w, s in ws for a, t in ((w, U8), (s, F32))))


def sum_error(K, size, dtype):
    return ((-(-K // 128) + 276) * 2.0 ** -24 + (2.0 ** -10 if dtype == BF else 0)) * size


def half(dtype):
    return 2.0 ** -8 if dtype == BF else 2.0 ** -24


SHAPES = [  # T, K, N: few rows, tiles of every kind, odd and ragged sizes
    (1, 128, 16), (1, 1, 1), (1, 4096, 384), (2, 100, 7), (5, 1001, 130), (16, 384, 300), (16, 2000, 64),
    (17, 128, 128), (33, 1000, 257), (64, 640, 640), (100, 17, 1000), (128, 256, 129), (130, 1001, 520),
    (257, 129, 257), (300, 2064, 388), (600, 256, 1100), (1025, 384, 771), (2100, 272, 520)]


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("group,dtype,bias", [(0, BF, False), (128, BF, True), (128, F32, False), (0, F32, True)])
def test_linear(T, K, N, group, dtype, bias):
    rng = np.random.default_rng(T * 7 + K * 3 + N)
    x, xs, ws = operands(rng, T, K, N, group)
    b = f32(rng.normal(size=N)) if bias else None
    y = G.linear_fp8(*to_gpu(x, xs, ws), bias=None if b is None else put(b), dtype=dtype)
    assert y.shape == (T, N) and y.dtype == dtype
    want, size = ref.product(x, xs, *ws[0])
    if bias:
        want, size = want + b.astype(np.float64), size + np.abs(b)
    e = np.abs(to_f64(y) - want)
    tol = sum_error(K, size, dtype)
    assert (e <= tol + half(dtype) * (np.abs(want) + tol)).all(), (e - tol).max()


@pytest.mark.parametrize("T,K,N", [
    (2100, 128, 3700), (2100, 272, 3700), (2100, 400, 3800), (2060, 112, 3800),    # the largest tiles, one to four runs
    (2100, 272, 2100), (700, 1040, 2000), (700, 1024, 2000), (130, 1168, 520), (40, 528, 640),          # shared K
    (1500, 272, 100), (500, 528, 250), (300, 145, 100)])                             # many rows of few outputs
@pytest.mark.parametrize("group,dtype", [(128, BF), (0, F32)])
def test_linear_tiles(T, K, N, group, dtype):
    rng = np.random.default_rng(T + K + N)
    x, xs, ws = operands(rng, T, K, N, group)
    y = G.linear_fp8(*to_gpu(x, xs, ws), dtype=dtype)
    want, size = ref.product(x, xs, *ws[0])
    tol = sum_error(K, size, dtype)
    e = np.abs(to_f64(y) - want)
    assert (e <= tol + half(dtype) * (np.abs(want) + tol)).all(), (e - tol).max()


def check_gated(x, xs, ws, act, got, dtype):
    K = x.shape[1]
    g, gsize = ref.product(x, xs, *ws[0])
    u, usize = ref.product(x, xs, *ws[1])
    a = ref.act(g, act)
    want = a * u
    dg, du = sum_error(K, gsize, dtype), sum_error(K, usize, dtype)
    z = np.abs(g) if act == "silu" else 1.6 * (np.abs(g) + 0.0447 * np.abs(g) ** 3) if act == "gelu_tanh" else 0 * g
    # 2 g^2 and 4 |z| reach past 1 only where the activation itself is below fp32's range
    rel = np.minimum((16 + 2 * g * g * (act == "gelu") + 4 * z) * 2.0 ** -24, 1.0)
    tol = np.abs(u) * 1.13 * dg + np.abs(a) * du + dg * du * 1.13 + rel * np.abs(want) + 2.0 ** -126 * (1 + np.abs(u))
    if dtype is not None:
        e = np.abs(to_f64(got) - want)
        assert (e <= tol + half(dtype) * (np.abs(want) + tol)).all(), (e - tol).max()
        return
    q, scale = got
    T, N = want.shape
    c, sc = decode(raw(q)), to_f64(scale)
    assert c.shape == want.shape and sc.shape == (T, -(-N // 128))
    for i in range(sc.shape[1]):
        run = slice(i * 128, (i + 1) * 128)
        top, t = np.abs(want[:, run]).max(1), tol[:, run].max(1)
        # a run of values below fp32's range (2^-149; the gelu of -18 is 2^-240) is a run of zeros there, scale 1
        lost = (top < 2.0 ** -120) & (sc[:, i] == 1)
        off = np.abs(sc[:, i] - np.where(top > 0, np.maximum(top / 448, 2.0 ** -140), 1.0))
        assert (lost | (off <= (t + 2.0 ** -22 * top) / 448)).all()
        e = np.abs(c[:, run] * sc[:, i:i + 1] - want[:, run])
        step = np.maximum(2.0 ** -4 * np.abs(want[:, run]), 2.0 ** -10 * sc[:, i:i + 1])
        assert (e <= (step + tol[:, run]) * (1 + 2.0 ** -20) + 2.0 ** -4 * tol[:, run]).all(), i


@pytest.mark.parametrize("T,K,N", [(1, 128, 128), (1, 1, 1), (3, 1001, 200), (16, 512, 384), (17, 200, 129),
                                   (64, 384, 256), (130, 1000, 300), (300, 272, 1100), (1030, 256, 520)])
@pytest.mark.parametrize("act,dtype,group", [("gelu", None, 128), ("silu", BF, 0), ("gelu_tanh", F32, 128),
                                             ("none", None, 0), ("silu", None, 128), ("gelu", F32, 0)])
def test_gated(T, K, N, act, dtype, group):
    rng = np.random.default_rng(T + 5 * K + N)
    x, xs, ws = operands(rng, T, K, N, group, 2)
    # sums of a few units: the activations' bends
    xs = xs / f32(60 * math.sqrt(K))
    got = G.gated_linear_fp8(*to_gpu(x, xs, ws), act=act, dtype=dtype or F8)
    check_gated(x, xs, ws, act, got, dtype)


@pytest.mark.parametrize("T,K,N,act,dtype", [
    (2100, 400, 1900, "none", BF), (2100, 272, 1900, "silu", F32), (5200, 144, 2500, "gelu", None), (5200, 145, 2500, "silu", None),
    (1500, 272, 100, "silu", BF), (300, 145, 100, "gelu", None), (700, 1040, 1000, "gelu", BF), (700, 1040, 1000, "gelu", None), (2000, 128, 1100, "silu", BF)])
def test_gated_tiles(T, K, N, act, dtype):
    rng = np.random.default_rng(T + K + N)
    x, xs, ws = operands(rng, T, K, N, 128, 2)
    xs = xs / f32(60 * math.sqrt(K))
    check_gated(x, xs, ws, act, G.gated_linear_fp8(*to_gpu(x, xs, ws), act=act, dtype=dtype or F8), dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_columns_of_two_launches(dtype):
    """A little more than a round of the largest tiles: the last columns take a launch of their own."""
    rng = np.random.default_rng(17)
    x, xs, ws = operands(rng, 4200, 144, 4100, 128)
    b = f32(rng.normal(size=4100) * 100)
    y = torch.full((4200, 4104), 7.0, dtype=dtype, device=dev())
    G.linear_fp8(*to_gpu(x, xs, ws), bias=put(b), out=y[:, :4100])
    assert (y[:, 4100:] == 7).all()
    want, size = ref.product(x, xs, *ws[0])
    want, tol = want + b.astype(np.float64), sum_error(144, size + np.abs(b), dtype)
    e = np.abs(to_f64(y[:, :4100]) - want)
    assert (e <= tol + half(dtype) * (np.abs(want) + tol)).all(), (e - tol).max()
    x, xs, ws = operands(rng, 2100, 144, 3700, 128, 2)
    xs = xs / f32(60 * 12)
    check_gated(x, xs, ws, "gelu", G.gated_linear_fp8(*to_gpu(x, xs, ws), dtype=dtype), dtype)


@pytest.mark.parametrize("T,K,N", [(1, 256, 200), (70, 301, 130), (600, 144, 300)])
def test_gated_codes_by_way_of_a_workspace(T, K, N):
    """Whatever the workspace holds, and nothing behind the bytes that the size function names."""
    rng = np.random.default_rng(T)
    x, xs, ws = operands(rng, T, K, N, 128, 2)
    args = to_gpu(x, xs / f32(60 * math.sqrt(K)), ws)
    need = G.gated_linear_fp8_workspace_size(T, N, K)
    assert need == 4 * T * N
    want = G.gated_linear_fp8(*args, dtype=F8)
    for fill in (0x00, 0xFF, 0x7F):
        buf = torch.full((need + 64,), fill, dtype=U8, device=dev())
        got = G.gated_linear_fp8(*args, dtype=F8, workspace=buf[:need])
        assert bits_equal(got[0], want[0]) and bits_equal(got[1], want[1])
        assert (buf[need:] == fill).all()
    with pytest.raises(RuntimeError):
        G.gated_linear_fp8(*args, dtype=F8, workspace=buf[:need - 4])
    with pytest.raises(ValueError):
        G.gated_linear_fp8(*args, dtype=F8, workspace=buf[:need].cpu())
    with pytest.raises(ValueError):
        G.gated_linear_fp8(*args, dtype=F8, workspace=torch.empty(2 * need, dtype=U8, device=dev())[::2])
    # the codes of the fp32 product, as quantize_fp8 makes them
    h = G.gated_linear_fp8(*args, dtype=F32)
    q, scale = G.quantize_fp8(h, 128)
    assert bits_equal(q, want[0]) and bits_equal(scale, want[1])


@pytest.mark.parametrize("T,K,at", [(3, 300, 5), (40, 300, 5), (600, 300, 5), (40, 304, 16), (200, 304, 16),
                                    (1300, 304, 16)])
def test_strided_operands(T, K, at):
    """Rows of x, of its scales and of y at strides of their own; a single token of a batch."""
    rng = np.random.default_rng(T)
    N = 200
    x, xs, ws = operands(rng, T, K, N, 128)
    gx, gxs, gw, gws = to_gpu(x, xs, ws)
    want = G.linear_fp8(gx, gxs, gw, gws)
    wide = torch.zeros((T, K + (13 if at == 5 else 32)), dtype=U8, device=dev())
    wide[:, at:at + K] = gx
    scales = torch.zeros((T, 7), device=dev())
    scales[:, 2:5] = gxs
    buf = torch.full((T, N + 9), 7.0, dtype=BF, device=dev())
    G.linear_fp8(wide[:, at:at + K], scales[:, 2:5], gw, gws, out=buf[:, 3:3 + N])
    assert bits_equal(buf[:, 3:3 + N], want)
    assert (buf[:, :3] == 7).all() and (buf[:, 3 + N:] == 7).all()
    # one token of each sequence, one scale per row
    seq = gx[None].expand(2, T, K).contiguous()
    rows = torch.rand((2, T), device=dev())
    got = G.linear_fp8(seq[:, -1:], rows[:, -1:], gw, gws)
    assert got.shape == (2, 1, N)
    assert bits_equal(got[:, 0], G.linear_fp8(seq[:, -1].contiguous(), rows[:, -1].contiguous(), gw, gws))
    # the same row for every token
    one = G.linear_fp8(gx[:1].expand(T, K), gxs[:1].expand(T, 3), gw, gws)
    first = to_f64(one[:1])
    assert (np.abs(to_f64(one) - first) <= 2.0 ** -7 * np.abs(first) + 1e-30).all()


def test_float8_and_uint8_are_the_same_codes():
    rng = np.random.default_rng(0)
    x, xs, ws = operands(rng, 40, 256, 256, 128, 2)
    a = to_gpu(x, xs, ws)
    f = [t.view(F8) if t.dtype == U8 else t for t in a]
    assert bits_equal(G.linear_fp8(*a[:4]), G.linear_fp8(*f[:4]))
    q, s = G.gated_linear_fp8(*f, dtype=F8)
    r, t = G.gated_linear_fp8(*a, dtype=U8)
    assert q.dtype == F8 and r.dtype == U8 and bits_equal(q, r) and bits_equal(s, t)


@pytest.mark.parametrize("T", [2, 100, 700])
def test_nan_stays_in_its_row_or_column(T):
    rng = np.random.default_rng(T)
    K, N = 200, 300
    x, xs, ws = operands(rng, T, K, N, 128)
    x[1, 150], ws[0][0][7, 3] = 0x7F, 0xFF
    y = to_f64(G.linear_fp8(*to_gpu(x, xs, ws)))
    bad = np.isnan(y)
    assert bad[1].all() and bad[:, 7].all()
    bad[1] = bad[:, 7] = False
    assert not bad.any()
    # a scale that is not finite reaches its own rows only
    xs[0, 1] = np.inf
    y = to_f64(G.linear_fp8(*to_gpu(x, xs, ws)))
    assert not np.isfinite(y[0]).any() and np.isfinite(np.delete(y[2:], 7, 1)).all()


@pytest.mark.parametrize("T", [4, 90])
def test_zero_and_unusual_gated_rows(T):
    """Rows of zeros have scale 1 and zero codes; a NaN row has scale 1 and NaN codes."""
    rng = np.random.default_rng(T)
    x, xs, ws = operands(rng, T, 256, 260, 128, 2)
    x[0], x[2, 9] = 0, 0x7F
    q, s = G.gated_linear_fp8(*to_gpu(x, xs, ws), dtype=F8)
    assert (raw(q)[0] & 0x7F == 0).all() and (s[0] == 1).all()
    assert (raw(q)[2] & 0x7F == 0x7F).all() and (s[2] == 1).all()
    assert np.isfinite(decode(raw(q)[[1, 3]])).all()


def test_empty_sizes():
    f = torch.empty
    d = dev()
    x = f((0, 256), dtype=F8, device=d)
    w, ws = f((128, 256), dtype=F8, device=d), f((1, 2), device=d)
    assert G.linear_fp8(x, f((0, 2), device=d), w, ws).shape == (0, 128)
    assert G.linear_fp8(f((3, 256), dtype=F8, device=d), f(3, device=d), w[:0], ws[:0]).shape == (3, 0)
    bias = torch.randn(128, device=d)
    for T in (3, 50):                                  # no columns to sum over
        y = G.linear_fp8(f((T, 0), dtype=F8, device=d), f(T, device=d), w[:, :0].contiguous(), f((1, 0), device=d),
                         bias=bias, dtype=F32)
        assert bits_equal(y, bias.expand(T, 128).contiguous())
    q, s = G.quantize_fp8(f((0, 100), device=d))
    assert q.shape == (0, 100) and s.shape == (0,)
    q, s = G.gated_linear_fp8(x, f((0, 2), device=d), w, ws, w, ws, dtype=F8)
    assert q.shape == (0, 128) and s.shape == (0, 1)


def test_repeatable():
    rng = np.random.default_rng(1)
    for T in (7, 100, 1500):
        a = to_gpu(*operands(rng, T, 700, 400, 128, 2))
        first, gated = G.linear_fp8(*a[:4]), G.gated_linear_fp8(*a, dtype=F8)
        for _ in range(3):
            assert bits_equal(G.linear_fp8(*a[:4]), first)
            again = G.gated_linear_fp8(*a, dtype=F8)
            assert bits_equal(again[0], gated[0]) and bits_equal(again[1], gated[1])


# ------------------------------------------------------------------ quantisation
def check_quantized(x, q, scale, rows, cols):
    want, each = ref.block_scales(x, rows, cols)
    sc = to_f64(scale).reshape(want.shape)
    assert (np.abs(sc - want) <= 2.0 ** -23 * want).all()
    c = decode(raw(q)).reshape(x.shape)
    e = np.abs(c * each - x)
    step = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * each)
    assert (e <= step * (1 + 2.0 ** -3 * 2.0 ** -15) + 2.0 ** -20 * np.abs(x)).all()


@pytest.mark.parametrize("T,D", [(1, 1), (1, 4096), (3, 100), (16, 128), (5, 1001), (300, 515), (70, 2048), (33, 5000),
                                 (9, 16384), (2, 32768)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [0, 128])
def test_quantize(T, D, dtype, group):
    rng = np.random.default_rng(T + D)
    x = put(rng.normal(size=(T, D)) * np.exp(3 * rng.normal(size=(T, 1))), dtype)
    x[0, : D // 2] = 0
    q, s = G.quantize_fp8(x, group)
    check_quantized(to_f64(x), q, s, 1, group)
    # rows at a stride, at addresses of no alignment
    wide = torch.zeros((T, D + 3), dtype=dtype, device=dev())
    wide[:, 1:1 + D] = x
    q2, s2 = G.quantize_fp8(wide[:, 1:1 + D], group)
    assert bits_equal(q, q2) and bits_equal(s, s2)


@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (129, 257), (1000, 300), (300, 1001), (64, 4096)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_weight(N, K, dtype):
    rng = np.random.default_rng(N + K)
    w = put(rng.normal(size=(N, K)) * np.exp(rng.normal(size=(N, 1))), dtype)
    q, s = G.quantize_weight_fp8(w)
    assert s.shape == (-(-N // 128), -(-K // 128))
    check_quantized(to_f64(w), q, s, 128, 128)


@pytest.mark.parametrize("group", [0, 128])
def test_quantize_as_the_norm_does(group):
    """The codes and scales of add_rmsnorm_fp8, from the values that it quantises."""
    x = torch.randn((50, 1000), device=dev())
    y, _ = G.add_rmsnorm(x)
    q, s, _ = G.add_rmsnorm_fp8(x, group=group)
    q2, s2 = G.quantize_fp8(y, group)
    assert bits_equal(q, q2) and bits_equal(s, s2)


def test_quantize_special_values():
    x = torch.randn((6, 256), device=dev())
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 200] = float("inf")
    x[3] = 1e-44
    x[4, :128] = 3e38
    q, s = G.quantize_fp8(x, 128)
    c = decode(raw(q))
    assert (c[0] == 0).all() and (s[0] == 1).all()
    assert s[1, 0] == 1 and np.isnan(c[1, 3]) and np.isfinite(c[1, 4:]).all()
    assert np.isinf(s[2, 1].item()) and np.isnan(c[2, 200]) and np.isfinite(c[2, :128]).all()
    assert (s[3].double() == 2.0 ** -140).all() and np.isfinite(c[3]).all()
    assert (np.abs(c[4, :128]) == 448).all()


# ------------------------------------------------------------------ rotary positions
def check_rope(x, positions, inv, interleaved, eps, weight, got, dtype):
    want, size = ref.rope(to_f64(x), positions, inv, interleaved, eps, weight)
    keep = positions >= 0
    e = np.abs(to_f64(got) - want)[keep]
    tol = ((2.0 ** -21 + (2.0 ** -19 if eps is not None else 0)) * size)[keep]
    assert (e <= tol + half(dtype) * (np.abs(want[keep]) + tol) + 2.0 ** -140).all(), (e - tol).max()


HEADS = [  # DH, rotary
    (128, 128), (64, 64), (128, 64), (96, 96), (80, 80), (80, 40), (256, 256), (2, 2), (100, 20), (250, 250), (64, 0),
    (7, 4), (1, 0), (254, 32), (48, 16)]


@pytest.mark.parametrize("DH,R", HEADS)
@pytest.mark.parametrize("dtype,interleaved,norm,T", [(BF, False, True, 9), (F32, True, False, 5), (F32, False, True, 70),
                                                      (BF, True, True, 1), (F32, False, False, 1100)])
def test_rope(DH, R, dtype, interleaved, norm, T):
    rng = np.random.default_rng(DH + R + T)
    Hq, Hk = 5, 2
    x = put(rng.normal(size=(T, Hq + 2 * Hk, DH)), dtype)
    q, k = x[:, :Hq], x[:, Hq:Hq + Hk]
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    pos[rng.random(T) < 0.2] = -1
    pos[0] = 0 if T > 1 else 262143
    inv = G.rotary_inv_freq(R, device="cpu")
    qw, kw = f32(1 + 0.2 * rng.normal(size=DH)), f32(rng.normal(size=DH))
    qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
    args = dict(q_weight=put(qw), k_weight=put(kw), eps=1e-6) if norm else {}
    a, b = G.qk_norm_rope(q, k, put(pos, torch.int32), inv.to(dev()) if R else None, interleaved=interleaved,
                          q_out=qo, k_out=ko, **args)
    assert a is qo and b is ko
    eps = 1e-6 if norm else None
    inv = inv.numpy()
    check_rope(q, pos, inv, interleaved, eps, qw if norm else None, qo, dtype)
    check_rope(k, pos, inv, interleaved, eps, kw if norm else None, ko, dtype)
    skip = torch.from_numpy(pos < 0).to(dev())
    assert (qo[skip] == 7).all() and (ko[skip] == 7).all()
    # in place, in the projection's own rows; the values beside them stay
    before = x.clone()
    G.qk_norm_rope(q, k, put(pos, torch.int32), put(inv) if R else None, interleaved=interleaved, q_out=q, k_out=k,
                   **args)
    assert bits_equal(q[~skip], qo[~skip]) and bits_equal(k[~skip], ko[~skip])
    assert bits_equal(q[skip], before[:, :Hq][skip]) and bits_equal(x[:, Hq + Hk:], before[:, Hq + Hk:])


def test_rope_far_positions_keep_their_angle():
    """The largest position: the angle in fp32 would be off by 64 radians."""
    inv = G.rotary_inv_freq(64)
    q = torch.randn((3, 2, 64), device=dev())
    pos = np.array([2 ** 31 - 1, 2 ** 30 + 1, 262143], dtype=np.int32)
    a, b = G.qk_norm_rope(q, None, put(pos, torch.int32), inv)
    assert b is None
    # the product of two such numbers has 55 bits in 64-bit arithmetic's 53, about 2^-22 of the reference's angle
    want, size = ref.rope(to_f64(q), pos, inv.cpu().numpy(), False)
    assert (np.abs(to_f64(a) - want) <= (2.0 ** -21 + 2.0 ** -20) * size).all()


def test_rope_keeps_lengths_and_distances():
    """Turned queries and keys have the products of their distance: positions shifted alike agree."""
    inv = G.rotary_inv_freq(128)
    q, k = torch.randn((1, 1, 128), device=dev()), torch.randn((1, 1, 128), device=dev())
    dots = []
    for shift in (0, 1000, 250000):
        a, _ = G.qk_norm_rope(q, None, put([shift + 37], torch.int32), inv)
        b, _ = G.qk_norm_rope(k, None, put([shift], torch.int32), inv)
        dots.append(float((a.double() * b.double()).sum()))
    size = float((q.double().abs() * k.double().abs()).sum())
    assert max(dots) - min(dots) <= 2.0 ** -18 * 4 * size


def test_rope_norm_of_unusual_rows():
    x = torch.randn((5, 1, 128), device=dev())
    x[0] *= 1e25
    x[1] *= 1e-30
    x[2] = 0
    x[3, 0, 5] = float("nan")
    a, _ = G.qk_norm_rope(x, None, None, None, eps=1e-6)
    y = to_f64(a)
    for r, e in ((0, 1e-6), (2, 1e-6), (4, 1e-6)):
        want, _ = ref.rope(to_f64(x[r:r + 1]), np.zeros(1), None, False, e)
        assert (np.abs(y[r:r + 1] - want) <= 2.0 ** -18 * np.abs(want)).all()
    assert np.isnan(y[3]).all()
    b, _ = G.qk_norm_rope(x[1:2], None, None, None, eps=0.0)
    assert abs((to_f64(b) ** 2).mean() - 1) < 2.0 ** -17


def test_rope_refusals_on_the_gpu():
    q = torch.zeros((2, 3, 64), device=dev())
    inv, pos = G.rotary_inv_freq(64), torch.zeros(2, dtype=torch.int32, device=dev())
    with pytest.raises(ValueError):
        G.qk_norm_rope(q, None, None, inv)
    with pytest.raises(ValueError):
        G.qk_norm_rope(q, q.bfloat16(), pos, inv)
    with pytest.raises(ValueError):
        G.qk_norm_rope(q, None, pos, G.rotary_inv_freq(66))
    with pytest.raises(ValueError):
        G.qk_norm_rope(q, None, pos, inv, q_weight=torch.ones(64, device=dev()))
    with pytest.raises(ValueError):
        G.qk_norm_rope(q, None, pos[:1], inv)
    with pytest.raises(G.HyenaError):
        G.qk_norm_rope(q, None, pos, inv, q_out=q[:1].expand(2, 3, 64))


def test_linear_refusals_on_the_gpu():
    d = dev()
    x, xs = torch.zeros((4, 256), dtype=F8, device=d), torch.ones((4, 2), device=d)
    w, ws = torch.zeros((128, 256), dtype=F8, device=d), torch.ones((1, 2), device=d)
    for bad in ((x, xs[:3], w, ws), (x, xs, w[:, :128], ws), (x, xs, w, ws[:, :1]), (x, xs, w.t(), ws),
                (x.t(), xs, w, ws), (x, xs, w[0], ws)):
        with pytest.raises(ValueError):
            G.linear_fp8(*bad)
    with pytest.raises(TypeError):
        G.linear_fp8(x, xs, w, ws, dtype=torch.float16)
    with pytest.raises(ValueError):
        G.linear_fp8(x, xs, w, ws, out=torch.empty((4, 127), dtype=BF, device=d))
    with pytest.raises(ValueError):
        G.gated_linear_fp8(x, xs, w, ws, w[:64], ws)
    with pytest.raises(ValueError):
        G.gated_linear_fp8(x, xs, w, ws, w, ws, scale=xs)
