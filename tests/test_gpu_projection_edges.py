"""The 8-bit projections where they can go wrong, and every kernel of the products at sizes that take it
(projection_sizes.py).

Tolerances, stated before any run: those of test_gpu_projection.py for single elements.  For the norm of a bf16
output's error against that of the output, where the signs of the products are random: the rounding of a value in [2^e, 2^(e+1))
is spread evenly over 2^(e-8) to either side, at most 2^-8 / sqrt 3 of the value in the mean square; a product cut below
2^-13 of the largest of its eight loses up to that much, 2^-13 / sqrt 3 of it in the mean square, the largest squared is at
most the eight squares' sum, so the cuts of a sum of K products of mean square p2 come to at most
sqrt(K 8 p2 / 3) 2^-13 against sqrt(K p2): 2^-13 sqrt(8 / 3).  Together 2.27e-3, allowed 2.3e-3; a column of
K = 1040 left out is 3e-2.

Small whole numbers (and scales that are powers of two) have exact sums in any order, and no product below 2^-13 of
another: those outputs are compared for equality."""
import numpy as np
import pytest
import torch

import genomic_lm_amd as G
from tests import projection_ref as ref
from tests import projection_sizes as sizes
from tests.gpu_util import dev, to_f64
from tests.test_gpu_projection import bits_equal, check_gated, f32, half, operands, put, sum_error, to_gpu

pytestmark = pytest.mark.gpu

BF, F32, F8, U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.lib()
    yield


@pytest.mark.parametrize("T,I", [(1, 200), (40, 384), (300, 4000), (25600, 384)])
def test_gated_without_columns(T, I):
    """K = 0: h is act(0) * 0 = 0, in codes with scale 1, and nothing is written behind them (25600 rows
    take one launch, the others go by way of a workspace)."""
    e = torch.empty
    args = (e((T, 0), dtype=F8, device=dev()), e(T, device=dev())) + 2 * (
        e((I, 0), dtype=F8, device=dev()), e((-(-I // 128), 0), device=dev()))
    for dtype in (BF, F32):
        h = torch.full((T, I), 7.0, dtype=dtype, device=dev())
        assert (G.gated_linear_fp8(*args, out=h) == 0).all()
    buf = torch.full((5 * T * I,), 0x38, dtype=U8, device=dev())
    scale = torch.full((T, -(-I // 128)), 7.0, device=dev())
    q, s = G.gated_linear_fp8(*args, dtype=U8, out=buf[:T * I].view(T, I), scale=scale)
    assert (q & 0x7F == 0).all() and (s == 1).all()
    assert (buf[T * I:] == 0x38).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_without_columns(dtype):
    """An empty row has no magnitude: scale 1, as a row of zeros."""
    for shape in ((5, 0), (2, 3, 0)):
        scale = torch.full(shape[:-1], 7.0, device=dev())
        q, s = G.quantize_fp8(torch.empty(shape, dtype=dtype, device=dev()), scale=scale)
        assert q.shape == shape and s is scale and (s == 1).all()
        q, s = G.quantize_fp8(torch.empty(shape, dtype=dtype, device=dev()), group=128)
        assert s.shape == shape


# ------------------------------------------------------------------ every kernel
def whole(rng, most, T, K, N, group, weights=1):
    """Operands of whole numbers up to `most` with scales 1/2, 1 and 2, and what they stand for."""
    runs = -(-K // 128)
    x = rng.integers(-most, most + 1, (T, K))
    xs = 2.0 ** rng.integers(-1, 2, (T, runs) if group else (T,))
    out, wide = [put(x).to(F8), put(xs)], []
    each = np.repeat(xs, 128, 1)[:, :K] if group else xs[:, None]
    xw = x * each
    for _ in range(weights):
        w = rng.integers(-most, most + 1, (N, K))
        ws = 2.0 ** rng.integers(-1, 2, (-(-N // 128), runs))
        out += [put(w).to(F8), put(ws)]
        wide.append(xw @ (w * np.repeat(np.repeat(ws, 128, 0)[:N], 128, 1)[:, :K]).T)
    return out, wide


def rounded(a, dtype):
    """Values of at most 24 bits in a type: one rounding."""
    assert (a == f32(a)).all()
    return put(a).to(dtype)


@pytest.mark.parametrize("T,K,N", sizes.cases(sizes.PLAIN))
def test_exact_sums(T, K, N):
    rng = np.random.default_rng(T + K + N)
    for group in (128, 0):
        args, (want,) = whole(rng, 4, T, K, N, group)
        b = rng.integers(-100, 101, N)
        for dtype in (BF, F32):
            assert bits_equal(G.linear_fp8(*args, dtype=dtype), rounded(want, dtype)), (group, dtype)
            assert bits_equal(G.linear_fp8(*args, bias=put(b), dtype=dtype), rounded(want + b, dtype)), (group, dtype)


@pytest.mark.parametrize("T,K,N", sizes.cases(sizes.GATED) + sizes.cases(sizes.CODES))
def test_exact_gated(T, K, N):
    rng = np.random.default_rng(T + K + N)
    args, (g, u) = whole(rng, 1, T, K, N, 128, 2)
    h = g * u
    for dtype in (BF, F32):
        assert bits_equal(G.gated_linear_fp8(*args, act="none", dtype=dtype) + 0, rounded(h, dtype) + 0), dtype
    q, scale = G.gated_linear_fp8(*args, act="none", dtype=F8)
    want, wscale = G.quantize_fp8(rounded(h, F32), 128)
    assert bits_equal(scale, wscale) and torch.equal(q.float(), want.float())


@pytest.mark.parametrize("T,K,N", [c for c in sizes.cases(sizes.PLAIN) if c[0] == 2100])
@pytest.mark.parametrize("group", [0, 128])
def test_large_tiles(T, K, N, group):
    rng = np.random.default_rng(T + K + N + group)
    x, xs, ws = operands(rng, T, K, N, group)
    b = f32(rng.normal(size=N))
    args = to_gpu(x, xs, ws)
    want, size = ref.product(x, xs, *ws[0])
    want, size = want + b.astype(np.float64), size + np.abs(b)
    for dtype in (BF, F32):
        e = np.abs(to_f64(G.linear_fp8(*args, bias=put(b), dtype=dtype)) - want)
        tol = sum_error(K, size, dtype)
        assert (e <= tol + half(dtype) * (np.abs(want) + tol)).all(), (dtype, (e - tol).max())
        far = np.linalg.norm(e) / np.linalg.norm(want)
        assert dtype == F32 or far <= 2.3e-3, far


@pytest.mark.parametrize("T,K,N,act", [(*c, act) for (c, act) in zip(
    [c for c in sizes.cases(sizes.GATED) if c[0] == 2100], 4 * ("gelu", "silu", "gelu_tanh"))])
def test_large_gated_tiles(T, K, N, act):
    rng = np.random.default_rng(T + K + N)
    x, xs, ws = operands(rng, T, K, N, 128, 2)
    xs = xs / f32(60 * K ** 0.5)
    args = to_gpu(x, xs, ws)
    for dtype in (BF, F32):
        check_gated(x, xs, ws, act, G.gated_linear_fp8(*args, act=act, dtype=dtype), dtype)


@pytest.mark.parametrize("T,K,N,act", [(*c, act) for (c, act) in zip(sizes.cases(sizes.CODES), 4 * ("gelu", "silu"))])
def test_large_code_tiles(T, K, N, act):
    rng = np.random.default_rng(T + K + N)
    x, xs, ws = operands(rng, T, K, N, 128, 2)
    xs = xs / f32(60 * K ** 0.5)
    check_gated(x, xs, ws, act, G.gated_linear_fp8(*to_gpu(x, xs, ws), act=act, dtype=F8), None)


@pytest.mark.parametrize("T,N", [(4, 400), (40, 400), (700, 1500), (1100, 1500), (2100, 2100), (2100, 4000)])
@pytest.mark.parametrize("K,apart", [(1040, 1), (1040, 500), (1041, 1)])
def test_large_products_that_cancel(T, N, K, apart):
    """Two products of 448 * 448 that cancel, side by side or in different groups of eight columns, among whole
    numbers up to 4: fp32 outputs and calls of few rows keep every bit; bf16 outputs of many rows may lose what lies
    below 2^-13 of the largest product of eight columns, at most 2^-10 of the magnitudes."""
    rng = np.random.default_rng(T + N + K + apart)
    runs = -(-K // 128)
    x, w = rng.integers(-4, 5, (T, K)).astype(np.float64), rng.integers(-4, 5, (N, K)).astype(np.float64)
    a = 7 if apart == 1 else 130
    x[:, [a, a + apart]] = 448
    w[:, a], w[:, a + apart] = 448, -448
    want, size = x @ w.T, np.abs(x) @ np.abs(w).T
    assert np.abs(want).max() < 2 ** 20
    args = (put(x).to(F8), torch.ones((T, runs), device=dev()), put(w).to(F8),
            torch.ones((-(-N // 128), runs), device=dev()))
    assert bits_equal(G.linear_fp8(*args, dtype=F32), rounded(want, F32))
    y = G.linear_fp8(*args)
    if T <= (64 if K % 16 == 0 else 16):
        assert bits_equal(y, rounded(want, BF))
    cut = 2.0 ** -10 * size
    e = np.abs(to_f64(y) - want)
    assert (e <= cut + half(BF) * (np.abs(want) + cut)).all()
    h = G.gated_linear_fp8(*args, *args[2:], act="none", dtype=F32)
    q, scale = G.gated_linear_fp8(*args, *args[2:], act="none", dtype=F8)
    want = rounded(f32(want) * f32(want), F32)           # one rounding, of the product
    qw, sw = G.quantize_fp8(want, 128)
    assert bits_equal(h, want) and bits_equal(scale, sw) and torch.equal(q.float(), qw.float())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 128])
def test_codes_by_the_stated_steps(dtype, rows):
    """scale = max|x| / 448 and the code of x * (1 / scale), each step rounded to fp32."""
    rng = np.random.default_rng(rows)
    x = put(rng.normal(size=(256, 384)) * np.exp(2 * rng.normal(size=(256, 1))), dtype)
    q, s = G.quantize_weight_fp8(x) if rows > 1 else G.quantize_fp8(x, 128)
    v = x.float().cpu().numpy()
    top = np.abs(v).reshape(256 // rows, rows, 3, 128).max((1, 3))
    scale = top / f32(448)
    z = v * np.repeat(np.repeat(f32(1) / scale, rows, 0), 128, 1)
    assert scale.dtype == z.dtype == np.float32
    assert bits_equal(s, put(scale)) and bits_equal(q, torch.from_numpy(z).to(F8).to(dev()))
