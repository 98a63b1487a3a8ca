"""The 8-bit projections where they can go wrong."""
import numpy as np
import pytest
import torch

import genomic_lm_amd as G
from tests.gpu_util import dev

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
