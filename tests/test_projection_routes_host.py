"""Which kernel a product of a size takes, and that it is one of the product that was asked for (no GPU)."""
import os

import pytest

import genomic_lm_amd as G
from tests.launches import BF, F8, F32, gated, launches

OUT = {F32: 0, BF: 1, F8: 2}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(G.LIB_PATH):
        from genomic_lm_amd import build
        build.build()
    yield


def is_gated(name, args):
    """Whether a kernel of the products is one of two weights, and the kind of its output."""
    if name == "linear_turns_kernel":
        return bool(args[0]), OUT[BF]
    return bool(args[-2]), args[-1]


GATED = [(T, K, I, out, odd)
         for T, I in ((1, 1), (5, 384), (20, 9000), (70, 384), (300, 4000), (1030, 520), (2100, 1900), (5200, 2500),
                      (8192, 11008), (25600, 384))
         for K in (0, 1, 128, 4096) for out in (BF, F32, F8) for odd in (False, True)]


def test_gated_products_take_gated_kernels():
    """Whether or not there are columns of K and with them pointers to the weights: no other kernel has a
    gated product's output (an fp32 one is four times as large as the codes)."""
    calls = [gated(T, K, I, out, odd, weights=0x100000 if K else None) for T, K, I, out, odd in GATED]
    for case, (status, found) in zip(GATED, launches(calls)):
        assert status == G.OK and found, case
        T, K, I, out, odd = case
        two = out == F8 and G.gated_linear_fp8_workspace_size(T, I, K) > 0
        products = found[:-1] if two else found
        if two:
            assert found[-1][0] == "quantize_runs_kernel", (case, found)
        for name, args, _, _ in products:
            assert is_gated(name, args) == (True, OUT[F32 if two else out]), (case, name, args)
