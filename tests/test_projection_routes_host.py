"""Which kernel a product of a size takes, and that it is one of the product that was asked for (no GPU)."""
import os

import pytest

import genomic_lm_amd as G
from tests import projection_sizes as sizes
from tests.launches import BF, F8, F32, gated, launches, library_kernels, linear

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


def rope(qo, ko, T=3, Hq=4, Hk=2, DH=128):
    """Strides (token, head) of the outputs."""
    at = 1 << 40
    return ("hyena_qk_norm_rope", [at, 768, 128, 2 * at, 768, 128, at, at, DH, 0, 0, 0.0, None, None, 3 * at, *qo, 4 * at,
                                   *ko, T, Hq, Hk, DH, G.BF16, None])


def test_rotated_rows_that_meet_are_refused():
    """Two (token, head) of an output in one place: written by different waves, in no order."""
    fine = [((512, 128), (256, 128)), ((128, 384), (128, 384)), ((1000, 130), (300, 150)),
            ((512, 128), (384, 256)), ((512, 128), (383, 255)),        # rows of one token in the gaps of another
            ((1 << 40, 128), (256, 128))]
    meet = [((128, 128), (256, 128)), ((512, 128), (128, 128)), ((256, 128), (256, 128)), ((128, 256), (256, 128)),
            ((511, 128), (256, 128)), ((128, 383), (256, 128)), ((385, 257), (255, 128)), ((0, 128), (256, 128)),
            ((512, 128), (382, 255))]
    # one token, or one head: the other stride has no say
    alone = [rope((0, 128), (0, 128), T=1), rope((128, 0), (128, 0), Hq=1, Hk=1)]
    # every pair of strides against every pair of rows
    cases = [(a, b, T, H) for a in (3, 4, 5, 6, 8, 9, 12, 13, 20, 21) for b in (4, 5, 6, 8, 10, 12, 15, 16, 24)
             for T, H in ((2, 2), (3, 5), (6, 3))]
    got = launches([rope(*c) for c in fine] + alone + [rope(*c) for c in meet]
                   + [rope((a, b), (H * b + 4, b), T, H, 1, 4) for a, b, T, H in cases])
    n = len(fine) + len(alone)
    for i, (status, found) in enumerate(got[:n]):
        assert status == G.OK and len(found) == 1, i
    for case, (status, found) in zip(meet, got[n:]):
        assert status == G.ERR_INVALID_ARG and not found, case
    for (a, b, T, H), (status, _) in zip(cases, got[n + len(meet):]):
        at = sorted(t * a + h * b for t in range(T) for h in range(H))
        apart = all(y - x >= 4 for x, y in zip(at, at[1:]))
        assert (status == G.OK) == apart, (a, b, T, H)


def test_rows_of_no_columns_are_given_a_scale():
    at = 1 << 40
    f, w = "hyena_quantize_fp8", "hyena_quantize_weight_fp8"
    calls = [(f, [None, 0, None, at, 0, 5, 0, G.BF16, None]), (f, [None, 0, None, at, 0, 5, 0, G.F32, None]),
             # nothing to write: no runs, no rows
             (f, [None, 0, None, None, 128, 5, 0, G.BF16, None]), (f, [None, 0, None, None, 0, 0, 0, G.BF16, None]),
             (w, [None, 0, None, None, 5, 0, G.BF16, None]),
             # what is needed and missing
             (f, [None, 0, None, None, 0, 5, 0, G.BF16, None]), (f, [None, 4, at, at, 0, 5, 4, G.BF16, None]),
             (f, [at, 4, None, at, 0, 5, 4, G.BF16, None])]
    got = [(status, [k[0] for k in found]) for status, found in launches(calls)]
    assert got[:2] == [(G.OK, ["quantize_rows_kernel"])] * 2
    assert got[2:5] == [(G.OK, [])] * 3
    assert got[5:] == [(G.ERR_INVALID_ARG, [])] * 3


def test_the_tests_sizes_take_every_kernel():
    """Each size of projection_sizes.py takes the kernel that it names, and together they take all that there are."""
    calls, want = [], []
    for make, table, outs in ((linear, sizes.PLAIN, (BF, F32)), (gated, sizes.GATED, (BF, F32)), (gated, sizes.CODES, (F8,))):
        for T, N, ks, kernel in table:
            for K in ks:
                for out in outs:
                    calls.append(make(T, K, N, out))
                    name, *tile = kernel[out] if isinstance(kernel, dict) else kernel
                    want.append((T, K, N, out, name, tuple(tile)))
    taken = set()
    for case, (status, found) in zip(want, launches(calls)):
        assert status == G.OK and len(found) == 1, (case, found)
        name, args, _, _ = found[0]
        assert (name, args[:len(case[-1])]) == case[-2:], (case, name, args)
        taken.add((name, args))
    there = {k for k in library_kernels() if k[0].startswith("linear_")}
    assert taken == there, (there - taken, taken - there)
