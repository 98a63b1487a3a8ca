"""The serving example end to end: chunked prefill and decode of a small striped stack against
one prefill of each whole sequence.

Both runs see the same tokens, so they differ by what is rounded differently: the cache's
block scales, which grow as tokens arrive in one run and are set at once in the other (a code moved
to a larger scale is not rounded again unless it falls below e4m3's normal range), the order of the
sums, and the activations' 8-bit codes, where a sum near the middle of two codes may fall either
way (2^-4 of that value).  Such steps reach few values, so the hidden states agree to a few per cent."""
import os
import sys

import pytest
import torch

import genomic_lm_amd as G

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("page", ["16", "64"])
def test_served_equals_one_prefill(page):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import striped_serving
    finally:
        sys.path.pop(0)
    far, finite = striped_serving.main(["--dim", "256", "--heads", "4", "--steps", "20", "--page", page,
                                        "--prompts", "150", "1", "64", "17", "--chunk", "48"])
    assert finite and max(far) < 0.05, far
