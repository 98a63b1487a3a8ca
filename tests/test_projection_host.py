"""The 8-bit projections and rotary positions without a GPU: refusals of the C entry points, all
of which return before any HIP call, and of the binding; the tests' own formulas by hand."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import genomic_lm_amd as G
from tests import projection_ref as ref
from tests.test_serving_host import refusals

P = ctypes.c_void_p
FAKE = P(0x10000)            # never dereferenced
ODD = P(0x10001)
BAD, UNS, OK = G.ERR_INVALID_ARG, G.ERR_UNSUPPORTED, G.OK


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(G.LIB_PATH):
        from genomic_lm_amd import build
        build.build()
    yield


def test_linear_refusals():
    # x xs scale ss group w ws bias y ys T N K io stream
    good = [FAKE, 256, FAKE, 2, 128, FAKE, FAKE, FAKE, FAKE, 384, 5, 384, 256, G.BF16, None]
    refusals(G.lib().hyena_linear_fp8, good, [
        ({0: None}, BAD), ({2: None}, BAD), ({5: None}, BAD), ({6: None}, BAD), ({8: None}, BAD),
        ({2: ODD}, BAD), ({6: ODD}, BAD), ({7: P(0x10002)}, BAD), ({8: ODD}, BAD),
        ({8: P(0x10002), 13: G.F32}, BAD), ({1: -1}, BAD), ({3: -1}, BAD), ({4: 64}, BAD), ({9: 383}, BAD),
        ({10: -1}, BAD), ({11: -1}, BAD), ({12: -1}, BAD), ({13: 3}, BAD),
        ({11: (1 << 20) + 1, 9: 1 << 21}, UNS), ({12: (1 << 20) + 1}, UNS), ({10: 1 << 31}, UNS),
        ({1: 1 << 60}, UNS), ({10: 1 << 30, 11: 1 << 20, 9: 1 << 20}, UNS),
        ({10: 0, 0: None, 8: None}, OK), ({11: 0, 5: None, 8: None}, OK)])


def test_gated_refusals():
    # x xs scale ss group wg gs wu us act h hs T I K io stream
    good = [FAKE, 256, FAKE, 1, 0, FAKE, FAKE, FAKE, FAKE, 1, FAKE, 384, 5, 384, 256, G.F32, None]
    refusals(G.lib().hyena_gated_linear_fp8, good, [
        ({5: None}, BAD), ({6: None}, BAD), ({7: None}, BAD), ({8: None}, BAD), ({8: ODD}, BAD), ({10: None}, BAD),
        ({9: 4}, BAD), ({9: -1}, BAD), ({10: P(0x10002)}, BAD), ({11: 100}, BAD), ({15: 2}, BAD), ({4: 1}, BAD),
        ({13: 1 << 21, 11: 1 << 21}, UNS), ({12: 0, 10: None}, OK)])
    # x xs scale ss group wg gs wu us act q qs T I K ws bytes stream
    size = G.lib().hyena_gated_linear_fp8_workspace_size
    need = size(5, 384, 256)
    assert need == 5 * 384 * 4 and size(8192, 11008, 4096) == 0 and size(0, 384, 256) == 0
    good = [FAKE, 256, FAKE, 1, 0, FAKE, FAKE, FAKE, FAKE, 1, ODD, FAKE, 5, 384, 256, FAKE, need, None]
    refusals(G.lib().hyena_gated_linear_fp8_quant, good, [
        ({10: None}, BAD), ({11: None}, BAD), ({11: ODD}, BAD), ({9: 4}, BAD), ({7: None}, BAD), ({13: -2}, BAD),
        ({15: None}, G.ERR_WORKSPACE), ({16: need - 1}, G.ERR_WORKSPACE), ({15: P(0x10008)}, G.ERR_WORKSPACE),
        ({14: 1 << 21}, UNS), ({13: 0, 10: None}, OK)])


def test_quantize_refusals():
    # x xs q scale group T D io stream
    good = [FAKE, 64, FAKE, FAKE, 128, 4, 64, G.BF16, None]
    f = G.lib().hyena_quantize_fp8
    refusals(f, good, [
        ({0: None}, BAD), ({2: None}, BAD), ({3: None}, BAD), ({0: ODD}, BAD), ({3: P(0x10002)}, BAD), ({1: -1}, BAD),
        ({4: 127}, BAD), ({5: -1}, BAD), ({6: -1}, BAD), ({7: 9}, BAD), ({4: 0, 6: 32769}, UNS),
        ({6: (1 << 20) + 1}, UNS), ({5: 1 << 60}, UNS), ({1: 1 << 60}, UNS), ({5: 0, 0: None}, OK), ({6: 0}, OK)])
    # w ws q scale N K io stream
    good = [FAKE, 64, FAKE, FAKE, 4, 64, G.BF16, None]
    refusals(G.lib().hyena_quantize_weight_fp8, good, [
        ({0: None}, BAD), ({2: None}, BAD), ({3: None}, BAD), ({1: -5}, BAD), ({4: -1}, BAD), ({6: 4}, BAD),
        ({5: 1 << 21}, UNS), ({4: 0, 0: None}, OK)])


def test_rope_refusals():
    # q qt qh k kt kh pos f R il norm eps qw kw qo qot qoh ko kot koh T Hq Hk DH io stream
    good = [FAKE, 768, 128, FAKE, 768, 128, FAKE, FAKE, 128, 0, 1, 1e-6, FAKE, FAKE, FAKE, 512, 128, FAKE, 256, 128,
            3, 4, 2, 128, G.BF16, None]
    refusals(G.lib().hyena_qk_norm_rope, good, [
        ({0: None}, BAD), ({3: None}, BAD), ({14: None}, BAD), ({17: None}, BAD), ({6: None}, BAD), ({7: None}, BAD),
        ({0: ODD}, BAD), ({12: P(0x10002)}, BAD), ({6: ODD}, BAD), ({8: 63}, BAD), ({8: 130}, BAD), ({8: -2}, BAD),
        ({11: -1.0}, BAD), ({11: math.nan}, BAD), ({11: math.inf}, BAD), ({16: 64}, BAD), ({18: 64}, BAD),
        ({1: -1}, BAD), ({19: -1}, BAD), ({20: -1}, BAD), ({21: -1}, BAD), ({24: 7}, BAD),
        ({23: 260, 16: 260, 19: 260, 15: 2000, 18: 2000}, UNS), ({21: 1025}, UNS), ({20: (1 << 25) + 1}, UNS),
        ({1: 1 << 61}, UNS), ({20: 0, 0: None}, OK), ({23: 0, 8: 0}, OK), ({21: 0, 22: 0, 0: None}, OK)])


def test_binding_refusals():
    x = torch.zeros((2, 4), dtype=torch.uint8)
    f = torch.zeros(2)
    with pytest.raises(ValueError):
        G.linear_fp8(x, f, x, f)
    with pytest.raises(TypeError):
        G.linear_fp8(x.float(), f, x, f)
    with pytest.raises(ValueError):
        G.gated_linear_fp8(x, f, x, f, x, f, act="relu")
    with pytest.raises(ValueError):
        G.quantize_fp8(f)
    with pytest.raises(TypeError):
        G.quantize_weight_fp8(x)
    with pytest.raises(ValueError):
        G.qk_norm_rope(torch.zeros(1, 1, 8), None, None, None)
    with pytest.raises(ValueError):
        G.rotary_inv_freq(7, device="cpu")


# ------------------------------------------------------------------ the tests' own formulas
def test_inv_freq():
    got = G.rotary_inv_freq(8, 10000.0, 32.0, device="cpu")
    assert got.tolist() == [np.float32(v / 32) for v in (1, 0.1, 0.01, 0.001)]
    assert G.rotary_inv_freq(0, device="cpu").numel() == 0


def test_ref_product():
    one, half, two = 0x38, 0x30, 0x40             # e4m3 codes of 1, 0.5, 2
    x = np.array([[one, two], [half, one]], dtype=np.uint8)
    w = np.array([[two, 0xC0], [one, one], [0, half]], dtype=np.uint8)
    y, size = ref.product(x, np.array([1.0, 4.0]), w, np.array([[0.5]]))
    assert y.tolist() == [[-1.0, 1.5, 0.5], [-2.0, 3.0, 1.0]]
    assert size.tolist() == [[3.0, 1.5, 0.5], [6.0, 3.0, 1.0]]
    wide = ref.widen(np.full((1, 130), one, dtype=np.uint8), np.array([[2.0, 3.0]]))
    assert wide[0, 127] == 2.0 and wide[0, 128] == 3.0


def test_ref_act():
    g = np.array([-3.0, -0.5, 0.0, 2.0])
    assert np.allclose(ref.act(g, "silu"), g * 0.5 * (1 + np.tanh(g / 2)), rtol=1e-14)
    assert np.allclose(ref.act(g, "gelu_tanh"),
                       0.5 * g * (1 + np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))), rtol=1e-12)
    assert np.allclose(ref.act(g, "gelu"), [0.5 * v * (1 + math.erf(v / math.sqrt(2))) for v in g], rtol=1e-12)


def test_ref_rope():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    quarter = [math.pi / 2, math.pi]               # position 1: a quarter and a half turn
    y, _ = ref.rope(x, np.array([1]), quarter, False)
    assert np.allclose(y[0, 0], [-3, -2, 1, -4, 5, 6], atol=1e-12)
    y, _ = ref.rope(x, np.array([1]), quarter, True)
    assert np.allclose(y[0, 0], [-2, 1, -3, -4, 5, 6], atol=1e-12)
    y, _ = ref.rope(x, np.array([0]), quarter, True, eps=0.0, weight=np.full(6, 2.0))
    assert np.allclose((y / 2) ** 2 @ np.ones(6), 6)
