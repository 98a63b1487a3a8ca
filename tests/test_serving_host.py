"""Serving operators without a GPU: refusals of the C entry points, all of which
return before any HIP call, and the tests' own 64-bit implementations against
values worked by hand."""
import ctypes
import math
import os

import numpy as np
import pytest

import genomic_lm_amd as G
from tests import serving_ref as ref

P = ctypes.c_void_p
FAKE = P(0x10000)            # never dereferenced
ODD = P(0x10001)
BAD, UNS, WS, OK = G.ERR_INVALID_ARG, G.ERR_UNSUPPORTED, G.ERR_WORKSPACE, G.OK


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(G.LIB_PATH):
        from genomic_lm_amd import build
        build.build()
    yield


def refusals(f, good, cases):
    for change, want in cases:
        a = list(good)
        for k, v in change.items():
            a[k] = v
        assert f(*a) == want, change


def test_norm_refusals():
    # x xs res rs w eps y ys ro ros T D io stream
    good = [FAKE, 8, FAKE, 8, FAKE, 1e-6, FAKE, 8, FAKE, 8, 4, 8, G.BF16, None]
    refusals(G.lib().hyena_add_rmsnorm, good, [
        ({0: None}, BAD), ({6: None}, BAD), ({2: None}, BAD),     # residual_out without a residual
        ({0: ODD}, BAD), ({2: ODD}, BAD), ({4: P(0x10002)}, BAD), ({6: ODD}, BAD), ({8: ODD}, BAD),
        ({1: -1}, BAD), ({3: -1}, BAD), ({7: 7}, BAD), ({9: 7}, BAD),
        ({5: -1.0}, BAD), ({5: math.nan}, BAD), ({5: math.inf}, BAD),
        ({10: -1}, BAD), ({11: -1}, BAD), ({12: 5}, BAD), ({11: 32769, 7: 40000, 9: 40000}, UNS),
        ({10: 1 << 60}, UNS), ({10: 0, 0: None}, OK), ({11: 0, 0: None}, OK)])
    # x xs res rs w eps q scale group ro ros T D io stream
    good = [FAKE, 8, FAKE, 8, None, 1e-6, FAKE, FAKE, 0, FAKE, 8, 4, 8, G.F32, None]
    refusals(G.lib().hyena_add_rmsnorm_fp8, good, [
        ({6: None}, BAD), ({7: None}, BAD), ({7: ODD}, BAD), ({8: 64}, BAD), ({8: -1}, BAD),
        ({2: None}, BAD), ({0: P(0x10002)}, BAD), ({12: 32769, 10: 40000}, UNS), ({11: 0}, OK)])


def test_page_map_refusals():
    # old new R table stride width free F head P cu lens pos slots T status stream
    good = [FAKE, FAKE, 2, FAKE, 4, 4, FAKE, 9, None, 16, FAKE, FAKE, None, FAKE, 5, FAKE, None]
    refusals(G.lib().hyena_page_map, good, [
        ({0: None}, BAD), ({1: None}, BAD), ({3: None}, BAD), ({6: None}, BAD), ({10: None}, BAD),
        ({11: None}, BAD), ({13: None}, BAD), ({15: None}, BAD), ({2: -1}, BAD), ({5: -1}, BAD),
        ({4: 3}, BAD), ({7: -1}, BAD), ({14: -1}, BAD), ({9: 24}, BAD), ({9: 0}, BAD),
        ({9: 8}, UNS), ({9: 512}, UNS), ({2: 4097}, UNS), ({0: ODD}, BAD), ({13: P(0x10004)}, BAD),
        ({5: 1 << 40, 4: 1 << 40}, UNS)])


def test_append_refusals():
    # k kt kh v vt vh slots kc vc ks vs N P T H DH io stream
    good = [FAKE, 256, 128, FAKE, 256, 128, FAKE, FAKE, FAKE, FAKE, FAKE, 3, 64, 5, 2, 128, G.BF16, None]
    refusals(G.lib().hyena_kv_append_fp8, good, [
        ({0: None}, BAD), ({3: None}, BAD), ({6: None}, BAD), ({7: None}, BAD), ({8: P(0x10008)}, BAD),
        ({9: None}, BAD), ({10: ODD}, BAD), ({11: 0}, BAD), ({12: 48}, BAD), ({12: 8}, UNS),
        ({13: -1}, BAD), ({14: -1}, BAD), ({15: 96}, UNS), ({14: 1025}, UNS), ({16: 2}, BAD),
        ({1: -1}, BAD), ({0: ODD}, BAD), ({6: P(0x10004)}, BAD), ({13: 0, 0: None}, OK),
        ({13: 1 << 31}, UNS), ({1: 1 << 60}, UNS)])


def test_attention_refusals():
    # q qt qh kc vc ks vs N P table ts width lens cu R T max_q Hq Hkv DH scale out io ws bytes stream
    good = [FAKE, 512, 128, FAKE, FAKE, FAKE, FAKE, 3, 64, FAKE, 2, 2, FAKE, FAKE, 2, 5, 3, 4, 2, 128,
            0.1, FAKE, G.BF16, None, 0, None]
    f = G.lib().hyena_attn_paged_fp8
    refusals(f, good, [
        ({0: None}, BAD), ({21: None}, BAD), ({9: None}, BAD), ({12: None}, BAD), ({13: None}, BAD),
        ({3: P(0x10008)}, BAD), ({5: None}, BAD), ({17: 5}, BAD), ({18: 0}, BAD), ({19: 32}, UNS),
        ({8: 20}, BAD), ({8: 8}, UNS), ({7: 0}, BAD), ({20: math.nan}, BAD), ({22: 7}, BAD),
        ({10: 1}, BAD), ({14: 4097}, UNS), ({14: -1}, BAD), ({16: -1}, BAD), ({1: -1}, BAD),
        ({17: 2048}, UNS), ({14: 0, 0: None}, OK), ({15: 0, 0: None}, OK), ({16: 0, 0: None}, OK)])
    size = G.lib().hyena_attn_paged_workspace_size
    need = size(2, 5, 3, 64, 64, 4, 2, 128)
    assert need > 0 and size(2, 5, 3, 2, 64, 4, 2, 128) == 0      # 128 tokens are never split
    assert size(0, 5, 3, 64, 64, 4, 2, 128) == 0 and size(2, 5, 3, 64, 24, 4, 2, 128) == 0
    long = {10: 64, 11: 64}
    refusals(f, good, [(long, WS), ({**long, 23: FAKE, 24: need - 1}, WS),
                       ({**long, 23: P(0x10008), 24: need}, WS)])


def test_binding_refuses_cpu_tensors():
    import torch
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        G.add_rmsnorm(x)
    with pytest.raises(TypeError):
        G.add_rmsnorm_fp8(x.half())
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        G.page_map(i, i, i.view(2, 1), i, None, 16, 2)
    k = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError):
        G.kv_append_fp8(k, k, i.long(), k, k, k, k)
    with pytest.raises(ValueError):
        G.attn_paged_fp8(k, k, k, k, k, i.view(2, 1), i, i, 1)


# ------------------------------------------------------------------ the tests' own formulas
def test_ref_codes():
    assert ref.decode([0x00, 0x01, 0x08, 0x38, 0x7E, 0xBC]).tolist() == [0, 2 ** -9, 2 ** -6, 1.0, 448.0, -1.5]
    assert np.isnan(ref.decode([0x7F])).all()
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    back = ref.encode(ref.decode(codes))
    assert (back == codes).all()
    # halfway values go to the even code
    assert ref.encode([1.0625]).tolist() == [0x38] and ref.encode([1.1875]).tolist() == [0x3A]
    assert ref.encode([2.0 ** -10, 3 * 2.0 ** -10]).tolist() == [0x00, 0x02]


def test_ref_block_scale():
    assert ref.block_scale(448.0) == 1.0 and ref.block_scale(449.0) == 2.0
    assert ref.block_scale(0.0) == ref.MIN_SCALE and ref.block_scale(3.5) == 2.0 ** -7


def test_ref_norm_and_map():
    s, y = ref.rmsnorm(np.array([[3.0, 4.0]]), np.array([[0.0, 0.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(y, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]])
    table = np.full((2, 3), -1)
    table[0, 0] = 7
    cu, lens, pos, slots, status = ref.page_map([15, 0], [2, 1], table, [4, 5], 0, 16, 5)
    assert cu.tolist() == [0, 2, 3] and lens.tolist() == [17, 1]
    assert pos.tolist() == [15, 16, 0, -1, -1] and slots.tolist() == [7 * 16 + 15, 4 * 16, 5 * 16, -1, -1]
    assert table.tolist() == [[7, 4, -1], [5, -1, -1]] and status.tolist() == [2, 0]


def test_ref_attention_hand_worked():
    """Two tokens with scores 0 and log 3: weights 1/4 and 3/4."""
    kc = np.zeros((1, 1, 16, 64), np.uint8)
    vc = np.zeros((1, 1, 64, 16), np.uint8)
    kc[0, 0, 1, 0] = 0x38                                     # 1.0
    vc[0, 0, 0, 0], vc[0, 0, 0, 1] = 0x38, 0x40                # 1.0, 2.0
    vc[0, 0, 0, 2] = 0x7F                                     # past the end
    q = np.zeros((1, 1, 64))
    q[0, 0, 0] = math.log(3.0)
    one = np.ones((1, 1))
    out, mag, _ = ref.attention(q, kc, vc, one, one, np.array([[0]]), [2], [0, 1], 1.0, 16)
    assert abs(out[0, 0, 0] - 1.75) < 1e-12 and abs(mag[0, 0, 0] - 1.75) < 1e-12
