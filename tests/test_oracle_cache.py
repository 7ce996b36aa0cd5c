"""The definitions of the 4-bit cache, the token scores and the eviction, pinned by hand."""

import numpy as np
import pytest

from oracle import cache as oc


def test_e2m1_codes_and_scales():
    codes = np.array([[0x10, 0x32, 0x54, 0x76, 0x98, 0xba, 0xdc, 0xfe] * 2], dtype=np.uint8)
    want = [0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6] * 2
    for code, f in ((127, 1.0), (126, 0.5), (130, 8.0), (0, 2.0 ** -127), (254, 2.0 ** 127)):
        assert oc.fp4_decode(codes, np.array([[code]], dtype=np.uint8)).tolist() == [[f * x for x in want]]
    assert np.isnan(oc.fp4_decode(codes, np.array([[255]], dtype=np.uint8))).all()


@pytest.mark.parametrize("top,code", [(1.0, 125), (6.0, 127), (7.99, 127), (8.0, 128), (0.0, 0), (448.0, 133)])
def test_encode_scale_is_two_below_the_largest_exponent(top, code):
    x = np.zeros(32)
    x[5] = -top
    assert oc.fp4_encode(x)[1].tolist() == [code]


def test_encode_rounds_to_nearest_even_and_saturates():
    # the block's largest value 4 gives scale 1
    x = np.array([4, .25, .26, .75, 1.25, 1.75, 2.5, 3.5, 5, 5.01, -0.2, -.25, -.75, 7.9, 0, -0.0] + [0] * 16)
    x[13] = 4.0
    nib, code = oc.fp4_encode(x)
    assert code.tolist() == [127]
    got = oc.fp4_decode((nib[0::2] | nib[1::2] << 4), code)
    assert got.tolist() == [4, 0, .5, 1, 1, 2, 2, 4, 4, 6, -0.0, -0.0, -1, 4, 0, -0.0] + [0] * 16
    x[0] = 7.9  # scale still 1, past the largest magnitude
    nib, code = oc.fp4_encode(x)
    assert code.tolist() == [127] and (nib[0] & 7) == 7


def test_encode_blocks_that_are_not_finite():
    x = np.ones(64)
    x[40] = np.inf
    nib, code = oc.fp4_encode(x)
    assert code.tolist() == [125, 255] and (nib[32:] == 0).all()


def test_a_decode_steps_weights_sum_to_its_heads():
    rng = np.random.default_rng(3)
    cache = rng.standard_normal((4, 2, 2, 8, 64))
    q = rng.standard_normal((2, 6, 64))
    ptr, idx, last = np.array([0, 3, 4]), np.array([2, 0, 3, 1]), np.array([5, 8])
    _, lse = oc.paged_decode(q, cache, ptr, idx, last, 8, 0.125)
    s = oc.attn_weights(q, cache[:, 0], lse, np.full((4, 2, 8), 7.0), np.arange(3), ptr, idx, last, 8, 0.125,
                        True, 0.0)
    assert np.allclose(s[[2, 0]].sum((0, 2)) + s[3, :, :5].sum(-1), 3.0)
    assert np.allclose(s[1].sum(-1), 3.0)
    assert (s[3, :, 5:] == 7.0).all()  # past the last token


def test_weights_decay_and_new_tokens():
    keys, q = np.zeros((1, 1, 8, 64)), np.zeros((1, 1, 64))
    lse = np.full((1, 1), np.log(4.0))
    s = oc.attn_weights(q, keys, lse, np.arange(8.0)[None, None], np.array([0, 1]), np.array([0, 1]),
                        np.array([0]), np.array([4]), 8, 1.0, True, 0.5)
    assert np.allclose(s[0, 0], [0.25, 0.75, 1.25, 0.25, 4, 5, 6, 7])


def test_evict_kept():
    nan, inf = float("nan"), float("inf")
    assert oc.evict_kept([5, 1, nan, 1, -inf, 0.0, -0.0, 9], 8, 4, 1, 1) == [0, 1, 2, 7]
    assert oc.evict_kept([0.0, -0.0, 0.0, -0.0], 4, 2, 0, 0) == [0, 1]
    assert oc.evict_kept([1, 2], 2, 5, 9, 9) == [0, 1]
    assert oc.evict_kept([1, 2, 3], 3, 0, 0, 0) == []
