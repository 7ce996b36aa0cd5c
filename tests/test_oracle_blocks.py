"""The block-sparse step's definitions against brute force and library routines."""

import numpy as np

from oracle import blocks as ob
from oracle import rope


def test_page_table_worked_example():
    table = [[7, -1, -1], [3, 4, -1], [-1, -1, -1]]
    free = [9, 8, 6]  # the last goes first
    got = ob.page_table([5, 8, 0], [2, 1, 0], table, 4, free)
    assert got == ([0, 2, 4, 4], [7, 6, 3, 4], [1, 4, 0], [0, 2, 3, 3], [0, 0, 1], [3, 4, 7],
                   [31, 24, 19])
    assert free == [9, 8] and table[0] == [7, 6, -1]


def test_scores_bound_every_key():
    rng = np.random.default_rng(0)
    k, q = rng.standard_normal((6, 16, 32)), rng.standard_normal((4, 32))
    bounds = np.stack([k.min(1), k.max(1)], 1)
    score = ob.block_scores(q, bounds)
    assert (score[:, None] >= (k @ q.T).sum(-1) - 1e-12).all()
    direct = np.maximum(q[:, None] * bounds[None, :, 0], q[:, None] * bounds[None, :, 1]).sum((0, 2))
    np.testing.assert_allclose(score, direct, rtol=1e-12)
    # a block of one token has its logits' sum
    one = np.stack([k[:, 0], k[:, 0]], 1)
    np.testing.assert_allclose(ob.block_scores(q, one), (k[:, 0] @ q.T).sum(-1), rtol=1e-12)


def test_select_order():
    s = np.array([0.0, 5.0, np.nan, 5.0, -np.inf, 5.0, np.inf, 1.0])
    assert ob.select(s, 8, 0, 1) == list(range(8))
    assert ob.select(s, 9, 0, 1) == list(range(8)) + [-1]
    assert ob.select(s, 2, 0, 1) == [2, 7]          # NaN above infinity
    assert ob.select(s, 5, 1, 1) == [0, 1, 2, 6, 7]  # the first of the equal ones
    assert ob.select(s, 3, 2, 1) == [0, 1, 7]


def test_rotation_is_the_prologue_s():
    rng = np.random.default_rng(1)
    x, t = rng.standard_normal((3, 64)), rng.standard_normal((1, 64))
    for neox in (True, False):
        y, _ = ob.norm_rope(x, None, 0.0, t[0], 64, neox)
        # a rotation by unit vectors keeps lengths; by any table it is the complex product
        one, two = (slice(0, 32), slice(32, 64)) if neox else (slice(0, 64, 2), slice(1, 64, 2))
        z = (x[:, one] + 1j * x[:, two]) * (t[0, :32] + 1j * t[0, 32:])
        np.testing.assert_allclose(y[:, one], z.real)
        np.testing.assert_allclose(y[:, two], z.imag)
    assert hasattr(rope, "mla_rope_quantize_fp8")


def test_attend_is_a_softmax():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((2, 8)), rng.standard_normal((5, 8)), rng.standard_normal((5, 8))
    out, lse, size = ob.attend(q, k, v, 0.5)
    e = np.exp(q @ k.T * 0.5)
    np.testing.assert_allclose(out, e @ v / e.sum(-1, keepdims=True))
    np.testing.assert_allclose(lse, np.log(e.sum(-1)))
    assert (size >= np.abs(out)).all()
    out, lse, _ = ob.attend(q, k[:0], v[:0], 0.5)
    assert (out == 0).all() and (lse == -np.inf).all()


def test_scores_of_infinite_bounds_are_the_sums_of_greater_products():
    """A channel whose bounds are infinite on either side or both, under queries of one sign, of both, and of zero."""
    inf = np.inf
    pairs = [(-inf, -inf), (-inf, 2.0), (-3.0, inf), (-inf, inf), (inf, inf), (1.0, 2.0)]
    bounds = np.ones((len(pairs), 2, 3))
    bounds[:, 0, 1], bounds[:, 1, 1] = [x[0] for x in pairs], [x[1] for x in pairs]
    for q1 in ([0.5], [-0.5], [0.0], [0.5, 2.0], [-0.5, -1.0], [0.5, -1.0], [0.0, 3.0]):
        q = np.full((len(q1), 3), 0.25)
        q[:, 1] = q1
        with np.errstate(invalid="ignore"):
            direct = np.maximum(q[:, None] * bounds[None, :, 0], q[:, None] * bounds[None, :, 1]).sum((0, 2))
        np.testing.assert_array_equal(ob.block_scores(q, bounds), direct)
    assert ob.block_scores(np.full((1, 3), 0.25), bounds)[0] == -inf  # no key of it can have weight
    assert ob.block_scores(np.full((1, 3), 0.25), bounds)[1] == 1.0


def test_rotation_agrees_with_the_prologue_s():
    """The rotation of 64 dims is the one that the latent rows' prologue makes of its tail."""
    rng = np.random.default_rng(3)
    x, t = rng.standard_normal((5, 64)), rng.standard_normal(64)
    for neox in (True, False):
        y, _ = ob.norm_rope(x, None, 0.0, t, 64, neox)
        np.testing.assert_allclose(y, rope.rotate(x, t[:32], t[32:], neox), rtol=1e-14, atol=1e-14)
