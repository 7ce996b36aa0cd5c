"""4-bit decode where weights and value scales leave the ordinary range: values of zero, blocks of
zeros under any scale, and scales up to the format's end.

Gate, from the arithmetic. As in the ordinary cases a weight times scale is rounded once to f16 (2^-11
of it) and the output once to its type, with fp32 sums and ex2 within 2^-12 of A = sum_j w_j |v_j|.
Below f16's normal range a product is off by up to 2^-25 in the kernel's unit. That unit puts the
largest product M of the head at 2^10 or more (M counts the blocks that hold a value other than zero:
a block of zeros gives nothing whatever its scale), unless tokens of zeros outweigh it by more than 2^84: then the
largest weight stands at 2^94. So each of the L products is off by 2^-35 M + 2^-119 at most, and its
value's code is at most 6. The lse carries the fp32 rounding of logits of its size: 2^-18 (1 + |lse|).
"""

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
from oracle import cache as oc
from gpu_util import to64

pytestmark = pytest.mark.gpu
PS = 16


def _split(v):
    """v >= 0 as a sum of numbers 1 or 1.5 times a power of two: (E2M1 code, scale code) each."""
    parts = []
    while v > 0:
        e = int(np.floor(np.log2(v)))
        big = v >= 1.5 * 2.0 ** e
        parts.append((3 if big else 2, 127 + e))
        v -= (1.5 if big else 1.0) * 2.0 ** e
    return parts


def _keys(logits, H, D):
    """Codes and scales of keys whose products with ones at dims 0, 32, .. are the given logits."""
    codes = np.zeros((H, len(logits), D // 2), dtype=np.uint8)
    scales = np.full((H, len(logits), D // 32), 127, dtype=np.uint8)
    for v in set(logits):
        at = np.array(logits) == v
        parts = _split(v)
        assert len(parts) <= D // 32
        for i, (code, scale) in enumerate(parts):
            codes[:, at, 16 * i] = code
            scales[:, at, i] = scale
    return codes, scales


def _check(cuda, lens, codes, scales, q, sm, workers):
    """Runs the decode over codes[b] [2, H, L, D / 2], scales[b] [2, H, L, D / 32] and q [B, Hq, D]."""
    B, Hq, D = q.shape
    H = codes[0].shape[1]
    n = [-(-x // PS) for x in lens]
    indptr = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32)
    pages = sum(n) + 1
    indices = torch.randperm(pages, generator=torch.Generator().manual_seed(1))[:sum(n)].to(torch.int32)
    last = torch.tensor([x - (c - 1) * PS for x, c in zip(lens, n)], dtype=torch.int32)
    pc = np.zeros((pages, 2, H, PS, D // 2), dtype=np.uint8)
    px = np.full((pages, 2, H, PS, D // 32), 255, dtype=np.uint8)
    for b, L in enumerate(lens):
        t = np.arange(L)
        at = indices.numpy()[int(indptr[b]) + t // PS]
        pc[at, :, :, t % PS] = np.moveaxis(codes[b], 2, 0)
        px[at, :, :, t % PS] = np.moveaxis(scales[b], 2, 0)
    p = bskv.bskv_plan_decode_fp4(indptr, indices, last, pages, PS, Hq, H, D, q.dtype, max_workers=workers)
    out, lse = bskv.bskv_run_decode_fp4(p, q.to(cuda), torch.from_numpy(pc).to(cuda), torch.from_numpy(px).to(cuda),
                                        return_lse=True, sm_scale=sm)
    out, lse = to64(out), lse.cpu().double().numpy()
    half, least = (2.0 ** -8, 2.0 ** -134) if q.dtype == torch.bfloat16 else (2.0 ** -11, 2.0 ** -25)
    for b, L in enumerate(lens):
        for h in range(Hq):
            kv = h // (Hq // H)
            k, v = (oc.fp4_decode(codes[b][i, kv], scales[b][i, kv]) for i in (0, 1))
            s = sm * (k @ q[b, h].double().numpy())
            m = s.max()
            w = np.exp(s - m)
            z = m + np.log(w.sum())
            w /= w.sum()
            lives = ((codes[b][1, kv] & 0x77).reshape(L, D // 32, 16) != 0).any(-1)
            M = (w[:, None] * np.ldexp(1.0, scales[b][1, kv].astype(np.int64) - 127) * lives).max()
            want, size = w @ v, w @ np.abs(v)
            tol = (2.0 ** -11 + 2.0 ** -12) * size + 6 * L * (2.0 ** -35 * M + 2.0 ** -119) + half * np.abs(want) + least
            err = np.abs(out[b, h] - want)
            assert (err <= tol).all(), (b, h, (err / tol).max(), out[b, h][:3], want[:3])
            assert abs(lse[b, h] - z) <= 2.0 ** -18 * (1 + abs(z)), (b, h, lse[b, h], z)
    assert bskv.bskv_get_device_status() == 0


def _ones(B, Hq, H, D, dtype):
    """Queries of ones at dims 0, 32, ..; a group's second head has twos, its third halves."""
    q = torch.zeros(B, Hq, D, dtype=dtype)
    g = Hq // H
    for h in range(Hq):
        q[:, h, ::32] = {1: 2.0, 2: 0.5}.get(h % g, 1.0)
    return q


def _values(seed, H, L, D, lo=118, hi=126):
    g = np.random.default_rng(seed)
    return (g.integers(0, 256, (H, L, D // 2), dtype=np.uint8),
            g.integers(lo, hi, (H, L, D // 32)).astype(np.uint8))


@pytest.mark.parametrize("workers", [1, 7])
@pytest.mark.parametrize("Hq, D, dtype", [(8, 128, torch.bfloat16), (16, 64, torch.float16), (32, 128, torch.bfloat16)])
@pytest.mark.parametrize("rise", [8, 12, 19, 25])
def test_values_of_zero_and_rising_logits(cuda, rise, Hq, D, dtype, workers):
    """A kv head whose values are zero (scale code 0, as the append writes them): outputs of zero and the
    log-sum-exp of its logits, which rise after the first tile; the other head has values."""
    L, H = 4200, 2
    kc, ks = _keys([0.0] * 32 + [float(rise)] * (L - 32), H, D)
    vc, vs = _values(11, H, L, D)
    vc[1], vs[1] = 0, 0
    _check(cuda, [L], [np.stack([kc, vc])], [np.stack([ks, vs])], _ones(1, Hq, H, D, dtype), 1.0, workers)


def test_values_of_zero_over_a_long_context(cuda):
    L, D = 131104, 64
    kc, ks = _keys([0.0] * 32 + [8.0] * (L - 32), 1, D)
    _check(cuda, [L], [np.stack([kc, kc * 0])], [np.stack([ks, ks * 0])], _ones(1, 4, 1, D, torch.bfloat16), 1.0, 1)


@pytest.mark.parametrize("workers", [1, 5])
@pytest.mark.parametrize("Hq", [4, 8, 16])
@pytest.mark.parametrize("rise", [40, 80, 144])
def test_values_of_zero_behind_ordinary_ones(cuda, rise, Hq, workers):
    """Tokens of zeros that outweigh the ordinary ones before them, and ordinary ones of theirs again."""
    L, D = 700, 128
    kc, ks = _keys([0.0] * 200 + [float(rise)] * (L - 200), 1, D)
    vc, vs = _values(12, 1, L, D)
    vc[:, 200:600], vs[:, 200:600] = 0, 0
    for end in (600, L):  # without and with the last ordinary ones
        _check(cuda, [end], [np.stack([kc, vc])[:, :, :end]], [np.stack([ks, vs])[:, :, :end]],
               _ones(1, Hq, 1, D, torch.bfloat16), 1.0, workers)


@pytest.mark.parametrize("workers", [1, 4])
@pytest.mark.parametrize("Hq", [4, 8, 16])
@pytest.mark.parametrize("scale", [160, 250])
def test_blocks_of_zeros_under_large_scales(cuda, scale, Hq, workers):
    """Blocks of zeros, of either sign, whose scale is far above that of the values beside them."""
    L, D = 500, 128
    g = np.random.default_rng(13)
    kc, ks = _values(14, 1, L, D, 120, 123)
    vc, vs = _values(15, 1, L, D)
    zero = g.random(vs.shape) < 0.3
    zero[:, :40] = False
    zero[0, 20, 1] = zero[0, 470, 3] = True
    vs[zero] = scale
    vc.reshape(vs.shape + (16,))[zero] &= 0x88
    q = torch.from_numpy(g.standard_normal((1, Hq, D))).to(torch.bfloat16)
    _check(cuda, [L], [np.stack([kc, vc])], [np.stack([ks, vs])], q, D ** -0.5, workers)
    first = np.roll(vs, -20, 1), np.roll(vc, -20, 1)  # and on the first token
    _check(cuda, [L], [np.stack([kc, first[1]])], [np.stack([ks, first[0]])], q, D ** -0.5, workers)


@pytest.mark.parametrize("workers", [1, 4])
@pytest.mark.parametrize("Hq, D", [(4, 128), (3, 64), (8, 128), (16, 64)])
@pytest.mark.parametrize("lo, hi", [(223, 249), (100, 249), (1, 30)])
def test_values_to_the_ends_of_the_range(cuda, lo, hi, Hq, D, workers):
    """Values of 2^96 to 2^124, alone and beside ordinary ones that follow or precede them, and of
    less than 2^-96."""
    L = 500
    kc, ks = _values(16, 1, L, D, 120, 123)
    vc, vs = _values(17, 1, L, D, lo, hi)
    rows = [(vc, vs)]
    if hi > 127:
        late, early = vs.copy(), vs.copy()
        late[:, :300] = 124
        early[:, 100:] = 124
        rows += [(vc, late), (vc, early)]
    q = torch.from_numpy(np.random.default_rng(18).standard_normal((3, Hq, D))).to(torch.bfloat16)
    q[1] = 0
    q[2] *= 16
    _check(cuda, [L] * len(rows), [np.stack([kc, c]) for c, _ in rows], [np.stack([ks, s]) for _, s in rows],
           q[:len(rows)], D ** -0.5, workers)


@pytest.mark.parametrize("workers", [1, 4])
@pytest.mark.parametrize("Hq, D", [(4, 128), (8, 64), (16, 128)])
@pytest.mark.parametrize("scale", [160, 170, 200])
def test_large_values_behind_zeros(cuda, scale, Hq, D, workers):
    """Tokens of zeros, then as many of large values with the same logits: both count in the sum."""
    L = 320
    kc, ks = _keys([4.0] * L, 1, D)
    vc, vs = _values(25, 1, L, D)
    vs[:] = scale
    for zeros in (slice(0, 160), slice(32, 200), slice(100, 320)):
        c, s = vc.copy(), vs.copy()
        c[:, zeros], s[:, zeros] = 0, 0
        _check(cuda, [L], [np.stack([kc, c])], [np.stack([ks, s])], _ones(1, Hq, 1, D, torch.bfloat16), 1.0, workers)


@pytest.mark.parametrize("workers", [1, 3])
@pytest.mark.parametrize("Hq, D", [(4, 128), (8, 64), (16, 128)])
def test_large_values_that_only_some_heads_see(cuda, Hq, D, workers):
    """Tokens of values around 2^110 that weigh 2^-184 for most heads, 2^-369 and 2^-92 for one each: only
    the last one's result is theirs, the others' tokens before and after keep their 16 bits."""
    L = 700
    kc, ks = _keys([128.0] * 32 + [0.0] * 32 + [128.0] * (L - 64), 1, D)
    vc, vs = _values(24, 1, L, D)
    vs[:, 32:64] = 237
    _check(cuda, [L], [np.stack([kc, vc])], [np.stack([ks, vs])], _ones(1, Hq, 1, D, torch.bfloat16), 1.0, workers)


@pytest.mark.parametrize("Hq", [4, 8])
def test_a_scale_that_leaves_no_logits(cuda, Hq):
    """bf16 queries of zeros or near the type's smallest under a tiny sm_scale: every token weighs the
    same, and those past the end nothing."""
    L, D = 37, 128
    kc, ks = _values(19, 1, L, D)
    vc, vs = _values(20, 1, L, D)
    for size in (0.0, 1e-38):
        q = torch.full((1, Hq, D), size, dtype=torch.bfloat16)
        _check(cuda, [L], [np.stack([kc, vc])], [np.stack([ks, vs])], q, 1e-9, 1)
