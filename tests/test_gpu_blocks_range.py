"""The block-sparse step where its numbers are hardest to hold: weights finer than 16 bits, infinite keys and bounds."""

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
from blocks_util import batch, lists, pages_of, to64
from oracle import blocks as ob

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


# ---- attention --------------------------------------------------------------------------

@pytest.mark.parametrize("group", [1, 4, 8, 9, 16])
@pytest.mark.parametrize("d,ps,dtype", [(128, 16, BF), (64, 8, BF), (128, 48, FP), (64, 16, FP)])
def test_weights_keep_more_than_16_bits(cuda, group, d, ps, dtype):
    """Against 64 bits, with queries and keys of small whole numbers: their products are exact in fp32, so what the
    weights are rounded to is the largest error but the output's own rounding."""
    lens, new, hkv = [100, 1, 37, 128, 17, 64], [1, 1, 2, 1, 1, 1], 2
    g = torch.Generator().manual_seed(group)
    s = batch(lens, new, ps, group)
    n, scale = sum(new), 1.0 / 8
    q = torch.randint(-2, 3, (n, hkv * group, d), generator=g).to(dtype)
    kv = torch.randn(s["pages"], 2, hkv, ps, d, generator=g).to(dtype)
    kv[:, 0] = torch.randint(-2, 3, kv[:, 0].shape, generator=g).to(dtype)
    most = -(-max(lens) // ps)
    blocks = torch.full((n, hkv, most), -1, dtype=torch.int32)
    for t in range(n):
        seen = int(s["pos"][t]) // ps + 1
        blocks[t, :, :seen] = torch.arange(seen, dtype=torch.int32)
    p = bskv.bskv_plan_decode_blocks(n, most, s["pages"], ps, hkv * group, hkv, d, most, dtype=dtype)
    out, lse = bskv.bskv_run_decode_blocks(p, q.to(cuda), kv.to(cuda), blocks.to(cuda), *lists(s, cuda), return_lse=True,
                                           sm_scale=scale)
    assert bskv.bskv_get_device_status() == 0
    half = torch.finfo(dtype).eps / 2
    q64, kv64 = to64(q), to64(kv)
    for t in range(n):
        pages, tokens = pages_of(s, int(s["req"][t])), np.arange(int(s["pos"][t]) + 1)
        for h in range(hkv):
            x = q64[t, h * group:(h + 1) * group]
            k, v = kv64[pages[tokens // ps], 0, h, tokens % ps], kv64[pages[tokens // ps], 1, h, tokens % ps]
            want, z, size = ob.attend(x, k, v, scale)
            # a logit is rounded with its scale, with the scale's conversion and as a difference to the maximum, the weight
            # moves by that times the largest logit; the exponentials, sums of a few tiles and the joins are fp32
            rel = (4 * np.abs(x @ k.T * scale).max(-1) + 4 * len(tokens) / 16 + 40)[:, None] * 2.0 ** -23
            # two parts of a weight miss half a step of a half step; in fp16 not less than half the least number
            parts = half * half * size + (2.0 ** -25 * np.abs(v).sum(0) if dtype == FP else 0.0)
            tol = half * np.abs(want) + (1 + half) * (rel * size + parts) + (2.0 ** -25 if dtype == FP else 0.0)
            bad = ~(np.abs(to64(out[t, h * group:(h + 1) * group]) - want) <= tol)
            assert not bad.any(), (t, h, int(bad.sum()), float((np.abs(to64(out[t, h * group:(h + 1) * group]) - want) / tol).max()))
            assert (np.abs(to64(lse[t, h * group:(h + 1) * group]) - z) <= 4 * rel[:, 0] + 2.0 ** -22 * np.abs(z)).all()


@pytest.mark.parametrize("group", [1, 8, 12])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("below", [10, 16, 18, 24])
@pytest.mark.parametrize("at", [0, 2000, 4999])
def test_many_small_weights_in_fp16(cuda, group, d, below, at):
    """One key takes nearly all weight, and 4999 others e^-below each, which 16 bits alone do not hold: they are all that
    the output has."""
    n, ps, dtype = 5000, 16, FP
    s = batch([n], [1], ps, 1)
    q = torch.zeros(1, group, d, dtype=dtype)
    q[:, :, 0] = 1.0
    kv = torch.zeros(s["pages"], 2, 1, ps, d, dtype=dtype)
    kv[:, 1] = 1024.0
    page = pages_of(s, 0)[at // ps]
    kv[page, 0, 0, at % ps, 0], kv[page, 1, 0, at % ps] = float(below), 0.0
    most = -(-n // ps)
    p = bskv.bskv_plan_decode_blocks(1, most, s["pages"], ps, group, 1, d, most, dtype=dtype)
    blocks = torch.arange(most, dtype=torch.int32).view(1, 1, most).to(cuda)
    out, lse = bskv.bskv_run_decode_blocks(p, q.to(cuda), kv.to(cuda), blocks, *lists(s, cuda), return_lse=True, sm_scale=1.0)
    w = np.exp(-float(below))
    want, z = 1024.0 * (n - 1) * w / (1 + (n - 1) * w), below + np.log1p((n - 1) * w)
    # the output's rounding; the logit with its factor of log2 e, the exponentials and sums of 313 tiles; what a
    # weight loses, half of 2^-39, for each of them
    assert (np.abs(to64(out) - want) <= (2.0 ** -11 + (4 * below + 4 * 313 + 40) * 2.0 ** -23) * want + 1024 * n * 2.0 ** -40 + 2.0 ** -25).all()
    assert (np.abs(to64(lse) - z) <= (4 * below + 4 * 313 + 40) * 2.0 ** -23 + 2.0 ** -22 * z).all()


@pytest.mark.parametrize("group", [1, 4, 8, 9, 16])
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, BF), (128, FP), (64, FP)])
def test_infinite_values_stay_infinite(cuda, group, d, dtype):
    """Values of either sign, of both and NaN among those that are attended to: the weighted sum is the same one as in 64
    bits, whatever the weights are (one key alone has a weight of one)."""
    lens, ps, hkv = [100, 1, 37, 300, 16], 16, 2
    g = torch.Generator().manual_seed(group)
    s = batch(lens, [1] * 5, ps, group)
    q = torch.randint(-2, 3, (5, hkv * group, d), generator=g).to(dtype)
    kv = torch.randn(s["pages"], 2, hkv, ps, d, generator=g).to(dtype)
    kv[:, 0] = torch.randint(-2, 3, kv[:, 0].shape, generator=g).to(dtype)
    inf = float("inf")
    for b, n in enumerate(lens):
        pages = pages_of(s, b)
        for c, at in ((3, 0), (5, n - 1), (9, n // 2), (20, n // 3), (d - 1, 0)):
            kv[pages[at // ps], 1, :, at % ps, c] = -inf if c == 9 else inf
        kv[pages[(n - 1) // ps], 1, :, (n - 1) % ps, 20] = -inf
        kv[pages[0], 1, :, 0, 40] = float("nan")
    most = 19
    blocks = torch.full((5, hkv, most), -1, dtype=torch.int32)
    for t, n in enumerate(lens):
        blocks[t, :, :-(-n // ps)] = torch.arange(-(-n // ps), dtype=torch.int32)
    p = bskv.bskv_plan_decode_blocks(5, most, s["pages"], ps, hkv * group, hkv, d, most, dtype=dtype)
    out = to64(bskv.bskv_run_decode_blocks(p, q.to(cuda), kv.to(cuda), blocks.to(cuda), *lists(s, cuda), sm_scale=1 / 32))
    assert bskv.bskv_get_device_status() == 0
    q64, kv64, half = to64(q), to64(kv), torch.finfo(dtype).eps / 2
    for t, n in enumerate(lens):
        tokens = np.arange(n)
        for h in range(hkv):
            r = slice(h * group, (h + 1) * group)
            pages = pages_of(s, t)[tokens // ps]
            with np.errstate(invalid="ignore"):
                want, _, size = ob.attend(q64[t, r], kv64[pages, 0, h, tokens % ps], kv64[pages, 1, h, tokens % ps], 1 / 32)
            fine = np.isfinite(want)
            assert (~fine).any()
            np.testing.assert_array_equal(out[t, r][~fine], want[~fine])
            # finite channels: the output's rounding, and logits of a few units in fp32
            assert (np.abs(out[t, r][fine] - want[fine]) <= (half * np.abs(want) + 2.0 ** -14 * size)[fine] + 2.0 ** -24).all()


# ---- the choice -------------------------------------------------------------------------

KINDS = ["masked", "lower", "upper", "one sign", "zero", "query", "near", "lost page"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("blocks,ps,hkv,group,d,dtype", [(60, 16, 2, 1, 128, BF), (300, 8, 1, 3, 64, FP), (2500, 8, 1, 2, 64, BF),
                                                        (2100, 8, 1, 1, 128, FP)])
def test_choice_by_infinite_bounds(cuda, kind, blocks, ps, hkv, group, d, dtype):
    """Bounds of keys that are infinite, by which the choice is still that of the sum of max(q lo, q hi)."""
    g = torch.Generator().manual_seed(len(kind))
    lens, new, top, sink, recent = [blocks * ps - 3, 5 * ps], [2, 1], 20, 1, 2
    s = batch(lens, new, ps, 3)
    n, hq = sum(new), hkv * group
    kv = torch.randn(s["pages"], 2, hkv, ps, d, generator=g).to(dtype)
    q = torch.randn(n, hq, d, generator=g).to(dtype)
    row = pages_of(s, 0)
    pick = lambda m: torch.tensor(row[torch.randperm(blocks - 4, generator=g)[:m].numpy() + 1])  # noqa: E731
    q[:, :, 7] = q[:, :, 7].abs() + 0.5
    q[:, :, 9] = -q[:, :, 9].abs() - 0.5
    inf = float("inf")
    if kind == "near":  # most blocks differ in what fp32 sums lose
        kv[:, 0] = kv[row[0], 0, :, :1].expand_as(kv[:, 0]).clone() * 64
        kv[:, 0, :, 0, d // 2] = (torch.randint(0, 2, kv[:, 0, :, 0, 0].shape, generator=g) * 2.0 ** -12).to(dtype)
        kv[:, 0, :, 1:, d // 2] = 0
        q[:, :, d // 2] = 1.0
    if kind == "masked":  # every key of a block, as a mask does; most blocks of the row, or a few
        kv[pick(blocks - 4 - (top // 2 if d == 64 else 2 * top)), 0, :, :, 7] = -inf
    if kind in ("lower", "near", "one sign", "lost page"):  # a key only: the block counts by its others
        kv[pick(blocks // 3), 0, :, 2, 7] = -inf
    if kind in ("upper", "one sign", "lost page"):
        kv[pick(blocks // 3), 0, :, 2, 9] = inf
    if kind == "one sign":  # some heads the other way: the score is infinite
        q[1, ::2, 7] = -1.0
        q[1, :, 9] = -1.0
        kv[pick(5), 0, :, 1, 9] = -inf
    if kind == "zero":  # a product with zero is not a number
        q[0, 0, 7] = 0.0
        q[1, :, 7] = -0.0
        kv[pick(top // 2), 0, :, 3, 7] = -inf
    if kind == "query":
        q[0, 0, 11] = inf
        q[1, 0, 11] = float("nan")
    cache, bounds = kv.to(cuda), torch.zeros(s["pages"], hkv, 2, d, dtype=dtype, device=cuda)
    whole = batch(lens, lens, ps, 3)
    bskv.bskv_block_bounds_paged(cache, bounds, *lists(whole, cuda), s["last"].to(cuda))
    assert bskv.bskv_get_device_status() == 0
    b64, q64 = to64(bounds), to64(q)
    req, pos, indptr, indices = lists(s, cuda)
    lost = []
    if kind == "lost page":
        lost = [3, 4, blocks // 2]
        indices[lost] = s["pages"]
    p = bskv.bskv_plan_decode_blocks(n, blocks, s["pages"], ps, hq, hkv, d, top, sink, recent, dtype)
    for _ in range(2):
        got = bskv.bskv_run_select_blocks(p, q.to(cuda), bounds, req, pos, indptr, indices).cpu().numpy()
        assert bskv.bskv_get_device_status() == (6 if lost else 0)
        for t in range(n):
            pages = pages_of(s, int(s["req"][t]))[:int(s["pos"][t]) // ps + 1]
            for h in range(hkv):
                x = q64[t, h * group:(h + 1) * group]
                score = ob.block_scores(x, b64[pages, h])
                with np.errstate(invalid="ignore"):
                    direct = np.maximum(x[:, None] * b64[None, pages, h, 0], x[:, None] * b64[None, pages, h, 1]).sum((0, 2))
                if kind != "query":  # there a product of infinity and zero may stand beside the greater one
                    np.testing.assert_allclose(score, direct, rtol=1e-12, atol=1e-9)
                if int(s["req"][t]) == 0:
                    score[lost] = -np.inf
                assert got[t, h].tolist() == ob.select(score, top, sink, recent), (t, h)


@pytest.mark.parametrize("d,dtype", [(64, BF), (128, FP)])
@pytest.mark.parametrize("group", [1, 2, 3, 8])
def test_choice_by_bounds_that_are_infinite_anywhere(cuda, group, d, dtype):
    """Infinite bounds of both signs in random places of rows of 40 and of 2300 blocks, under heads whose query values are
    above, below and zero in the same channel."""
    inf, ps, hkv, top = float("inf"), 8, 2, 12
    for seed in range(6):
        g = torch.Generator().manual_seed(seed)
        s = batch([2300 * ps, 40 * ps, 700 * ps], [1, 2, 1], ps, seed)
        n = sum(s["new"])
        q = torch.randn(n, hkv * group, d, generator=g)
        q[torch.rand(q.shape, generator=g) < (0.0, 0.02, 0.3)[seed % 3]] = 0.0
        if seed % 2:
            q = q.abs()
        q = q.to(dtype)
        bounds = torch.randn(s["pages"], hkv, 2, d, generator=g).sort(2).values.to(dtype)
        lo, hi = bounds[:, :, 0], bounds[:, :, 1]
        for x, value in ((lo, -inf), (hi, inf)):
            x[torch.rand(x.shape, generator=g) < 0.002] = value
        for value in (-inf, inf):
            both = torch.rand(lo.shape, generator=g) < 0.002
            lo[both], hi[both] = value, value
        p = bskv.bskv_plan_decode_blocks(n, 2300, s["pages"], ps, hkv * group, hkv, d, top, 1, 2, dtype)
        got = bskv.bskv_run_select_blocks(p, q.to(cuda), bounds.to(cuda), *lists(s, cuda)).cpu().numpy()
        assert bskv.bskv_get_device_status() == 0
        q64, b64 = to64(q), to64(bounds)
        for t in range(n):
            pages = pages_of(s, int(s["req"][t]))[:int(s["pos"][t]) // ps + 1]
            for h in range(hkv):
                score = ob.block_scores(q64[t, h * group:(h + 1) * group], b64[pages, h])
                assert got[t, h].tolist() == ob.select(score, top, 1, 2), (seed, t, h)


@pytest.mark.parametrize("bad", ["first", "last", "short row", "scored", "unseen", "no token"])
@pytest.mark.parametrize("top,hkv", [(12, 2), (3, 3)])  # with 3 there is no choice: the first and the last are all
def test_pages_out_of_range_are_reported(cuda, bad, top, hkv):
    """Whether a block is listed by its place or competes by its score."""
    g = torch.Generator().manual_seed(7)
    ps, d, sink, recent = 16, 64, 1, 2
    s = batch([640, 100, 640], [1, 2, 1], ps, 1)
    s["pos"][3] = 299  # sees 19 of 40 blocks
    req, pos, indptr, indices = lists(s, cuda)
    at = {"first": 0, "last": 38, "short row": 40 + 5, "scored": 20, "unseen": 47 + 30, "no token": 41}[bad]
    n = 4
    if bad == "short row" and top == 3:
        at = 40 + 6
    if bad == "no token":
        req[1:3] = -1
    q = torch.randn(n, 2 * hkv, d, generator=g).to(BF)
    bounds = torch.randn(s["pages"], hkv, 2, d, generator=g).sort(2).values.to(BF)
    p = bskv.bskv_plan_decode_blocks(n, 40, s["pages"], ps, 2 * hkv, hkv, d, top, sink, recent, BF)
    want = bskv.bskv_run_select_blocks(p, q.to(cuda), bounds.to(cuda), req, pos, indptr, indices)
    assert bskv.bskv_get_device_status() == 0
    for value in (s["pages"], -1):
        indices[at] = value
        got = bskv.bskv_run_select_blocks(p, q.to(cuda), bounds.to(cuda), req, pos, indptr, indices)
        # a block that neither competes nor is listed is not looked at
        assert bskv.bskv_get_device_status() == (0 if bad in ("unseen", "no token") or (bad == "scored" and top == 3) else 6)
        live = (req >= 0).nonzero()[:, 0]
        if bad != "scored":
            assert torch.equal(got[live], want[live])
        else:
            assert top == 3 or not (got[0] == at).any()


@pytest.mark.parametrize("kind", ["normal", "near"])
def test_choice_in_slices_by_memory(cuda, kind):
    """A plan for long requests has room for the scores of 85 queries at a time; 301 of several requests, some without
    a token, with scores that fp32 orders and with ones that it does not."""
    g = torch.Generator().manual_seed(2)
    ps, hkv, d, top, sink, recent = 8, 4, 64, 30, 1, 2
    lens, new = [1600, 40, 900, 2, 1601], [100, 20, 81, 1, 99]
    s = batch(lens, new, ps, 4)
    n = sum(new)
    kv = torch.randn(s["pages"], 2, hkv, ps, d, generator=g).to(BF)
    q = torch.randn(n, hkv, d, generator=g).to(BF)
    if kind == "near":
        kv[:, 0] = kv[:1, 0, :, :1].expand_as(kv[:, 0]).clone() * 64
        kv[:, 0, :, 0, d // 2] = (torch.randint(0, 2, kv[:, 0, :, 0, 0].shape, generator=g) * 2.0 ** -12).to(BF)
        kv[:, 0, :, 1:, d // 2] = 0
        q[:, :, d // 2] = 1.0
    bounds = torch.zeros(s["pages"], hkv, 2, d, dtype=BF, device=cuda)
    bskv.bskv_block_bounds_paged(kv.to(cuda), bounds, *lists(batch(lens, lens, ps, 4), cuda), s["last"].to(cuda))
    req, pos, indptr, indices = lists(s, cuda)
    gone = list(range(80, 95)) + [n - 1]
    req[gone] = -1
    blocks = torch.full((n, hkv, top), -9, dtype=torch.int32, device=cuda)
    p = bskv.bskv_plan_decode_blocks(n, 49152, s["pages"], ps, hkv, hkv, d, top, sink, recent, BF)
    bskv.bskv_run_select_blocks(p, q.to(cuda), bounds, req, pos, indptr, indices, blocks=blocks)
    assert bskv.bskv_get_device_status() == 0
    b64, q64, got = to64(bounds), to64(q), blocks.tolist()
    for t in range(n):
        pages = pages_of(s, int(s["req"][t]))[:int(s["pos"][t]) // ps + 1]
        for h in range(hkv):
            want = [-9] * top if t in gone else ob.select(ob.block_scores(q64[t, h:h + 1], b64[pages, h]), top, sink, recent)
            assert got[t][h] == want, (t, h)


# ---- both -------------------------------------------------------------------------------

def test_shared_pages_give_what_the_definition_gives(cuda):
    """Requests that list the same pages and a row that comes twice: each is the definition's, and nothing is reported."""
    ps, hq, hkv, d, top = 16, 4, 2, 64, 3
    s = batch([100], [1], ps, 3)
    pages = pages_of(s, 0)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    where = i32([0, 1, 0, 1]), i32([99, 99, 99, 63]), i32([0, 7, 14]), i32(pages.tolist() * 2)
    g = torch.Generator().manual_seed(3)
    kv = torch.randn(s["pages"], 2, hkv, ps, d, generator=g).to(BF)
    q = torch.randn(2, hq, d, generator=g).to(BF)[[0, 0, 0, 1]]
    bounds = torch.zeros(s["pages"], hkv, 2, d, dtype=BF, device=cuda)
    bskv.bskv_block_bounds_paged(kv.to(cuda), bounds, *lists(batch([100], [100], ps, 3), cuda), s["last"].to(cuda))
    p = bskv.bskv_plan_decode_blocks(4, 7, s["pages"], ps, hq, hkv, d, top, dtype=BF)
    blocks = bskv.bskv_run_select_blocks(p, q.to(cuda), bounds, *where)
    out, lse = bskv.bskv_run_decode_blocks(p, q.to(cuda), kv.to(cuda), blocks, *where, return_lse=True)
    assert bskv.bskv_get_device_status() == 0
    q64, kv64, b64 = to64(q), to64(kv), to64(bounds)
    for t, pos in enumerate([99, 99, 99, 63]):
        for h in range(hkv):
            x = q64[t, 2 * h:2 * h + 2]
            want = ob.select(ob.block_scores(x, b64[pages[:pos // ps + 1], h]), top, 0, 1)
            assert blocks[t, h].tolist() == want
            at = np.array([j for c in want for j in range(c * ps, min(pos + 1, (c + 1) * ps))])
            k, v = kv64[pages[at // ps], 0, h, at % ps], kv64[pages[at // ps], 1, h, at % ps]
            ref, z, size = ob.attend(x, k, v, d ** -0.5)
            # a logit is off by 64 + 8 roundings of the sum of its terms' sizes, a weight by twice that
            err = (np.abs(x) @ np.abs(k).T).max(-1) * d ** -0.5 * 72 * 2.0 ** -24
            tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (2 * err[:, None] + 2.0 ** -15) * size
            assert (np.abs(to64(out[t, 2 * h:2 * h + 2]) - ref) <= tol).all()
            assert (np.abs(to64(lse[t, 2 * h:2 * h + 2]) - z) <= err + 2.0 ** -18 + 2.0 ** -22 * np.abs(z)).all()
