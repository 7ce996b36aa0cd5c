"""Bounds of blocks and the choice by them: exactly the definition's."""

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
from blocks_util import batch, lists, pages_of, to64
from oracle import blocks as ob

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


# ---- bounds ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens,new,ps,hkv,d,dtype", [
    ([1], [1], 16, 1, 128, BF), ([700, 33, 16], [1, 1, 1], 16, 8, 128, BF), ([100, 7, 64], [100, 7, 40], 8, 3, 64, FP),
    ([130, 2], [130, 2], 48, 9, 128, FP), ([129, 300], [5, 300], 64, 2, 64, BF), ([50] * 200, [50] * 200, 16, 2, 64, BF),
])
@pytest.mark.parametrize("order", ["rows", "mixed"])
def test_bounds_of_touched_pages(cuda, lens, new, ps, hkv, d, dtype, order):
    g = torch.Generator().manual_seed(1)
    s = batch(lens, new, ps, 2)
    if order == "mixed":
        perm = torch.randperm(sum(new), generator=g)
        s["req"], s["pos"] = s["req"][perm], s["pos"][perm]
    cache = torch.randn(s["pages"], 2, hkv, ps, d, generator=g).to(dtype)
    want = torch.randn(s["pages"], hkv, 2, d, generator=g).to(dtype)
    bounds = want.to(cuda)
    for b, n in enumerate(lens):  # slots past the end may hold anything
        if n % ps:
            cache[pages_of(s, b)[-1], :, :, n % ps:] = float("nan")
    c64 = to64(cache)
    for b, (n, m) in enumerate(zip(lens, new)):
        for j in range((n - m) // ps, -(-n // ps)):
            p = pages_of(s, b)[j]
            want[p] = torch.tensor(ob.block_bounds(c64, p, min(ps, n - j * ps))).to(dtype)
    got = bskv.bskv_block_bounds_paged(cache.to(cuda), bounds, *lists(s, cuda), s["last"].to(cuda))
    assert got is bounds and torch.equal(bounds.cpu(), want)
    assert bskv.bskv_get_device_status() == 0


def test_bounds_strides_nan_and_rows_without_a_token(cuda):
    g = torch.Generator().manual_seed(3)
    s = batch([20, 40], [20, 40], 16, 4)
    cache = torch.randn(s["pages"], 2, 2, 16, 128, generator=g).to(BF)
    first = pages_of(s, 0)[0]
    cache[first, 0, 1, 3, 5] = float("nan")
    cache[first, 0, 0, 2, 7] = float("inf")
    other = cache.permute(1, 0, 3, 2, 4).contiguous().to(cuda).permute(1, 0, 3, 2, 4)
    wide = torch.zeros(s["pages"], 2, 2, 256, dtype=BF, device=cuda)
    bounds = wide.view(s["pages"], 2, 4, 128)[:, :, 1:3]
    req, pos, indptr, indices = lists(s, cuda)
    req[20:40] = -1  # the second request's first pages and some of its second
    req[40:52] = -1
    bskv.bskv_block_bounds_paged(other, bounds, req, pos, indptr, indices, s["last"].to(cuda))
    got = bounds.cpu()
    assert got[first, 1, :, 5].isnan().all() and got[first, 0, 1, 7] == float("inf")
    assert not got[first, 1, :, 6].isnan().any()
    assert (got[pages_of(s, 1)[0]] == 0).all() and (got[pages_of(s, 1)[1]] == 0).all()
    k = cache[pages_of(s, 1)[2], 0, :, :8]
    assert torch.equal(got[pages_of(s, 1)[2]], torch.stack([k.amin(1), k.amax(1)], 1))
    assert (wide.view(s["pages"], 2, 4, 128)[:, :, [0, 3]] == 0).all()
    assert bskv.bskv_get_device_status() == 0


@pytest.mark.parametrize("bad", ["request", "position", "negative", "page", "last"])
def test_bounds_rows_out_of_range(cuda, bad):
    s = batch([20, 40], [1, 1], 16, 4)
    cache = torch.randn(s["pages"], 2, 2, 16, 64).to(BF)
    bounds = torch.zeros(s["pages"], 2, 2, 64, dtype=BF, device=cuda)
    req, pos, indptr, indices = lists(s, cuda)
    last = s["last"].to(cuda)
    if bad == "request":
        req[0] = 2
    elif bad == "position":
        pos[0] = 32
    elif bad == "negative":
        pos[0] = -1
    elif bad == "page":
        indices[1] = -1
    else:
        last[0] = 17
    bskv.bskv_block_bounds_paged(cache.to(cuda), bounds, req, pos, indptr, indices, last)
    assert bskv.bskv_get_device_status() == 6
    touched = (bounds != 0).any(-1).any(-1).any(-1).nonzero()[:, 0].tolist()
    assert touched == [pages_of(s, 1)[2]]


# ---- selection ------------------------------------------------------------------------

def _select_inputs(lens, new, ps, hq, hkv, d, dtype, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    s = batch(lens, new, ps, seed)
    q = torch.randn(sum(new), hq, d, generator=g)
    mid, half = torch.randn(s["pages"], hkv, d, generator=g), torch.rand(s["pages"], hkv, d, generator=g) * 2
    if kind == "few values":   # many equal scores
        q, mid, half = q.round(), torch.randint(-1, 2, mid.shape, generator=g).float(), torch.zeros_like(half)
    elif kind == "equal":      # all scores of a row equal and not zero
        mid, half = mid[:1].expand_as(mid), half[:1].expand_as(half)
    elif kind == "near":       # scores that differ in what fp32 sums lose
        mid = mid[:1] * 64 + 0 * mid
        half = half[:1] * 64 + 0 * half
        mid = mid.to(dtype).float().expand(s["pages"], -1, -1).clone()
        mid[:, :, d // 2] += torch.randint(0, 2, mid[:, :, 0].shape, generator=g) * 2.0 ** -12
        half = half.to(dtype).float()
        q[:, :, d // 2] = 1.0
    elif kind == "zero":
        q = torch.zeros_like(q)
    bounds = torch.stack([(mid - half).to(dtype), (mid + half).to(dtype)], 2)
    if kind == "near":  # one channel holds the difference exactly
        bounds[:, :, :, d // 2] = ((mid[:, :, d // 2] * 4096).round().remainder(2.0) * 2.0 ** -12)[:, :, None].to(dtype)
    if kind == "not numbers":
        bounds.view(-1)[torch.randint(0, bounds.numel(), (bounds.numel() // (40 * d),), generator=g)] = float("nan")
        bounds.view(-1)[torch.randint(0, bounds.numel(), (bounds.numel() // (20 * d),), generator=g)] = float("inf")
        bounds.view(-1)[torch.randint(0, bounds.numel(), (bounds.numel() // (20 * d),), generator=g)] = float("-inf")
    s.update(q=q.to(dtype), bounds=bounds)
    return s


def _expect(s, hkv, top, sink, recent):
    q, bounds = to64(s["q"]), to64(s["bounds"])
    n, hq, d = q.shape
    out = np.full((n, hkv, top), -1, dtype=np.int32)
    for t in range(n):
        pages = pages_of(s, int(s["req"][t]))[:int(s["pos"][t]) // s["ps"] + 1]
        for h in range(hkv):
            score = ob.block_scores(q[t].reshape(hkv, -1, d)[h], bounds[pages, h])
            out[t, h] = ob.select(score, top, sink, recent)
    return out


def _plan(s, hq, hkv, d, top, sink, recent, dtype, **k):
    most = max([-(-n // s["ps"]) for n in s["lens"]], default=1)
    return bskv.bskv_plan_decode_blocks(s["q"].shape[0], most, s["pages"], s["ps"], hq, hkv, d, top, sink, recent, dtype, **k)


SELECT = [
    ([700, 1, 33, 160], [1, 1, 1, 1], 16, 8, 2, 128, 4, 1, 2, BF),
    ([20000], [1], 16, 4, 1, 128, 64, 1, 8, BF),
    ([3000], [3], 8, 6, 1, 64, 50, 0, 1, FP),
    ([1025, 2000, 64], [4, 2, 1], 8, 24, 4, 64, 16, 2, 3, FP),
    ([5000, 4999], [1, 1], 16, 32, 2, 128, 100, 0, 1, BF),
    ([4000] * 40, [1] * 40, 48, 8, 8, 64, 7, 0, 7, BF),
    ([4000] * 40, [1] * 40, 32, 16, 8, 128, 31, 3, 4, BF),
    ([900], [1], 16, 3, 3, 64, 1, 0, 1, FP),
    ([1000], [1], 16, 1, 1, 128, 62, 0, 1, FP),
]


@pytest.mark.parametrize("case", range(len(SELECT)))
@pytest.mark.parametrize("kind", ["normal", "few values", "equal", "near", "zero", "not numbers"])
def test_selection(cuda, case, kind):
    lens, new, ps, hq, hkv, d, top, sink, recent, dtype = SELECT[case]
    s = _select_inputs(lens, new, ps, hq, hkv, d, dtype, case, kind)
    p = _plan(s, hq, hkv, d, top, sink, recent, dtype)
    want = _expect(s, hkv, top, sink, recent)
    q, bounds = s["q"].to(cuda), s["bounds"].to(cuda)
    for _ in range(2):  # the counters are ready again
        got = bskv.bskv_run_select_blocks(p, q, bounds, *lists(s, cuda))
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert bskv.bskv_get_device_status() == 0


def test_selection_of_many_blocks(cuda):
    """As many blocks as a plan takes: all of shared memory, several scoring parts of a row."""
    lens, ps, d, top = [49152 * 8 - 3], 8, 64, 300
    s = _select_inputs(lens, [1], ps, 2, 1, d, BF, 5)
    p = bskv.bskv_plan_decode_blocks(1, 49152, s["pages"], ps, 2, 1, d, top, 1, 1, BF)
    got = bskv.bskv_run_select_blocks(p, s["q"].to(cuda), s["bounds"].to(cuda), *lists(s, cuda))
    np.testing.assert_array_equal(got.cpu().numpy(), _expect(s, 1, top, 1, 1))


def test_selection_strides_and_rows_without_a_token(cuda):
    lens, new, ps, hq, hkv, d, top, sink, recent, dtype = SELECT[3]
    s = _select_inputs(lens, new, ps, hq, hkv, d, dtype, 7)
    p = _plan(s, hq, hkv, d, top, sink, recent, dtype)
    req, pos, indptr, indices = lists(s, cuda)
    req[2] = -1
    pos[2] = -1
    q = torch.zeros(hq, 2 * len(pos), d, dtype=dtype, device=cuda)[:, ::2].transpose(0, 1)
    q.copy_(s["q"])
    bounds = s["bounds"].transpose(0, 1).contiguous().to(cuda).transpose(0, 1)
    blocks = torch.full((len(pos), hkv, top), -5, dtype=torch.int32, device=cuda)
    got = bskv.bskv_run_select_blocks(p, q, bounds, req, pos, indptr, indices, blocks=blocks)
    want = _expect(s, hkv, top, sink, recent)
    want[2] = -5
    assert got is blocks
    np.testing.assert_array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("bad", ["request", "position", "negative", "long", "page"])
def test_selection_rows_out_of_range(cuda, bad):
    lens, new, ps, hq, hkv, d, top, sink, recent, dtype = SELECT[0]
    s = _select_inputs(lens, new, ps, hq, hkv, d, dtype, 8)
    p = _plan(s, hq, hkv, d, top, sink, recent, dtype)
    if bad == "long":
        p = bskv.bskv_plan_decode_blocks(4, 43, s["pages"], ps, hq, hkv, d, top, sink, recent, dtype)
    req, pos, indptr, indices = lists(s, cuda)
    if bad == "request":
        req[0] = 4
    elif bad == "position":
        pos[0] = 704
    elif bad == "negative":
        pos[0] = -1
    elif bad == "page":
        indices[7] = s["pages"]
    want = _expect(s, hkv, top, sink, recent)
    got = bskv.bskv_run_select_blocks(p, s["q"].to(cuda), s["bounds"].to(cuda), req, pos, indptr, indices).cpu().numpy()
    assert bskv.bskv_get_device_status() == 6
    np.testing.assert_array_equal(got[1:], want[1:])
    if bad == "page":
        s["bounds"][pages_of(s, 0)[7]] = 0
        q, b = to64(s["q"][0]), to64(s["bounds"])
        for h in range(hkv):
            score = ob.block_scores(q.reshape(hkv, -1, d)[h], b[pages_of(s, 0), h])
            score[7] = -np.inf
            assert got[0, h].tolist() == ob.select(score, top, sink, recent)
    else:
        assert (got[0] == -1).all()
