"""Normalised and rotated rows and the 16-bit append against the float64 definition."""

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
from blocks_util import batch, lists, to64
from oracle import blocks as ob

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def _close(got, ref, size, dtype):
    """One rounding to dtype of a value whose fp32 steps (a sum of up to 128 squares, a root, a quotient, three
    products and a sum, 2^-24 each, the sum's terms joined in chains and trees of at most 12) are off by less than 32
    steps of the terms' size; and half of the least step below dtype's normal numbers."""
    tiny = 2.0 ** -25 if dtype == FP else 2.0 ** -134
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + 33 * 2.0 ** -24 * size + tiny
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])


CASES = [
    # lens, new, page, hq, hkv, d, rot, neox, weights, dtype, table type
    ([700, 1, 33], [1, 1, 1], 16, 32, 8, 128, 128, True, (1, 1), BF, torch.float32),
    ([40, 3, 9], [40, 2, 9], 8, 24, 4, 64, 32, False, (0, 0), FP, torch.float32),
    ([17, 64], [17, 30], 16, 5, 1, 128, 48, True, (1, 0), BF, BF),
    ([17, 64], [17, 30], 48, 7, 7, 64, 16, False, (0, 1), BF, BF),
    ([20], [20], 5, 1, 1, 64, 64, True, (1, 1), FP, torch.float32),
    ([9, 1], [9, 1], 16, 40, 10, 128, 0, True, (1, 1), BF, None),
    ([300], [300], 64, 64, 8, 128, 64, False, (1, 1), FP, torch.float32),
    ([5], [5], 16, 3, 3, 128, 112, True, (0, 0), FP, torch.float32),
]


def _make(case, seed=0):
    lens, new, ps, hq, hkv, d, rot, neox, (wq, wk), dtype, table = case
    g = torch.Generator().manual_seed(seed)
    s = batch(lens, new, ps, seed)
    n = sum(new)
    rnd = lambda *sh, scale=1.0: (torch.randn(*sh, generator=g) * scale).to(dtype)  # noqa: E731
    s.update(q=rnd(n, hq, d, scale=3.0), k=rnd(n, hkv, d, scale=0.1), v=rnd(n, hkv, d),
             cache=rnd(s["pages"], 2, hkv, ps, d), wq=rnd(d) if wq else None, wk=rnd(d) if wk else None)
    s["cos_sin"] = None if table is None else torch.randn(max(lens) + 7, rot, generator=g).to(table)
    return s


def _dev(x, dev):
    return None if x is None else x.to(dev)


def _expect(s, name, w, rot, neox, at):
    x, eps = s[name], 1e-5
    ref, size = np.zeros(x.shape), np.zeros(x.shape)
    for i, row in enumerate(at):
        cs = to64(s["cos_sin"][row]) if rot else None
        ref[i], size[i] = ob.norm_rope(to64(x[i]), None if w is None else to64(w), eps, cs, rot, neox)
    return ref, size


@pytest.mark.parametrize("case", range(len(CASES)))
def test_rows_and_cache(cuda, case):
    lens, new, ps, hq, hkv, d, rot, neox, _, dtype, _ = CASES[case]
    s = _make(CASES[case])
    cache = s["cache"].to(cuda)
    req, pos, indptr, indices = lists(s, cuda)
    q = bskv.bskv_norm_rope_append_paged(
        s["q"].to(cuda), s["k"].to(cuda), s["v"].to(cuda), _dev(s["cos_sin"], cuda), req, pos, indptr, indices, cache,
        q_weight=_dev(s["wq"], cuda), k_weight=_dev(s["wk"], cuda), eps=1e-5, is_neox=neox)
    at = s["pos"].tolist()
    _close(to64(q), *_expect(s, "q", s["wq"], rot, neox, at), dtype)
    k, size = _expect(s, "k", s["wk"], rot, neox, at)
    page = s["indices"].long()[s["indptr"].long()[s["req"].long()] + s["pos"].long() // ps]
    slot = s["pos"].long() % ps
    got = cache.cpu()
    _close(to64(got[page, 0, :, slot]), k, size, dtype)
    assert torch.equal(got[page, 1, :, slot], s["v"])
    # nothing else of the cache changed
    got[page, :, :, slot] = s["cache"][page, :, :, slot]
    assert torch.equal(got.view(torch.int16), s["cache"].view(torch.int16))
    assert bskv.bskv_get_device_status() == 0


LONG = [
    # enough tokens that a warp takes whole ones, several in turn
    ([1500, 2200], [1500, 2100], 16, 5, 2, 64, 64, True, (1, 1), BF, torch.float32),
    ([4100], [4100], 8, 3, 1, 128, 32, False, (1, 0), FP, BF),
    ([2500], [2500], 16, 18, 9, 64, 16, False, (0, 1), BF, torch.float32),
]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_many_tokens(cuda, case):
    lens, new, ps, hq, hkv, d, rot, neox, _, dtype, _ = LONG[case]
    s = _make(LONG[case], 3)
    s["req"][[0, 77, 2431, sum(new) - 1]] = -1  # rows without a token
    cache, out = s["cache"].to(cuda), torch.full(s["q"].shape, 3.0, dtype=dtype, device=cuda)
    bskv.bskv_norm_rope_append_paged(
        s["q"].to(cuda), s["k"].to(cuda), s["v"].to(cuda), _dev(s["cos_sin"], cuda), *lists(s, cuda), cache,
        q_weight=_dev(s["wq"], cuda), k_weight=_dev(s["wk"], cuda), eps=1e-5, is_neox=neox, q_out=out)
    live = s["req"] >= 0
    assert (out[(~live).to(cuda)] == 3.0).all()
    at = s["pos"].tolist()
    q, size = _expect(s, "q", s["wq"], rot, neox, at)
    _close(to64(out)[live], q[live], size[live], dtype)
    k, size = _expect(s, "k", s["wk"], rot, neox, at)
    page = s["indices"].long()[s["indptr"].long()[s["req"][live].long()] + s["pos"][live].long() // ps]
    slot = s["pos"][live].long() % ps
    got = cache.cpu()
    _close(to64(got[page, 0, :, slot]), k[live], size[live], dtype)
    assert torch.equal(got[page, 1, :, slot], s["v"][live])
    got[page, :, :, slot] = s["cache"][page, :, :, slot]
    assert torch.equal(got.view(torch.int16), s["cache"].view(torch.int16))
    assert bskv.bskv_get_device_status() == 0


def test_strided_in_place_and_halves(cuda):
    """q, k and v as parts of one projection's output, q rotated in place, a cache in another order; and the
    same from two calls, of the queries and of the rest."""
    case = CASES[0]
    s = _make(case, 3)
    _, _, ps, hq, hkv, d, rot, neox, _, dtype, _ = case
    n = s["q"].shape[0]
    qkv = torch.cat([s["q"].reshape(n, -1), s["k"].reshape(n, -1), s["v"].reshape(n, -1)], 1).to(cuda)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    req, pos, indptr, indices = lists(s, cuda)
    w = dict(q_weight=s["wq"].to(cuda), k_weight=s["wk"].to(cuda), eps=1e-5)
    table = s["cos_sin"].to(cuda)
    cache = s["cache"].to(cuda)
    want = bskv.bskv_norm_rope_append_paged(q, k, v, table, req, pos, indptr, indices, cache, **w)
    # slots before heads, K and V of a page apart
    other = torch.zeros(2, s["pages"], ps, hkv, d, dtype=dtype, device=cuda).permute(1, 0, 3, 2, 4)
    other.copy_(s["cache"])
    only = bskv.bskv_norm_rope_append_paged(q, None, None, table, req, pos, None, None, None, q_weight=w["q_weight"], eps=1e-5)
    assert torch.equal(only, want)
    assert bskv.bskv_norm_rope_append_paged(None, k, v, table, req, pos, indptr, indices, other, k_weight=w["k_weight"], eps=1e-5) is None
    assert torch.equal(other, cache)
    got = bskv.bskv_norm_rope_append_paged(q, k, v, table, req, pos, indptr, indices, cache, q_out=q, **w)
    assert got is q and torch.equal(q, want)


def test_rows_without_a_token_and_rotary_positions(cuda):
    case = CASES[1]
    s = _make(case, 4)
    _, _, ps, hq, hkv, d, rot, neox, _, dtype, _ = case
    req, pos, indptr, indices = lists(s, cuda)
    req[3:5] = -1
    pos[3:5] = -1
    at = torch.arange(s["q"].shape[0], dtype=torch.int32).flip(0) % s["cos_sin"].shape[0]
    cache, q_out = s["cache"].to(cuda), torch.full_like(s["q"], 7.0).to(cuda)
    bskv.bskv_norm_rope_append_paged(s["q"].to(cuda), s["k"].to(cuda), s["v"].to(cuda), s["cos_sin"].to(cuda), req, pos,
                                     indptr, indices, cache, is_neox=neox, pos_ids=at.to(cuda), q_out=q_out)
    assert (q_out[3:5] == 7.0).all()
    ref, size = _expect(s, "q", None, rot, neox, at.tolist())
    live = [i for i in range(len(at)) if i not in (3, 4)]
    _close(to64(q_out)[live], ref[live], size[live], dtype)
    page = int(s["indices"][0])
    assert torch.equal(cache[page, :, :, 3:5].cpu(), s["cache"][page, :, :, 3:5])
    assert bskv.bskv_get_device_status() == 0


@pytest.mark.parametrize("bad", ["request", "position", "page", "rotary"])
def test_rows_out_of_range(cuda, bad):
    case = CASES[0]
    s = _make(case, 5)
    req, pos, indptr, indices = lists(s, cuda)
    at = None
    if bad == "request":
        req[1] = 3
    elif bad == "position":
        pos[1] = 16  # its request has one page
    elif bad == "page":
        indices[int(indptr[1])] = s["pages"]
    else:
        at = pos.clone()
        at[1] = s["cos_sin"].shape[0]
    cache, q_out = s["cache"].to(cuda), torch.full_like(s["q"], 7.0).to(cuda)
    bskv.bskv_norm_rope_append_paged(s["q"].to(cuda), s["k"].to(cuda), s["v"].to(cuda), s["cos_sin"].to(cuda), req, pos,
                                     indptr, indices, cache, pos_ids=at, q_out=q_out)
    assert bskv.bskv_get_device_status() == 6
    assert (q_out[1] == 7.0).all().item() == (bad == "rotary") and not (q_out[0] == 7.0).all()
    changed = (cache.cpu().view(torch.int16) != s["cache"].view(torch.int16)).any(-1).any(-1).any(-1).any(-1)
    page = [int(s["indices"][int(s["indptr"][b]) + int(s["pos"][b]) // 16]) for b in (0, 2)]
    assert sorted(changed.nonzero()[:, 0].tolist()) == sorted(page)


def test_zero_rows(cuda):
    s = _make(CASES[0])
    cache = s["cache"].to(cuda)
    e = torch.empty(0, dtype=torch.int32, device=cuda)
    got = bskv.bskv_norm_rope_append_paged(s["q"][:0].to(cuda), s["k"][:0].to(cuda), s["v"][:0].to(cuda), s["cos_sin"].to(cuda),
                                           e, e, s["indptr"].to(cuda), s["indices"].to(cuda), cache)
    assert got.shape[0] == 0 and torch.equal(cache.cpu(), s["cache"])


def test_norms_of_zeros_and_large_rows(cuda):
    """A row of zeros stays zero, values whose squares pass fp16's range are normalised in fp32."""
    s = _make(([2], [2], 16, 2, 1, 64, 64, True, (1, 1), FP, torch.float32), 6)
    s["q"][0] = 0.0
    s["q"][1] = 60000.0
    req, pos, indptr, indices = lists(s, cuda)
    got = bskv.bskv_norm_rope_append_paged(s["q"].to(cuda), s["k"].to(cuda), s["v"].to(cuda), s["cos_sin"].to(cuda), req, pos,
                                           indptr, indices, s["cache"].to(cuda), q_weight=s["wq"].to(cuda), k_weight=s["wk"].to(cuda), eps=1e-5)
    assert (got[0] == 0).all()
    _close(to64(got), *_expect(s, "q", s["wq"], 64, True, [0, 1]), FP)
