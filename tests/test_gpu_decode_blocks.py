"""Attention over chosen blocks against the float64 definition."""

import math

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
from blocks_util import batch, lists, pages_of, to64
from oracle import blocks as ob

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def _inputs(lens, new, ps, hq, hkv, d, top, dtype, seed, chosen="random"):
    g = torch.Generator().manual_seed(seed)
    s = batch(lens, new, ps, seed)
    s["q"] = torch.randn(sum(new), hq, d, generator=g).to(dtype)
    s["kv"] = torch.randn(s["pages"], 2, hkv, ps, d, generator=g).to(dtype)
    for b, n in enumerate(lens):  # slots past the end may hold anything
        if n % ps:
            s["kv"][pages_of(s, b)[-1], :, :, n % ps:] = float("nan")
    unused = sorted(set(range(s["pages"])) - set(s["indices"].tolist()))
    s["kv"][unused] = float("nan")
    rng = np.random.default_rng(seed)
    blocks = np.full((sum(new), hkv, top), -1, dtype=np.int32)
    for t in range(sum(new)):
        seen = int(s["pos"][t]) // ps + 1
        for h in range(hkv):
            n = min(top, seen)
            if chosen == "gaps":
                n = int(rng.integers(0, n + 1))
            pick = rng.permutation(seen)[:n]
            if chosen == "gaps":  # any order, and entries of no block between
                row = np.full(min(top, seen), -1)
                row[rng.permutation(min(top, seen))[:n]] = pick
                blocks[t, h, :len(row)] = row
            else:
                blocks[t, h, :n] = np.sort(pick)
    s["blocks"] = torch.tensor(blocks)
    return s


def _expect(s, scale):
    q, kv = to64(s["q"]), to64(s["kv"])
    n, hq, d = q.shape
    hkv, ps = kv.shape[2], s["ps"]
    out, lse, size, err = np.zeros_like(q), np.full((n, hq), -np.inf), np.zeros_like(q), np.zeros((n, hq))
    for t in range(n):
        pages, pos = pages_of(s, int(s["req"][t])), int(s["pos"][t])
        for h in range(hkv):
            at = [j * ps + i for j in s["blocks"][t, h].tolist() if j >= 0 for i in range(min(ps, pos + 1 - j * ps))]
            at = np.array(at, dtype=int)
            g = slice(h * hq // hkv, (h + 1) * hq // hkv)
            k, v = kv[pages[at // ps], 0, h, at % ps], kv[pages[at // ps], 1, h, at % ps]
            out[t, g], lse[t, g], size[t, g] = ob.attend(q[t, g], k, v, scale)
            if len(at):
                err[t, g] = (np.abs(q[t, g]) @ np.abs(k).T).max(-1) * scale * 136 * 2.0 ** -24
    return out, lse, size, err


def _check(out, lse, ref, dtype):
    """Weights and the output are rounded to dtype once each; a logit's fp32 sum of 128 products and eight more steps is off
    by `err`, which moves a weight by twice that (its own and the sum's), and the approximate exponentials by 2^-20."""
    want, z, size, err = ref
    half = torch.finfo(dtype).eps / 2
    rel = 2 * err[..., None] + 2.0 ** -18
    tol = half * np.abs(want) + (half * 1.01 + rel) * size + (2.0 ** -24 if dtype == FP else 0.0)
    bad = ~(np.abs(to64(out) - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], to64(out)[bad][:3], want[bad][:3])
    got = to64(lse)
    none = np.isneginf(z)
    assert (got[none] == -np.inf).all()
    got, z, err = got[~none], z[~none], err[~none]
    bad = ~(np.abs(got - z) <= err + 2.0 ** -18 + 2.0 ** -22 * np.abs(z))
    assert not bad.any(), (got[bad][:3], z[bad][:3])


CASES = [
    ([700, 1, 33, 160], [1, 1, 1, 1], 16, 8, 2, 128, 4, BF),
    ([20000], [1], 16, 32, 8, 128, 64, BF),
    ([999, 4, 300], [4, 4, 2], 8, 24, 4, 64, 32, FP),
    ([130, 17], [2, 1], 48, 5, 5, 128, 2, FP),
    ([300, 257], [1, 3], 64, 16, 1, 128, 5, BF),
    ([300, 257], [1, 3], 64, 32, 2, 64, 3, FP),
    ([2000] * 60, [1] * 60, 16, 12, 4, 128, 40, BF),
    ([500] * 90, [2] * 90, 8, 8, 8, 64, 20, BF),
    ([77] * 300, [1] * 300, 16, 4, 4, 128, 9, FP),
    ([8], [8], 8, 6, 2, 128, 1, BF),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("chosen", ["random", "gaps"])
def test_attention(cuda, case, chosen):
    lens, new, ps, hq, hkv, d, top, dtype = CASES[case]
    s = _inputs(lens, new, ps, hq, hkv, d, top, dtype, case, chosen)
    p = bskv.bskv_plan_decode_blocks(sum(new), max(-(-n // ps) for n in lens), s["pages"], ps, hq, hkv, d, top, dtype=dtype)
    ref = _expect(s, 1.0 / math.sqrt(d))
    args = s["q"].to(cuda), s["kv"].to(cuda), s["blocks"].to(cuda), *lists(s, cuda)
    out, lse = bskv.bskv_run_decode_blocks(p, *args, return_lse=True)
    _check(out, lse, ref, dtype)
    again = bskv.bskv_run_decode_blocks(p, *args)  # the counters are ready, and the sums have an order
    assert torch.equal(out, again)
    assert bskv.bskv_get_device_status() == 0


def test_all_blocks_are_the_paged_decode(cuda):
    """With every block listed it is the dense decode over the same table."""
    lens, ps, hq, hkv, d = [700, 129, 1, 1000], 16, 16, 4, 128
    s = _inputs(lens, [1] * 4, ps, hq, hkv, d, 63, BF, 3)
    p = bskv.bskv_plan_decode_blocks(4, 63, s["pages"], ps, hq, hkv, d, 63)
    q, kv = s["q"].to(cuda), s["kv"].to(cuda)
    out, lse = bskv.bskv_run_decode_blocks(p, q, kv, s["blocks"].to(cuda), *lists(s, cuda), return_lse=True, sm_scale=0.2)
    dense = bskv.bskv_plan_decode(s["indptr"], s["indices"], s["last"], s["pages"], ps, hq, hkv, d, BF)
    want, z = bskv.bskv_run_decode(dense, q, kv, return_lse=True, sm_scale=0.2)
    ref = _expect(s, 0.2)
    _check(out, lse, ref, BF)
    _check(want, z, ref, BF)


def test_strides_and_rows_without_a_token(cuda):
    lens, new, ps, hq, hkv, d, top, dtype = CASES[2]
    s = _inputs(lens, new, ps, hq, hkv, d, top, dtype, 9)
    n = sum(new)
    p = bskv.bskv_plan_decode_blocks(n, 125, s["pages"], ps, hq, hkv, d, top, dtype=dtype)
    req, pos, indptr, indices = lists(s, cuda)
    req[1] = -1
    req[n - 1] = -3
    kv = s["kv"].permute(1, 0, 3, 2, 4).contiguous().to(cuda).permute(1, 0, 3, 2, 4)
    q = torch.zeros(hq, n, d, dtype=dtype, device=cuda).transpose(0, 1)
    q.copy_(s["q"])
    out = torch.full((n, hq + 1, d), 7.0, dtype=dtype, device=cuda)[:, :hq]
    lse = torch.full((n, hq), 7.0, device=cuda)
    assert bskv.bskv_run_decode_blocks(p, q, kv, s["blocks"].to(cuda), req, pos, indptr, indices, out=out, lse=lse) is out
    for t in (1, n - 1):
        assert (out[t] == 7.0).all() and (lse[t] == 7.0).all()
    live = [t for t in range(n) if t not in (1, n - 1)]
    ref = _expect(s, 1.0 / math.sqrt(d))
    _check(out[live], lse[live], tuple(x[live] for x in ref), dtype)
    assert bskv.bskv_get_device_status() == 0


@pytest.mark.parametrize("bad", ["request", "position", "negative", "page", "block"])
def test_out_of_range(cuda, bad):
    lens, new, ps, hq, hkv, d, top, dtype = CASES[0]
    s = _inputs(lens, new, ps, hq, hkv, d, top, dtype, 10)
    p = bskv.bskv_plan_decode_blocks(4, 44, s["pages"], ps, hq, hkv, d, top, dtype=dtype)
    ref = [x.copy() for x in _expect(s, 1.0 / math.sqrt(d))]
    req, pos, indptr, indices = lists(s, cuda)
    blocks = s["blocks"].clone()
    if bad == "request":
        req[0] = 4
    elif bad == "position":
        pos[0] = 704
    elif bad == "negative":
        pos[0] = -1
    else:  # the row goes on without the block
        j = int(blocks[0, 1, 2])
        if bad == "page":
            indices[j] = s["pages"] + 5
            s["blocks"][0][s["blocks"][0] == j] = -1
        else:
            blocks[0, 1, 2] = 44
            s["blocks"][0, 1, 2] = -1
        for a, x in zip(ref, _expect(s, 1.0 / math.sqrt(d))):
            a[0] = x[0]
    if bad in ("request", "position", "negative"):
        for a, x in zip(ref, (0.0, -np.inf, 0.0, 0.0)):
            a[0] = x
    out, lse = bskv.bskv_run_decode_blocks(p, s["q"].to(cuda), s["kv"].to(cuda), blocks.to(cuda), req, pos, indptr, indices,
                                           return_lse=True)
    assert bskv.bskv_get_device_status() == 6
    _check(out, lse, ref, dtype)


def test_sharp_and_large_logits(cuda):
    """One key that takes all weight, in every place of a list; logits of both signs in the hundreds."""
    lens, new, ps, hq, hkv, d, top = [1024], [1], 16, 4, 1, 128, 64
    s = _inputs(lens, new, ps, hq, hkv, d, top, BF, 11)
    p = bskv.bskv_plan_decode_blocks(1, 64, s["pages"], ps, hq, hkv, d, top)
    s["q"] *= 12
    base = s["kv"].clone()
    for at in (0, 15, 16, 500, 1023):
        s["kv"] = base.clone()
        s["kv"][pages_of(s, 0)[at // ps], 0, 0, at % ps] = s["q"][0, 0]
        out, lse = bskv.bskv_run_decode_blocks(p, s["q"].to(cuda), s["kv"].to(cuda), s["blocks"].to(cuda), *lists(s, cuda),
                                               return_lse=True)
        _check(out, lse, _expect(s, 1.0 / math.sqrt(d)), BF)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_infinite_keys(cuda, dtype):
    """Logits of -inf have no weight: in whole blocks, wherever they stand in a list; heads that see nothing else get
    what a row without a block gets."""
    lens, new, ps, hq, hkv, d, top = [1024, 160, 40], [1, 1, 1], 16, 4, 2, 64, 64
    s = _inputs(lens, new, ps, hq, hkv, d, top, dtype, 13)
    p = bskv.bskv_plan_decode_blocks(3, 64, s["pages"], ps, hq, hkv, d, top, dtype=dtype)
    s["q"][:, :, 5] = s["q"][:, :, 5].abs() + 0.5
    for b, blocks in enumerate([(0, 1, 30, 31, 32, 63), (0, 9), (0, 1, 2)]):
        for j in blocks:
            s["kv"][pages_of(s, b)[j], 0, :, :min(ps, lens[b] - j * ps), 5] = -float("inf")
    out, lse = bskv.bskv_run_decode_blocks(p, s["q"].to(cuda), s["kv"].to(cuda), s["blocks"].to(cuda), *lists(s, cuda),
                                           return_lse=True)
    assert bskv.bskv_get_device_status() == 0
    assert (out[2] == 0).all() and (lse[2] == -float("inf")).all()
    # without those blocks nothing else changes
    for b, blocks in enumerate([(0, 1, 30, 31, 32, 63), (0, 9), (0, 1, 2)]):
        for j in blocks:
            s["blocks"][b][s["blocks"][b] == j] = -1
    _check(out, lse, _expect(s, 1.0 / math.sqrt(d)), dtype)


def test_forced_timeout(cuda):
    """Waits that give up are reported; after an upload the plan runs again."""
    lens, new, ps, hq, hkv, d, top, dtype = CASES[1]
    s = _inputs(lens, new, ps, hq, hkv, d, top, dtype, 12)
    p = bskv.bskv_plan_decode_blocks(1, 1250, s["pages"], ps, hq, hkv, d, top, dtype=dtype).upload(cuda)
    args = s["q"].to(cuda), s["kv"].to(cuda), s["blocks"].to(cuda), *lists(s, cuda)
    want = bskv.bskv_run_decode_blocks(p, *args)
    bskv.bskv_set_debug_force_timeout(True)
    try:
        bskv.bskv_run_decode_blocks(p, *args)
        torch.cuda.synchronize()
        assert bskv.bskv_get_device_status() == 5
    finally:
        bskv.bskv_set_debug_force_timeout(False)
    p.upload(cuda)
    assert torch.equal(bskv.bskv_run_decode_blocks(p, *args), want)
    assert bskv.bskv_get_device_status() == 0
