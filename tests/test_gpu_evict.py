"""Eviction on the GPU: the kept tokens and every moved byte equal the definition's exactly."""

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
from oracle import cache as oc

pytestmark = pytest.mark.gpu


def _setup(lens, ps, Hkv, D, seed, four, kept=None, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    n = [-(-x // ps) for x in lens]
    m = [-(-x // ps) for x in kept] if kept is not None else []
    total = sum(n) + sum(m) + 3
    perm = torch.randperm(total, generator=g).to(torch.int32)
    s = dict(indptr=torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32), indices=perm[:sum(n)],
             last=torch.tensor([x - (c - 1) * ps if c else 0 for x, c in zip(lens, n)], dtype=torch.int32),
             pages=total, scores=torch.randn(total, Hkv, ps, generator=g))
    if kept is not None:
        s["dst_indptr"] = torch.tensor([0] + list(np.cumsum(m)), dtype=torch.int32)
        s["dst_indices"] = perm[sum(n):sum(n) + sum(m)]
    if four:
        s["pools"] = [torch.randint(0, 256, (total, 2, Hkv, ps, w), generator=g, dtype=torch.uint8)
                      for w in (D // 2, D // 32)]
    else:
        s["pools"] = [torch.randint(-32768, 32768, (total, 2, Hkv, ps, D), generator=g,
                                    dtype=torch.int16).view(dtype)]
    return s


def _expect(s, lens, ps, Hkv, keep, sink, recent, compact):
    """(kept, pools, scores) by the definition, on copies."""
    raw = [x.view(torch.int16 if x.element_size() == 2 else torch.uint8).numpy() for x in s["pools"]]
    scores = s["scores"].numpy()
    out, osc = [x.copy() for x in raw], scores.copy()
    kept = [[] for _ in range(Hkv)]
    ptr, idx = s["indptr"].numpy(), s["indices"].numpy()
    dptr, didx = (s["dst_indptr"].numpy(), s["dst_indices"].numpy()) if "dst_indptr" in s else (ptr, idx)
    for b, L in enumerate(lens):
        for h in range(Hkv):
            sc = oc.request_rows(scores, ptr, idx, b, L)[h] if L else np.zeros(0)
            stay = oc.evict_kept(sc, L, keep[b], sink, recent)
            kept[h] += stay
            for j, t in enumerate(stay):
                sp, ss, dp, ds = idx[ptr[b] + t // ps], t % ps, didx[dptr[b] + j // ps], j % ps
                for o, r in zip(out, raw):
                    o[dp, :, h, ds] = r[sp, :, h, ss]
                if compact:
                    osc[dp, h, ds] = scores[sp, h, ss]
    return np.array(kept, dtype=np.int32).reshape(Hkv, -1), out, osc


def _run(cuda, s, lens, ps, Hkv, D, keep, sink, recent, compact):
    p = bskv.bskv_plan_evict(s["indptr"], s["indices"], s["last"], keep, sink, recent, s["pages"], ps,
                             Hkv, D, s.get("dst_indptr"), s.get("dst_indices"))
    scores, pools = s["scores"].to(cuda), [x.to(cuda) for x in s["pools"]]
    run = bskv.bskv_run_evict if len(pools) == 1 else bskv.bskv_run_evict_fp4
    kept = run(p, scores, *pools, compact_scores=compact)
    torch.cuda.synchronize()
    return kept.cpu().numpy(), [x.view(torch.int16 if x.element_size() == 2 else torch.uint8).cpu().numpy()
                                for x in pools], scores.cpu()


def _same(cuda, s, lens, ps, Hkv, D, keep, sink, recent, compact):
    want = _expect(s, lens, ps, Hkv, keep, sink, recent, compact)
    got = _run(cuda, s, lens, ps, Hkv, D, keep, sink, recent, compact)
    assert (got[0] == want[0]).all()
    for a, b in zip(got[1], want[1]):
        assert (a == b).all()
    assert torch.equal(got[2].view(torch.int32), torch.from_numpy(want[2]).view(torch.int32))


CASES = [
    # lens, keep, sink, recent, page_size, Hkv, D
    ([100, 1, 0, 333, 64], [50, 1, 5, 100, 64], 4, 16, 16, 2, 128),
    ([7, 40, 1], [0, 1, 0], 0, 0, 8, 3, 64),              # keep nothing, or one
    ([2000, 700], [1990, 20], 2, 5, 64, 2, 128),          # several waves of rows
    ([257, 129], [128, 128], 64, 64, 48, 1, 128),         # only the protected ones
    ([1500], [1499], 0, 0, 16, 4, 64),                    # one token leaves
]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("place", ["in", "copy"])
@pytest.mark.parametrize("case", CASES)
def test_evict(cuda, case, place, four):
    lens, keep, sink, recent, ps, Hkv, D = case
    kept = [min(a, b) for a, b in zip(lens, keep)]
    s = _setup(lens, ps, Hkv, D, 900 + len(lens), four, kept if place == "copy" else None)
    _same(cuda, s, lens, ps, Hkv, D, keep, sink, recent, compact=not four or place == "copy")


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("lens, keep, Hkv, D", [
    ([20011], [17001], 1, 128),            # a cluster of eight CTAs, slices of 64 bytes
    ([9000, 9, 6007], [7000, 9, 6000], 4, 128),
    ([5000, 4999], [4990, 2100], 2, 64),   # two CTAs
    ([4097], [1], 1, 64),
])
def test_evict_long_in_place(cuda, lens, keep, Hkv, D, four):
    """Waves of rows and shares of scores that several CTAs take."""
    s = _setup(lens, 16, Hkv, D, 941, four)
    _same(cuda, s, lens, 16, Hkv, D, keep, 1, 0, True)


def test_evict_more_scores_than_shared_memory(cuda):
    """Scores that a cluster's shared memory cannot hold are read in every pass."""
    L, keep, ps = 270007, 3, 64
    s = _setup([L], ps, 1, 64, 951, True, [keep])
    rows = s["scores"][s["indices"].long(), 0].reshape(-1)[:L]
    p = bskv.bskv_plan_evict(s["indptr"], s["indices"], s["last"], [keep], 0, 0, s["pages"], ps, 1, 64,
                             s["dst_indptr"], s["dst_indices"])
    kept = bskv.bskv_run_evict_fp4(p, s["scores"].to(cuda), *[x.to(cuda) for x in s["pools"]])
    assert kept.cpu().tolist() == [sorted(torch.sort(rows, descending=True, stable=True).indices[:keep].tolist())]


def test_evict_order_of_scores(cuda):
    """Equal scores, both zeros, NaN, infinities and subnormals: NaN first, then by value, the
    lowest slot among equals, at every cut."""
    vals = [0.0, -0.0, 1.0, 1.0, float("nan"), float("inf"), -float("inf"), 1e-45, -1e-45, -1.0, 2.0,
            -float("nan")]
    lens = [96]
    for keep in (1, 2, 3, 20, 31, 32, 33, 47, 64, 90, 95):
        s = _setup(lens, 16, 1, 64, 911, False)
        g = torch.Generator().manual_seed(keep)
        rows = torch.tensor(vals)[torch.randint(0, len(vals), (96,), generator=g)]
        for i in range(6):
            s["scores"][int(s["indices"][i]), 0] = rows[16 * i:16 * i + 16]
        _same(cuda, s, lens, 16, 1, 64, [keep], 0, 0, True)


def test_evict_all_scores_equal(cuda):
    s = _setup([900, 50], 16, 2, 128, 921, False)
    s["scores"].fill_(0.125)
    _same(cuda, s, [900, 50], 16, 2, 128, [300, 10], 3, 7, True)


def test_evict_long_request(cuda):
    """More scores than one CTA's shared memory holds; the kept list against torch's stable sort."""
    L, keep, sink, recent, ps = 70001, 9000, 5, 1000, 16
    s = _setup([L], ps, 2, 64, 931, True, [keep])
    s["scores"] = (s["scores"] * 64).round() / 64  # many equal ones
    kept, pools, _ = _run(cuda, s, [L], ps, 2, 64, [keep], sink, recent, False)
    idx = s["indices"].long()
    flat = s["scores"][idx].transpose(0, 1).reshape(2, -1)[:, :L].clone()
    flat[:, :sink] = float("inf")
    flat[:, L - recent:] = float("inf")
    order = flat.sort(dim=1, descending=True, stable=True).indices[:, :keep].sort(dim=1).values
    assert torch.equal(torch.from_numpy(kept).long(), order)
    dst = s["dst_indices"].long()
    for new, old in zip(pools, s["pools"]):
        a = torch.from_numpy(new)[dst].permute(2, 0, 3, 1, 4).reshape(2, -1, 2, new.shape[-1])[:, :keep]
        b = old[idx].permute(2, 0, 3, 1, 4).reshape(2, -1, 2, new.shape[-1])
        assert torch.equal(a, b.gather(1, order[:, :, None, None].expand(-1, -1, 2, new.shape[-1])))


def test_evict_strided_pools(cuda):
    """A token-major cache and scores inside a larger pool, in place."""
    lens, keep = [120, 40], [30, 30]
    s = _setup(lens, 16, 2, 128, 941, False)
    want = _expect(s, lens, 16, 2, keep, 2, 4, True)
    p = bskv.bskv_plan_evict(s["indptr"], s["indices"], s["last"], keep, 2, 4, s["pages"], 16, 2, 128)
    kv = s["pools"][0].to(cuda).transpose(2, 3).contiguous().transpose(2, 3)
    pool = torch.zeros((s["pages"], 4, 16), device=cuda)
    pool[:, 1:3] = s["scores"].to(cuda)
    kept = torch.full((2, 60), -1, dtype=torch.int32, device=cuda)
    bskv.bskv_run_evict(p, pool[:, 1:3], kv, kept=kept)
    assert (kept.cpu().numpy() == want[0]).all()
    assert (kv.contiguous().view(torch.int16).cpu().numpy() == want[1][0]).all()
    assert (pool[:, 1:3].cpu().numpy() == want[2]).all()
    assert bool((pool[:, 0] == 0).all()) and bool((pool[:, 3] == 0).all())
