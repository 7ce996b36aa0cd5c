"""Accumulated attention weights on the GPU against the float64 oracle.

Tolerance, from the arithmetic: products of 16-bit values are exact, their fp32 sum over D is off
by at most about D / 8 roundings of 2^-23 of the sum of magnitudes A = scale sum |q_d k_d|; the
exponent is rounded at its own size (2^-23 (|s| + |lse|)) and ex2 is good to 2^-22. A weight is
therefore off by w 2^-22 (A D / 16 + |s| + |lse| + 4) at most, and a score by that summed over the
queries plus two roundings of the sum: (weights below 2^-126 may flush to zero).
"""

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
import synth
from oracle import cache as oc
from oracle.numerics import bits_to_f64
from gpu_util import bits
from test_gpu_fp4 import _cache

pytestmark = pytest.mark.gpu
DT = {torch.bfloat16: "bf16", torch.float16: "fp16"}


def _f64(t):
    return bits_to_f64(bits(t), DT[t.dtype])


def _check(d, keys, lse, before, after, causal, decay):
    """Scores against the oracle, the slots that hold no token untouched bit for bit."""
    q, D, sm = _f64(d["q"]), d["head_dim"], d["sm_scale"]
    a = (d["qo_indptr"].numpy(), d["kv_indptr"].numpy(), d["kv_indices"].numpy(),
         d["kv_last_page_len"].numpy(), d["page_size"])
    z = lse.cpu().double().numpy()
    old = before.cpu().double().numpy()
    ref = oc.attn_weights(q, keys, z, old, *a, sm, causal, decay)
    w = oc.attn_weights(q, keys, z, np.zeros_like(old), *a, sm, causal, 0.0)
    fin = np.where(np.isfinite(keys), keys, 0.0)
    A = sm * np.abs(q).sum(-1).max() * np.abs(fin).max() if q.size and fin.size else 0.0
    s = np.abs(z[np.isfinite(z)]).max(initial=0.0) + sm * np.abs(q).max(initial=0.0) * np.abs(fin).sum(-1).max(initial=0.0)
    A = min(A, s)
    tol = w * 2.0 ** -22 * (A * D / 16 + 2 * s + 4) + 2.0 ** -22 * np.abs(ref) + 1e-30
    used = np.zeros(old.shape, dtype=bool)
    for b, L in enumerate(oc.lengths(a[1], a[3], a[4])):
        for j in range(L):
            used[a[2][a[1][b] + j // a[4]], :, j % a[4]] = True
    got = after.cpu().double().numpy()
    same = np.isnan(got) == np.isnan(ref)
    assert same[used].all()
    err = np.where(used & np.isfinite(ref), np.abs(got - ref), 0.0)
    assert (err <= np.nan_to_num(tol)).all(), np.nanmax(err / tol)
    keep = torch.from_numpy(~used)
    assert torch.equal(after.cpu().view(torch.int32)[keep], before.cpu().view(torch.int32)[keep])


CASES = [
    # Hq, Hkv, D, page_size, lengths, queries, dtype, causal, decay
    (8, 2, 128, 16, [40, 1, 0, 333, 64], None, torch.bfloat16, True, 1.0),
    (32, 8, 128, 64, [700, 129], None, torch.bfloat16, True, 0.5),
    (16, 1, 64, 8, [90, 300], None, torch.float16, False, 0.0),        # 16 rows
    (6, 2, 64, 32, [77, 500, 31], [2, 1, 0], torch.float16, True, 0.9),  # ragged, no query at all
    (3, 3, 128, 48, [200, 50], [8, 3], torch.bfloat16, False, 1.0),
    (8, 2, 128, 16, [130, 5, 260, 0], [33, 5, 1, 0], torch.bfloat16, True, 1.0),  # tile kernel
    (8, 2, 64, 8, [128, 300], [100, 300], torch.float16, True, 0.25),
    (40, 2, 128, 64, [257], [1], torch.bfloat16, True, 1.0),            # 20 query heads per kv head
    (4, 1, 64, 16, [100, 3], [70, 9], torch.bfloat16, True, 1.0),       # more queries than tokens
    (4, 4, 128, 16, [150], [90], torch.float16, False, 0.0),
]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_weights(cuda, case, four):
    Hq, Hkv, D, ps, lens, nq, dtype, causal, decay = case
    d = synth.paged_decode_inputs(800 + Hq + ps, len(lens), Hq, Hkv, D, ps, 0, 0, lengths=lens, dtype=dtype)
    nq = [1] * len(lens) if nq is None else nq
    d["qo_indptr"] = torch.tensor([0] + list(np.cumsum(nq)), dtype=torch.int32)
    g = torch.Generator().manual_seed(801)
    n = int(d["qo_indptr"][-1])
    d["q"] = torch.randn(n, Hq, D, generator=g).to(dtype)
    lse = torch.randn(n, Hq, generator=g) + 4.0
    if n > 1:
        lse[1, 0] = -float("inf")  # a query that saw nothing
    scores = torch.rand(d["num_pages"], Hkv, ps, generator=g) * 3
    scores.view(-1)[::7] = float("nan") if decay == 0 else 0.25
    p = bskv.bskv_plan_attn_weights(None if nq == [1] * len(lens) else d["qo_indptr"], d["kv_indptr"],
                                    d["kv_indices"], d["kv_last_page_len"], d["num_pages"], ps, Hq, Hkv,
                                    D, causal=causal, dtype=dtype)
    after = scores.clone().to(cuda)
    q = d["q"].to(cuda)
    if four:
        codes, scales = _cache(802, d, cuda, 120, 126)
        keys = oc.fp4_decode(codes[:, 0].cpu().numpy(), scales[:, 0].cpu().numpy())
        bskv.bskv_run_attn_weights_fp4(p, q, codes, scales, lse.to(cuda), after, decay=decay)
    else:
        keys = _f64(d["kv_cache"][:, 0])
        bskv.bskv_run_attn_weights(p, q, d["kv_cache"].to(cuda), lse.to(cuda), after, decay=decay)
    torch.cuda.synchronize()
    _check(d, keys, lse, scores, after, causal, decay)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nq", [1, 20, 70])
def test_weights_scales_of_any_size(cuda, dtype, nq):
    """Scales that differ by 2^18 within a key, and blocks of zeros with scales far above them."""
    lens, Hq, Hkv, D, ps = [150, 33], 4, 2, 128, 16
    d = synth.paged_decode_inputs(871, 2, Hq, Hkv, D, ps, 0, 0, lengths=lens, dtype=dtype)
    d["qo_indptr"] = torch.tensor([0, nq, 2 * nq], dtype=torch.int32)
    g = torch.Generator().manual_seed(872)
    d["q"] = torch.randn(2 * nq, Hq, D, generator=g).to(dtype)
    lse, scores = torch.randn(2 * nq, Hq, generator=g) + 4.0, torch.rand(d["num_pages"], Hkv, ps, generator=g)
    codes, scales = _cache(873, d, "cpu", 108, 127)
    zero = (torch.rand(scales.shape, generator=g) < 0.3) & (scales != 255)
    scales[zero] = 250
    codes.view(*scales.shape, 16)[zero] &= 0x88  # zeros of either sign
    p = bskv.bskv_plan_attn_weights(d["qo_indptr"], d["kv_indptr"], d["kv_indices"], d["kv_last_page_len"],
                                    d["num_pages"], ps, Hq, Hkv, D, causal=False, dtype=dtype)
    after = scores.clone().to(cuda)
    bskv.bskv_run_attn_weights_fp4(p, d["q"].to(cuda), codes.to(cuda), scales.to(cuda), lse.to(cuda), after)
    keys = oc.fp4_decode(codes[:, 0].numpy(), scales[:, 0].numpy())
    _check(d, keys, lse, scores, after, False, 1.0)


def test_weights_of_a_decode_sum_to_the_heads(cuda):
    """With the log-sum-exp of the decode itself, the weights of a request sum to its query heads."""
    d = synth.paged_decode_inputs(811, 6, 32, 8, 128, 16, 1, 900)
    q, kv = d["q"].to(cuda), d["kv_cache"].to(cuda)
    a = (d["kv_indptr"], d["kv_indices"], d["kv_last_page_len"])
    _, lse = bskv.bskv_run_decode(bskv.bskv_plan_decode(*a, d["num_pages"], 16, 32, 8, 128), q, kv,
                                  return_lse=True)
    scores = torch.zeros((d["num_pages"], 8, 16), device=cuda)
    p = bskv.bskv_plan_attn_weights(None, *a, d["num_pages"], 16, 32, 8, 128)
    bskv.bskv_run_attn_weights(p, q, kv, lse, scores, decay=0.0)
    for b in range(6):
        pages = d["kv_indices"][int(d["kv_indptr"][b]):int(d["kv_indptr"][b + 1])].long().to(cuda)
        total = scores[pages].double().sum((0, 2))
        assert float((total - 4).abs().max()) < 1e-4


def test_weights_nan_keys_and_infinite_lse(cuda):
    """A NaN key gives its token a NaN score and no other; lse = +inf weighs nothing."""
    for nq in (1, 40):
        d = synth.paged_decode_inputs(821, 1, 4, 2, 128, 16, 0, 0, lengths=[200])
        d["qo_indptr"] = torch.tensor([0, nq], dtype=torch.int32)
        d["q"] = torch.randn(nq, 4, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
        kv = d["kv_cache"].clone()
        page = int(d["kv_indices"][3])
        kv[page, 0, 1, 5, 100] = float("nan")
        lse = torch.full((nq, 4), 5.0)
        lse[0, 0] = float("inf")
        scores = torch.zeros(d["num_pages"], 2, 16)
        after = scores.clone().to(cuda)
        p = bskv.bskv_plan_attn_weights(d["qo_indptr"], d["kv_indptr"], d["kv_indices"],
                                        d["kv_last_page_len"], d["num_pages"], 16, 4, 2, 128)
        bskv.bskv_run_attn_weights(p, d["q"].to(cuda), kv.to(cuda), lse.to(cuda), after)
        d["kv_cache"] = kv
        _check(d, _f64(kv[:, 0]), lse, scores, after, True, 1.0)
        assert int(torch.isnan(after).sum()) == 1


def test_weights_strides(cuda):
    """q as a slice, a token-major cache, scores inside a larger pool, an explicit scale."""
    d = synth.paged_decode_inputs(831, 3, 8, 2, 128, 16, 10, 100)
    d["sm_scale"] = 0.04
    d["qo_indptr"] = torch.arange(4, dtype=torch.int32)
    big = torch.zeros((3, 16, 128), dtype=torch.bfloat16, device=cuda)
    big[:, 1::2] = d["q"].to(cuda)
    kv = d["kv_cache"].to(cuda).transpose(2, 3).contiguous().transpose(2, 3)
    lse = torch.full((3, 8), 3.0)
    pool = torch.rand((d["num_pages"], 6, 16), device=cuda)
    scores = pool[:, 1:5:2]
    before = scores.clone()
    rest = pool.clone()
    p = bskv.bskv_plan_attn_weights(None, d["kv_indptr"], d["kv_indices"], d["kv_last_page_len"],
                                    d["num_pages"], 16, 8, 2, 128)
    bskv.bskv_run_attn_weights(p, big[:, 1::2], kv, lse.to(cuda), scores, sm_scale=0.04)
    _check(d, _f64(d["kv_cache"][:, 0]), lse, before, scores, True, 1.0)
    assert torch.equal(pool[:, 0::2], rest[:, 0::2]) and torch.equal(pool[:, 5], rest[:, 5])


def _many(cuda, lens, Hq, Hkv, D, ps, nq, dtype, causal, decay, four, plans):
    """Scores of the same call by plans for several numbers of SMs: within the tolerance of the oracle,
    and, as a key's sum does not depend on who makes it, the same bits."""
    d = synth.paged_decode_inputs(840 + Hq, len(lens), Hq, Hkv, D, ps, 0, 0, lengths=lens, dtype=dtype)
    d["qo_indptr"] = torch.tensor([0] + list(np.cumsum(nq)), dtype=torch.int32)
    g = torch.Generator().manual_seed(841)
    n = int(d["qo_indptr"][-1])
    d["q"] = torch.randn(n, Hq, D, generator=g).to(dtype)
    lse = torch.randn(n, Hq, generator=g) + 5.0
    lse[n // 2, 0] = -float("inf")
    scores = torch.rand(d["num_pages"], Hkv, ps, generator=g) * 3
    q, z = d["q"].to(cuda), lse.to(cuda)
    if four:
        codes, scales = _cache(842, d, cuda, 120, 126)
        keys = oc.fp4_decode(codes[:, 0].cpu().numpy(), scales[:, 0].cpu().numpy())
    else:
        keys, kv = _f64(d["kv_cache"][:, 0]), d["kv_cache"].to(cuda)
    first = None
    for sms in plans:
        p = bskv.bskv_plan_attn_weights(d["qo_indptr"], d["kv_indptr"], d["kv_indices"], d["kv_last_page_len"],
                                        d["num_pages"], ps, Hq, Hkv, D, causal=causal, dtype=dtype, num_sms=sms)
        after = scores.clone().to(cuda)
        if four:
            bskv.bskv_run_attn_weights_fp4(p, q, codes, scales, z, after, decay=decay)
        else:
            bskv.bskv_run_attn_weights(p, q, kv, z, after, decay=decay)
        torch.cuda.synchronize()
        if first is None:
            first = after
            _check(d, keys, lse, scores, after, causal, decay)
        assert torch.equal(after.view(torch.int32), first.view(torch.int32)), sms
    assert bskv.bskv_get_device_status() == 0


@pytest.mark.parametrize("four", [False, True])
def test_weights_of_long_requests_without_a_mask(cuda, four):
    """Every row sees every key, over many whole tiles: one query and its last-query mask are the same."""
    for causal in (False, True):
        _many(cuda, [900, 40, 3001], 8, 2, 128, 16, [1, 1, 1], torch.bfloat16, causal, 0.5, four, (1, None))
    _many(cuda, [900, 40, 3001], 8, 2, 64, 16, [3, 1, 2], torch.float16, False, 1.0, four, (1, None))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("Hq, Hkv, D, ps, nq, dtype, causal, decay", [
    (12, 3, 128, 16, [1] * 5, torch.bfloat16, True, 0.75),         # two workers per warp in 16 bits
    (12, 3, 64, 8, [1] * 5, torch.float16, True, 1.0),
    (6, 2, 128, 48, [4, 1, 0, 5, 2], torch.bfloat16, True, 0.0),   # 9 to 16 rows
    (16, 1, 128, 64, [1] * 5, torch.float16, False, 0.5),
])
def test_weights_stream_of_many_tiles(cuda, four, Hq, Hkv, D, ps, nq, dtype, causal, decay):
    """16 workers for everything: rings that turn over, chunks of several units, windows of page ids."""
    _many(cuda, [2100, 33, 0, 1207, 5], Hq, Hkv, D, ps, nq, dtype, causal, decay, four, (1, 2, None))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("Hq, Hkv, D, ps, nq, dtype, causal, decay", [
    (8, 2, 128, 16, [20, 0, 7, 32, 1], torch.bfloat16, True, 0.75),    # one product an item, items without one
    (8, 2, 64, 8, [9, 30, 2, 31, 5], torch.float16, False, 0.0),
    (40, 2, 128, 64, [6, 3, 0, 1, 2], torch.bfloat16, True, 1.0),      # 20 heads per kv head
    (8, 2, 128, 16, [70, 0, 1, 333, 40], torch.bfloat16, True, 0.75),  # several products
    (6, 3, 64, 32, [200, 65, 0, 64, 129], torch.float16, False, 0.5),
    (4, 4, 128, 48, [500, 900, 1, 129, 2], torch.float16, True, 1.0),  # more queries than tokens
])
def test_weights_tile_of_many_items(cuda, four, Hq, Hkv, D, ps, nq, dtype, causal, decay):
    """Two CTAs, or four, for everything: both key buffers, queries that change, every parity."""
    _many(cuda, [1000, 150, 1, 2049, 260], Hq, Hkv, D, ps, nq, dtype, causal, decay, four, (1, 2, None))


@pytest.mark.parametrize("nq", [1, 30])
def test_weights_of_any_number_of_sms(cuda, nq):
    _many(cuda, [300, 41], 8, 2, 128, 16, [nq, nq], torch.bfloat16, True, 0.5, False, (None, 2 ** 30, 2 ** 31 - 1))
