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
