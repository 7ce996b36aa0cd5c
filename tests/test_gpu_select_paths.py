"""The choice of blocks where a launch takes other ways: kv heads that do not fill a set of warps or pass one, rows of more
blocks than the narrow selection takes, more queries than what they see is kept for."""

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
from blocks_util import lists
from test_gpu_select_blocks import _expect, _plan, _select_inputs

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
KINDS = ["normal", "few values", "equal", "near", "zero", "not numbers"]


def _check(cuda, s, hq, hkv, d, top, sink, recent, dtype, **plan):
    p = _plan(s, hq, hkv, d, top, sink, recent, dtype, **plan)
    want = _expect(s, hkv, top, sink, recent)
    for _ in range(2):
        got = bskv.bskv_run_select_blocks(p, s["q"].to(cuda), s["bounds"].to(cuda), *lists(s, cuda))
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert bskv.bskv_get_device_status() == 0


@pytest.mark.parametrize("hkv,group,d,dtype", [(3, 2, 128, BF), (5, 1, 64, FP), (6, 2, 64, BF), (7, 1, 128, FP), (9, 2, 64, BF), (12, 1, 128, BF),
                                               (17, 1, 64, FP)])
@pytest.mark.parametrize("kind", KINDS)
def test_heads_that_do_not_fill_a_set(cuda, hkv, group, d, dtype, kind):
    """Fewer than eight heads leave warps idle, more make several groups, the last with heads missing."""
    s = _select_inputs([1500, 33, 700, 250], [2, 1, 1, 3], 16, hkv * group, hkv, d, dtype, hkv, kind)
    _check(cuda, s, hkv * group, hkv, d, 9, 1, 2, dtype)
    _check(cuda, s, hkv * group, hkv, d, 9, 1, 2, dtype, num_sms=3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv,group,d,dtype,top", [(1, 4, 128, BF, 64), (3, 1, 64, FP, 700)])
def test_rows_of_the_wide_selection(cuda, kind, hkv, group, d, dtype, top):
    """About 3000 blocks of a row, beside rows of a few."""
    s = _select_inputs([3001 * 8 - 5, 24, 2049 * 8], [2, 1, 1], 8, hkv * group, hkv, d, dtype, 7, kind)
    _check(cuda, s, hkv * group, hkv, d, top, 2, 3, dtype)


@pytest.mark.parametrize("kind", ["normal", "few values", "not numbers"])
def test_more_queries_than_are_kept(cuda, kind):
    """1500 queries of ragged requests and three kv heads, whose rows are looked up again; some without a token."""
    hq, hkv, d, top, sink, recent, dtype = 6, 3, 64, 7, 1, 2, BF
    lens = [900, 3, 411, 160, 1, 77, 700, 16]
    new = [600, 3, 300, 60, 1, 20, 500, 16]
    s = _select_inputs(lens, new, 16, hq, hkv, d, dtype, 9, kind)
    n = sum(new)
    assert n == 1500
    p = _plan(s, hq, hkv, d, top, sink, recent, dtype)
    req, pos, indptr, indices = lists(s, cuda)
    gone = torch.arange(0, n, 7, device=cuda)
    req[gone], pos[gone] = -1, -1
    blocks = torch.full((n, hkv, top), -5, dtype=torch.int32, device=cuda)
    want = _expect(s, hkv, top, sink, recent)
    want[gone.cpu().numpy()] = -5
    for _ in range(2):
        bskv.bskv_run_select_blocks(p, s["q"].to(cuda), s["bounds"].to(cuda), req, pos, indptr, indices, blocks=blocks)
        np.testing.assert_array_equal(blocks.cpu().numpy(), want)
    assert bskv.bskv_get_device_status() == 0
