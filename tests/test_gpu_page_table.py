"""Page tables and token maps made on the GPU equal the definition's; what does not fit is reported."""

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
from oracle import blocks as ob

pytestmark = pytest.mark.gpu


def _i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def _table(lens, new, ps, most, seed, allocate):
    """block_table with the pages that the old tokens hold (all pages without allocate), and a free list."""
    rng = np.random.default_rng(seed)
    held = [-(-(n - m if allocate else n) // ps) for n, m in zip(lens, new)]
    need = sum(-(-n // ps) for n in lens)
    ids = rng.permutation(need + 5).tolist()
    table = []
    for h in held:
        table.append([ids.pop() for _ in range(h)] + [-7] * (most - h))
    return table, ids, need + 5


CASES = [
    ([], [], 16), ([0], [0], 16), ([1], [1], 8), ([16, 17, 15], [1, 1, 1], 16), ([0, 5, 0, 0, 33], [0, 5, 0, 0, 2], 8),
    ([700, 1, 129], [700, 1, 4], 16), (list(range(0, 600)), [min(n, 3) for n in range(600)], 16),
    ([4096] * 64, [1] * 64, 16), ([1000] * 37, [999] * 37, 48), ([5000], [5000], 64), ([3] * 8192, [1] * 8192, 8),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("allocate", [False, True])
def test_table_and_map(cuda, case, allocate):
    lens, new, ps = CASES[case]
    most = max([-(-n // ps) for n in lens], default=0) + 2
    table, free, pool = _table(lens, new, ps, most, case, allocate)
    total, entries = sum(new), sum(-(-n // ps) for n in lens)
    dev_table = torch.full((max(1, len(lens)), most + 3), -9, dtype=torch.int32, device=cuda)[:len(lens), :most]
    if lens:
        dev_table.copy_(torch.tensor(table, dtype=torch.int32))
    room = total + 6
    t = bskv.PageTable(_i32([5] * (len(lens) + 1), cuda), torch.full((len(lens) * most + 4,), -3, dtype=torch.int32, device=cuda),
                       _i32([5] * len(lens), cuda), _i32([5] * (len(lens) + 1), cuda), _i32([5] * room, cuda),
                       _i32([5] * room, cuda), torch.full((room,), 5, device=cuda), _i32([5], cuda))
    kw = dict(free_pages=_i32(free + [77], cuda), free_count=_i32([len(free)], cuda)) if allocate else {}
    assert bskv.bskv_build_page_table(_i32(lens, cuda), dev_table, ps, pool, new_lens=_i32(new, cuda), out=t, **kw) is t
    want_free = list(free)
    indptr, indices, last, qo, req, pos, slots = ob.page_table(lens, new, table, ps, want_free if allocate else None)
    assert t.kv_indptr.tolist() == indptr and t.qo_indptr.tolist() == qo and t.kv_last_page_len.tolist() == last
    assert t.kv_indices[:entries].tolist() == indices and (t.kv_indices[entries:] == -3).all()
    assert t.batch_indices.tolist() == req + [-1] * 6 and t.positions.tolist() == pos + [-1] * 6
    assert t.slots.tolist() == slots + [-1] * 6
    if lens:
        assert dev_table.tolist() == table
    assert t.free_left.tolist() == ([len(want_free)] if allocate else [5])
    assert bskv.bskv_get_device_status() == 0


def test_one_new_token_each_by_default(cuda):
    t = bskv.bskv_build_page_table(_i32([3, 0, 8], cuda), _i32([[4], [0], [2]], cuda), 8, 5)
    assert t.batch_indices.tolist() == [0, 2, -1] and t.positions.tolist() == [2, 7, -1]
    assert t.slots.tolist() == [34, 23, -1] and t.free_left is None


@pytest.mark.parametrize("what", ["negative", "new", "long", "page", "free", "room", "count"])
def test_what_does_not_fit(cuda, what):
    """The request, or the pages, concerned are left out and the others are as without them."""
    lens, new, table = [9, 20, 4], [1, 4, 4], [[0, 1, -1], [2, 3, -1], [5, -1, -1]]
    free, count, room = [8, 7, 6], 3, 9
    if what == "negative":
        lens[1] = -1
    if what == "new":
        new[1] = 21
    if what == "long":
        lens[1] = 25
    if what == "page":
        table[1][0] = 10
    if what == "free":
        count = 0
    if what == "room":
        room = 3
    if what == "count":
        count = 4
    t = bskv.bskv_build_page_table(
        _i32(lens, cuda), _i32(table, cuda), 8, 10, new_lens=_i32(new, cuda), free_pages=_i32(free, cuda),
        free_count=_i32([count], cuda), max_tokens=room)
    assert bskv.bskv_get_device_status() == 6
    if what in ("negative", "new", "long"):  # the next request takes the free page that it would have had
        assert t.kv_indptr.tolist() == [0, 2, 2, 3] and t.kv_last_page_len.tolist() == [1, 0, 4]
        assert t.batch_indices.tolist() == [0, 2, 2, 2, 2] + [-1] * 4
        assert t.slots.tolist() == [48, 56, 57, 58, 59] + [-1] * 4
    elif what == "page":
        assert t.kv_indices.tolist()[:6] == [0, 6, -1, 3, 7, 8]
        assert t.slots.tolist() == [48, 56, 57, 58, 59, 64, 65, 66, 67]
    elif what == "room":
        assert t.batch_indices.tolist() == [0, 1, 1] and t.qo_indptr.tolist() == [0, 1, 5, 9]
    else:
        assert t.kv_indices.tolist()[:6] == [0, -1, 2, 3, -1, -1] and t.free_left.tolist() == [0]
        assert t.slots.tolist() == [-1] * 9


def test_pages_of_rejected_drafts_go_back_to_the_free_list(cuda):
    """Requests that grow by drafted tokens and lose some of them: with their pages put back before the next step, every
    page of the pool is listed by one request or free, after every step."""
    ps, pool, batch, most = 4, 40, 3, 10
    rng = np.random.default_rng(0)
    i32 = dict(dtype=torch.int32, device=cuda)
    free_pages, free_count = torch.tensor(rng.permutation(pool), **i32), torch.full((1,), pool, **i32)
    block_table, lens = torch.full((batch, most), -1, **i32), torch.zeros(batch, **i32)
    for step in range(30):
        new = torch.tensor(rng.integers(0, 7, batch), **i32)
        new = torch.minimum(new, most * ps - lens)
        lens += new
        t = bskv.bskv_build_page_table(lens, block_table, ps, pool, new_lens=new, free_pages=free_pages, free_count=free_count,
                                       max_tokens=24)
        free_count.copy_(t.free_left)
        assert bskv.bskv_get_device_status() == 0
        n = int(t.kv_indptr[-1])
        assert sorted(t.kv_indices[:n].tolist() + free_pages[:int(free_count)].tolist()) == list(range(pool))
        drop = torch.minimum(torch.tensor(rng.integers(0, 9, batch), **i32), lens)
        if step % 10 == 9:
            drop = lens.clone()  # the requests end
        for b in range(batch):
            old = block_table[b, -(-int(lens[b] - drop[b]) // ps):-(-int(lens[b]) // ps)]
            at = int(free_count)
            free_pages[at:at + old.numel()] = old
            free_count += old.numel()
        lens -= drop
