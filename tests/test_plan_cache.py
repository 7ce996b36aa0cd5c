"""Plans and calls of the 4-bit cache, the token scores and the eviction on the host: every request
and token has its place once, and what does not fit is refused before anything is launched."""

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
from oracle import plan_ref

SMS = 152
PTR, IDX, LAST = [0, 3, 3, 5], [4, 0, 2, 1, 5], [3, 0, 16]  # 35, 0 and 32 tokens in pages of 16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _table(lens, ps, seed=0):
    n = [-(-x // ps) for x in lens]
    perm = np.random.default_rng(seed).permutation(sum(n) + 1)[:sum(n)]
    return ([0] + list(np.cumsum(n)), perm.tolist(),
            [x - (c - 1) * ps if c else 0 for x, c in zip(lens, n)], sum(n) + 1)


def _decode(ptr=PTR, idx=IDX, last=LAST, pages=6, ps=16, hq=8, hkv=2, d=128, dtype=torch.bfloat16, **k):
    return bskv.bskv_plan_decode_fp4(_i32(ptr), _i32(idx), _i32(last), pages, ps, hq, hkv, d, dtype,
                                     num_sms=k.pop("num_sms", SMS), **k)


def _weights(qo=None, ptr=PTR, idx=IDX, last=LAST, pages=6, ps=16, hq=8, hkv=2, d=128,
             dtype=torch.bfloat16, **k):
    return bskv.bskv_plan_attn_weights(None if qo is None else _i32(qo), _i32(ptr), _i32(idx), _i32(last),
                                       pages, ps, hq, hkv, d, dtype=dtype, num_sms=k.pop("num_sms", SMS), **k)


def _evict(keep=(20, 5, 10), sink=2, recent=3, ptr=PTR, idx=IDX, last=LAST, pages=9, ps=16, hkv=2, d=128,
           **k):
    return bskv.bskv_plan_evict(_i32(ptr), _i32(idx), _i32(last), _i32(list(keep)), sink, recent, pages, ps,
                                hkv, d, num_sms=k.pop("num_sms", SMS),
                                **{n: _i32(x) for n, x in k.items()})


# ---- what plans hold --------------------------------------------------------------------

def _records(meta, count):
    return np.array(meta[-8 * count:]).reshape(count, 8) if count else np.zeros((0, 8), dtype=int)


def _check_walk(meta, lens, hkv, ptr):
    """Every (request, kv head)'s tokens once, in whole tiles, each worker's in the records' order."""
    s = plan_ref.sections(meta)
    r = _records(meta, len(s["chunks"]))
    assert s["worker_ptr"][0] == 0 and s["worker_ptr"][-1] == len(r)
    assert (np.diff(s["worker_ptr"]) > 0).all()
    seen = {u: [] for u in range(len(lens) * hkv)}
    for unit, begin, end, slot, pbase, item, first, pieces in r.tolist():
        assert pbase == ptr[unit // hkv] and begin % 32 == 0
        seen[unit].append((begin, end, slot, first, pieces))
    for u, cs in seen.items():
        at = 0
        for i, (begin, end, slot, first, pieces) in enumerate(sorted(cs)):
            assert begin == at and end > begin
            at = end
            if slot >= 0:
                assert pieces == len(cs) and slot == first + i
        assert at == lens[u // hkv]
    return s, r, seen


@pytest.mark.parametrize("lens,hkv", [([35, 0, 32], 2), ([100000], 1), ([5] * 400, 3), ([1, 4000, 7], 8)])
def test_decode_plan_takes_every_token_once(lib, lens, hkv):
    ptr, idx, last, pages = _table(lens, 16)
    meta = _decode(ptr, idx, last, pages, hq=4 * hkv, hkv=hkv).metadata()
    s, r, seen = _check_walk(meta, lens, hkv, ptr)
    assert s["workers"] <= SMS * 4 * 4
    # what each piece publishes, and who merges it
    for u, cs in seen.items():
        assert all((c[2] >= 0) == (len(cs) > 1) for c in cs)
    slots = sorted(x for x in r[:, 3].tolist() if x >= 0)
    assert slots == list(range(len(slots)))


def test_decode_plan_is_reproducible_and_bounded_by_max_workers(lib):
    ptr, idx, last, pages = _table([3000, 10, 900], 16)
    a = _decode(ptr, idx, last, pages, max_workers=7).metadata()
    assert a == _decode(ptr, idx, last, pages, max_workers=7).metadata()
    assert plan_ref.sections(a)["workers"] <= 7


@pytest.mark.parametrize("lens,hkv", [([35, 0, 32], 2), ([70000], 1), ([5] * 300, 3)])
def test_weights_plan_of_a_step(lib, lens, hkv):
    ptr, idx, last, pages = _table(lens, 16)
    p = _weights(None, ptr, idx, last, pages, hq=4 * hkv, hkv=hkv)
    _, r, _ = _check_walk(p.metadata(), lens, hkv, ptr)
    assert (r[:, 3] == -1).all()  # every score is complete where it is computed
    assert p.info["q_shape"] == (len(lens), 4 * hkv, 128)


def test_weights_plan_of_windows(lib):
    """More than 16 query rows per kv head: a record per request with tokens."""
    lens, hkv = [300, 0, 128, 1], 2
    ptr, idx, last, pages = _table(lens, 16)
    p = _weights([0, 40, 41, 41, 42], ptr, idx, last, pages, hq=2, hkv=hkv)
    r = _records(p.metadata(), 3)
    assert r[:, :6].tolist() == [[0, 3, 300, ptr[0], 0, 40], [6, 1, 128, ptr[2], 41, 0], [8, 1, 1, ptr[3], 41, 1]]
    assert p.info["q_shape"] == (42, 2, 128)


def test_evict_plan(lib):
    p = _evict()
    assert p.info["kept_indptr"] == [0, 20, 20, 30]
    c = plan_ref.sections(p.metadata())["chunks"]
    assert [list(x) for x in c] == [[35, 20, 0, 0], [0, 0, 20, 3], [32, 10, 20, 3]]
    p = _evict(keep=(20, 0, 40), dst_indptr=[0, 2, 2, 4], dst_indices=[7, 3, 6, 8])
    assert p.info["kept_indptr"] == [0, 20, 20, 52]


def test_plans_of_a_pool_far_larger_than_the_table(lib):
    """What a plan takes depends on the pages listed, not on the pool."""
    big = 2 ** 31 - 1
    assert _weights(pages=big).info["num_pages"] == big
    assert _evict(pages=big).info["num_pages"] == big
    _evict(pages=big, dst_indptr=[0, 2, 2, 3], dst_indices=[7, big - 1, 8])
    with pytest.raises(bskv.BskvError):
        _evict(pages=big, dst_indptr=[0, 2, 2, 3], dst_indices=[7, big, 8])


def test_plans_of_nothing(lib):
    for p in (_decode([0], [], [], 0), _weights(None, [0], [], [], 0), _evict((), 0, 0, [0], [], [], 0)):
        assert p.info["batch"] == 0
    assert _decode([0, 0], [], [0], 0).info["batch"] == 1


# ---- refusals ---------------------------------------------------------------------------

BAD_TABLES = [
    dict(ptr=[0, 3, 2, 5]), dict(ptr=[1, 3, 3, 5]), dict(idx=[4, 0, 2, 1, 99]), dict(idx=[4, 0, 2, 1, -1]),
    dict(last=[0, 0, 16]), dict(last=[17, 0, 16]), dict(last=[3, 0]), dict(idx=[4, 0, 2, 1]),
]
BAD_SHAPES = [dict(ps=12), dict(ps=24), dict(ps=0), dict(d=96), dict(d=256), dict(hkv=0), dict(num_sms=0),
              dict(pages=-1)]


@pytest.mark.parametrize("bad", BAD_TABLES + BAD_SHAPES)
@pytest.mark.parametrize("make", [_decode, _weights, _evict])
def test_plans_refuse(lib, make, bad):
    with pytest.raises((ValueError, RuntimeError, NotImplementedError, bskv.BskvError)):
        make(**bad)


@pytest.mark.parametrize("bad", [dict(hq=7), dict(hq=34), dict(dtype=torch.float32), dict(max_workers=-1)])
def test_decode_plan_refuses(lib, bad):
    with pytest.raises((ValueError, KeyError, bskv.BskvError)):
        _decode(**bad)


@pytest.mark.parametrize("bad", [
    dict(hq=7), dict(hq=258), dict(dtype=torch.float32), dict(qo=[0, 1, 2]), dict(qo=[0, 2, 1, 3]),
    dict(qo=[1, 2, 3, 4]), dict(idx=[4, 0, 2, 1, 0]),  # a page of scores has one owner
])
def test_weights_plan_refuses(lib, bad):
    with pytest.raises((ValueError, KeyError, bskv.BskvError)):
        _weights(**bad)


@pytest.mark.parametrize("bad", [
    dict(keep=(20, 5)), dict(keep=(20, -1, 10)), dict(sink=-1), dict(recent=-1),
    dict(keep=(4, 0, 10)),                                         # fewer than are protected
    dict(idx=[4, 0, 2, 1, 0]),                                     # in place, a page listed twice
    dict(dst_indptr=[0, 2, 2, 3]),                                 # without its pages
    dict(dst_indptr=[0, 1, 1, 2], dst_indices=[7, 8]),             # 20 tokens into one page
    dict(dst_indptr=[0, 2, 2, 3], dst_indices=[7, 7, 8]),          # twice
    dict(dst_indptr=[0, 2, 2, 3], dst_indices=[7, 4, 8]),          # a source page
    dict(dst_indptr=[0, 2, 2, 3], dst_indices=[7, 9, 8]),          # no such page
    dict(dst_indptr=[0, 2, 1, 3], dst_indices=[7, 6, 8]),
])
def test_evict_plan_refuses(lib, bad):
    with pytest.raises((ValueError, bskv.BskvError)):
        _evict(**bad)


def test_evict_protects_only_where_something_leaves(lib):
    assert _evict(keep=(35, 0, 32), sink=30, recent=30).info["kept_indptr"] == [0, 35, 35, 67]


def _pools(d=128):
    return (torch.zeros(6, 2, 2, 16, d // 2, dtype=torch.uint8), torch.zeros(6, 2, 2, 16, d // 32, dtype=torch.uint8))


def test_calls_refuse_tensors_of_the_host(lib):
    codes, scales = _pools()
    q, rows = torch.zeros(3, 8, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    at = (_i32([0] * 4), _i32([0] * 4), _i32(PTR), _i32(IDX))
    sc, lse = torch.zeros(6, 2, 16), torch.zeros(3, 8)
    kv = torch.zeros(6, 2, 2, 16, 128, dtype=torch.bfloat16)
    for call in (lambda: bskv.bskv_run_decode_fp4(_decode(), q, codes, scales),
                 lambda: bskv.bskv_quantize_fp4_append_paged(rows, rows, *at, codes, scales),
                 lambda: bskv.bskv_dequantize_fp4_paged(codes, scales, *at),
                 lambda: bskv.bskv_run_attn_weights(_weights(), q, kv, lse, sc),
                 lambda: bskv.bskv_run_attn_weights_fp4(_weights(), q, codes, scales, lse, sc),
                 lambda: bskv.bskv_run_evict(_evict(pages=6), sc, kv),
                 lambda: bskv.bskv_run_evict_fp4(_evict(pages=6), sc, codes, scales)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_calls_refuse_what_is_no_tensor_and_other_plans(lib):
    codes, scales = _pools()
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        bskv.bskv_run_decode_fp4(_decode(), [1.0], codes, scales)
    with pytest.raises(TypeError):
        bskv.bskv_run_evict(_evict(), None, codes)
    for run, plan in ((bskv.bskv_run_decode_fp4, _weights()), (bskv.bskv_run_attn_weights, _decode()),
                      (bskv.bskv_run_evict_fp4, _decode())):
        with pytest.raises((ValueError, TypeError)):
            run(plan, q, codes, scales, q, q) if run is bskv.bskv_run_attn_weights else run(plan, q, codes, scales)


def test_entry_points_refuse_null_and_unaligned(lib):
    """The C entry points check what they can see before the first CUDA call."""
    import ctypes
    c = bskv.load_library()
    st = (ctypes.c_int64 * 4)(64, 64, 64, 64)
    assert c.bskv_run_decode_fp4(None, 16, st, 16, st, 16, st, 16, st, None, 0.0, None, 0, None) == 1
    assert c.bskv_run_evict(None, 16, st, 1, 16, st, 16, None) == 1
    assert c.bskv_run_attn_weights(None, 16, st, 16, st, 16, 16, st, 1.0, 0.0, None) == 1
    for plan, call in ((_decode(), lambda h: c.bskv_run_decode_fp4(h, 16, st, 16, st, 16, st, 16, st, None, 0.0, None, 0, None)),
                       (_weights(), lambda h: c.bskv_run_attn_weights(h, 16, st, 16, st, 16, 16, st, 1.0, 0.0, None)),
                       (_evict(), lambda h: c.bskv_run_evict(h, 16, st, 1, 16, st, 16, None))):
        assert call(plan.handle) == 1  # not uploaded
        assert "upload" in c.bskv_last_error_message().decode()
    args = dict(k=16, v=16, dt=1, nnz=1, heads=2, dim=128, codes=16, scales=16, batch=1, ps=16, pages=1)

    def append(**bad):
        a = dict(args, **bad)
        return c.bskv_quantize_fp4_append_paged(a["k"], st, a["v"], st, a["dt"], a["nnz"], a["heads"], a["dim"],
                                                16, 16, 16, 16, a["batch"], a["ps"], a["pages"], a["codes"], st,
                                                a["scales"], st, None)
    for bad in (dict(k=None), dict(k=24), dict(codes=8), dict(scales=None), dict(dim=96), dict(ps=12), dict(nnz=-1),
                dict(heads=0), dict(heads=129), dict(dt=77), dict(pages=-1), dict(batch=-1)):
        assert append(**bad) in (1, 2), bad


_HUGE = """
import resource, sys
import torch
import block_sparse_kv_gb300 as bskv
bskv.load_library()
pages = int(open("/proc/self/statm").read().split()[0])
limit = pages * resource.getpagesize() + (1 << 30)
resource.setrlimit(resource.RLIMIT_AS, (limit, limit))
z = torch.zeros(65, dtype=torch.int32)
for heads, message in ((1 << 30, "too many tokens"), (1 << 22, "out of host memory")):
    try:
        bskv.bskv_plan_decode_fp4(z, [], z, 0, 16, heads, heads, 128, num_sms=152)
    except bskv.BskvError as e:
        assert e.status == "ERR_UNSUPPORTED" and message in str(e), e
    else:
        raise AssertionError(heads)
t = torch.zeros(5001, dtype=torch.int32)
try:
    bskv.bskv_plan_attn_weights(None, t, [], t, 0, 16, 65535, 65535, 128, num_sms=152)
except bskv.BskvError as e:
    assert e.status == "ERR_UNSUPPORTED" and "out of host memory" in str(e), e
else:
    raise AssertionError("made")
assert bskv.bskv_plan_decode_fp4(z[:2], [], z[:1], 0, 16, 8, 8, 128, num_sms=152) is not None
"""


def test_plans_past_the_host_memory_are_refused(lib):
    """A child process with a gigabyte to spare: statuses, no exception out of a C entry point."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _HUGE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
