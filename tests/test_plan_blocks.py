"""Plans and calls of the block-sparse decode step on the host: runs of the attention cover every place once, and
what does not fit is refused before anything is launched."""

import ctypes

import pytest
import torch

import block_sparse_kv_gb300 as bskv

A = 1 << 20  # a 16-byte aligned address that nothing reads


def _plan(tokens=4, blocks=64, pages=100, ps=16, hq=8, hkv=2, d=128, top=16, sink=1, recent=2, dtype=torch.bfloat16, sms=152):
    return bskv.bskv_plan_decode_blocks(tokens, blocks, pages, ps, hq, hkv, d, top, sink, recent, dtype, num_sms=sms)


def test_plan_sizes(lib):
    p = _plan()
    ints, floats = p.workspace_sizes()
    assert ints >= 64 + 4 * 2 * 8  # two counters per (token, kv head)
    # fp64 keys and fp32 scores of 8 rows of 64 blocks, and partial states
    assert floats >= 8 * 64 * 12 + 8 * 4 * 128 * 4
    assert _plan(tokens=0).workspace_sizes()[1] == 0
    # the queries of a long chunk share the room for scores
    assert _plan(tokens=4096, blocks=1024, hkv=1).workspace_sizes()[1] < 2 * 2048 * 1024 * 12 + 4096 * 80 * 128 * 4


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), "ERR_INVALID_ARG"), (dict(blocks=0), "ERR_INVALID_ARG"), (dict(top=0), "ERR_INVALID_ARG"),
    (dict(recent=0), "ERR_INVALID_ARG"), (dict(sink=-1), "ERR_INVALID_ARG"), (dict(sink=15, recent=2), "ERR_INVALID_ARG"),
    (dict(pages=-1), "ERR_INVALID_ARG"), (dict(ps=0), "ERR_INVALID_ARG"), (dict(hq=9), "ERR_INVALID_ARG"),
    (dict(hkv=0), "ERR_INVALID_ARG"), (dict(sms=0), "ERR_INVALID_ARG"), (dict(blocks=49153), "ERR_UNSUPPORTED"),
    (dict(ps=24), "ERR_UNSUPPORTED"), (dict(d=96), "ERR_UNSUPPORTED"), (dict(hq=34), "ERR_UNSUPPORTED"),
    (dict(dtype=torch.float32), "ERR_UNSUPPORTED"), (dict(tokens=1 << 24), "ERR_UNSUPPORTED"),
    (dict(tokens=1 << 16, hkv=64, hq=64, top=1024, blocks=2048), "ERR_UNSUPPORTED"),
])
def test_plan_refusals(lib, kw, status):
    with pytest.raises(bskv.BskvError) as e:
        _plan(**kw)
    assert e.value.status == status and "plan_decode_blocks" in str(e.value)


@pytest.mark.parametrize("kw", [dict(top=1 << 27, sms=1), dict(top=1 << 25, ps=64, sms=1), dict(top=1, sink=0, recent=1, ps=1 << 30),
                                dict(top=64, ps=1 << 28, sms=1)])
def test_plan_of_lists_past_31_bits(lib, kw):
    """Lists whose steps, or a team's share of which, the kernels' 31 bits would not hold."""
    with pytest.raises(bskv.BskvError) as e:
        _plan(tokens=1, hq=1, hkv=1, **kw)
    assert e.value.status == "ERR_UNSUPPORTED" and "plan_decode_blocks" in str(e.value)


def test_plan_of_a_type_without_a_code(lib):
    with pytest.raises(ValueError, match="dtype"):
        _plan(dtype=torch.float64)


def _strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


def _call(name, *args):
    lib = bskv.load_library()
    return bskv.STATUS[getattr(lib, name)(*args)], lib.bskv_last_error_message().decode()


def _table(**kw):
    a = dict(lens=A, news=None, batch=2, ps=16, table=A, stride=4, max_pages=4, pages=9, free=None, max_free=0, count=None,
             left=None, indptr=A, indices=A, entries=8, last=A, qo=A, req=A, pos=A, slots=A, tokens=2)
    a.update(kw)
    return _call("bskv_build_page_table", *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), "ERR_INVALID_ARG"), (dict(ps=0), "ERR_INVALID_ARG"), (dict(tokens=-1), "ERR_INVALID_ARG"),
    (dict(lens=None), "ERR_INVALID_ARG"), (dict(table=None), "ERR_INVALID_ARG"), (dict(indptr=None), "ERR_INVALID_ARG"),
    (dict(req=None), "ERR_INVALID_ARG"), (dict(entries=7), "ERR_INVALID_ARG"), (dict(stride=3), "ERR_INVALID_ARG"),
    (dict(pos=A + 8), "ERR_INVALID_ARG"), (dict(lens=A + 2), "ERR_INVALID_ARG"), (dict(free=A, count=A), "ERR_INVALID_ARG"),
    (dict(free=A, count=A, left=A), "ERR_INVALID_ARG"), (dict(batch=8193, entries=1 << 20), "ERR_UNSUPPORTED"),
    (dict(max_pages=1 << 27, ps=16, stride=1 << 27, entries=1 << 28), "ERR_UNSUPPORTED"),
])
def test_page_table_refusals(lib, kw, status):
    got, text = _table(**kw)
    assert got == status and "build_page_table" in text


def _append(**kw):
    s2, s4 = _strides(1024, 128), _strides(8192, 4096, 2048, 128)
    a = dict(q=A, qs=s2, k=A, ks=s2, v=A, vs=s2, dtype=1, nnz=3, hq=8, hkv=2, d=128, wq=None, wk=None, eps=1e-6, table=A,
             table_type=2, limit=10, rot=128, neox=1, at=None, req=A, pos=A, indptr=A, indices=A, batch=1, ps=16, pages=5,
             out=A, outs=s2, cache=A, cs=s4)
    a.update(kw)
    return _call("bskv_norm_rope_append_paged", *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), "ERR_UNSUPPORTED"), (dict(d=96), "ERR_UNSUPPORTED"), (dict(nnz=-1), "ERR_INVALID_ARG"),
    (dict(rot=24), "ERR_UNSUPPORTED"), (dict(rot=144), "ERR_INVALID_ARG"), (dict(table=None), "ERR_INVALID_ARG"),
    (dict(table=A + 4), "ERR_INVALID_ARG"), (dict(table_type=0), "ERR_UNSUPPORTED"), (dict(eps=-1.0), "ERR_INVALID_ARG"),
    (dict(eps=float("nan")), "ERR_INVALID_ARG"), (dict(q=None, out=None, k=None, v=None, cache=None), "ERR_INVALID_ARG"),
    (dict(q=None), "ERR_INVALID_ARG"), (dict(out=None), "ERR_INVALID_ARG"), (dict(v=None), "ERR_INVALID_ARG"),
    (dict(q=A + 8), "ERR_INVALID_ARG"), (dict(wq=A + 2), "ERR_INVALID_ARG"), (dict(req=None), "ERR_INVALID_ARG"),
    (dict(indptr=None), "ERR_INVALID_ARG"), (dict(pos=A + 1), "ERR_INVALID_ARG"), (dict(qs=_strides(1028, 128)), "ERR_INVALID_ARG"),
    (dict(cs=_strides(8192, 4096, 2048, 132)), "ERR_INVALID_ARG"), (dict(hq=0), "ERR_INVALID_ARG"),
    (dict(pages=1 << 31), "ERR_UNSUPPORTED"), (dict(nnz=1 << 40), "ERR_UNSUPPORTED"),
])
def test_append_refusals(lib, kw, status):
    got, text = _append(**kw)
    assert got == status and "norm_rope_append_paged" in text


def _bounds(**kw):
    a = dict(cache=A, cs=_strides(8192, 4096, 2048, 128), dtype=1, hkv=2, d=128, ps=16, pages=5, req=A, pos=A, nnz=3, indptr=A,
             indices=A, last=A, batch=1, bounds=A, bs=_strides(512, 256))
    a.update(kw)
    return _call("bskv_block_bounds_paged", *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), "ERR_UNSUPPORTED"), (dict(d=32), "ERR_UNSUPPORTED"), (dict(ps=0), "ERR_INVALID_ARG"),
    (dict(nnz=-1), "ERR_INVALID_ARG"), (dict(cache=None), "ERR_INVALID_ARG"), (dict(bounds=A + 8), "ERR_INVALID_ARG"),
    (dict(bs=_strides(512, 128)), "ERR_INVALID_ARG"), (dict(last=None), "ERR_INVALID_ARG"), (dict(cs=None), "ERR_INVALID_ARG"),
    (dict(pages=1 << 31), "ERR_UNSUPPORTED"),
])
def test_bounds_refusals(lib, kw, status):
    got, text = _bounds(**kw)
    assert got == status and "block_bounds_paged" in text


def test_runs_of_other_or_new_plans_are_refused(lib):
    p = _plan()
    table = bskv.bskv_plan_mla_sparse([8], 1, 1, 4, 64, num_sms=4)
    for plan, text in ((p, "not uploaded"), (table, "not a block-sparse")):
        got, msg = _call("bskv_run_select_blocks", plan.handle, A, _strides(1024, 128), A, _strides(512, 256), A, A, A, A, 1, A, A,
                         1 << 30, None)
        assert got == "ERR_INVALID_ARG" and text in msg
        got, msg = _call("bskv_run_decode_blocks", plan.handle, A, _strides(1024, 128), A, _strides(8192, 4096, 2048, 128), A, A, A, A,
                         A, 1, A, _strides(1024, 128), None, 0.0, A, 1 << 30, None)
        assert got == "ERR_INVALID_ARG" and text in msg


def test_binding_refuses_tensors_on_the_host(lib):
    i = torch.zeros(4, dtype=torch.int32)
    q, kv = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(9, 2, 2, 16, 128, dtype=torch.bfloat16)
    bounds = torch.zeros(9, 2, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bskv.bskv_build_page_table(i, torch.zeros(4, 3, dtype=torch.int32), 16, 9)
    with pytest.raises(ValueError, match="CUDA"):
        bskv.PageTable(i, i, i, i, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        bskv.bskv_norm_rope_append_paged(q, q[:, :2], q[:, :2], torch.zeros(9, 128), i, i, i, i, kv)
    with pytest.raises(ValueError, match="CUDA"):
        bskv.bskv_block_bounds_paged(kv, bounds, i, i, i, i, i[:3])
    p = _plan(pages=9)
    with pytest.raises(ValueError, match="CUDA"):
        bskv.bskv_run_select_blocks(p, q, bounds, i, i, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        bskv.bskv_run_decode_blocks(p, q, kv, torch.zeros(4, 2, 16, dtype=torch.int32), i, i, i, i)
    with pytest.raises(ValueError, match="decode_blocks plan"):
        bskv.bskv_run_select_blocks(None, q, bounds, i, i, i, i)
    with pytest.raises(ValueError, match="give k, v"):
        bskv.bskv_norm_rope_append_paged(q, q, None, None, i, i, i, i, kv)


@pytest.mark.parametrize("tokens,blocks,hq,hkv", [(2048, 8192, 32, 8), (1 << 15, 8192, 8, 2), (512, 49152, 64, 64), (2048, 2048, 32, 8)])
def test_workspace_of_long_chunks(lib, tokens, blocks, hq, hkv):
    """Scores of long chunks share 64 MB; the rest are partial states, which grow with the queries alone."""
    states = (tokens * hkv + 8 * 152) * (hq // hkv) * 129 * 4
    assert _plan(tokens=tokens, blocks=blocks, hq=hq, hkv=hkv).workspace_sizes()[1] <= (64 << 20) + states + 4096


def test_workspace_of_a_query_past_the_scores_share(lib):
    """One query's scores always have room."""
    one, two = (_plan(tokens=t, blocks=49152, hq=400, hkv=400).workspace_sizes()[1] for t in (1, 2))
    assert one >= 400 * 49152 * 4 and two - one < 400 * 49152
