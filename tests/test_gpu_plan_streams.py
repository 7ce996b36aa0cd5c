"""Plans whose upload and runs are on different streams: a run waits for the upload, and a plan that is
dropped leaves its workspaces to nobody else before its runs are done."""

import gc

import pytest
import torch

import block_sparse_kv_gb300 as bskv

pytestmark = pytest.mark.gpu
PS, H, HQ, D = 16, 2, 16, 128
LENS = (700, 129, 1, 40)


def _inputs(cuda):
    g = torch.Generator().manual_seed(3)
    n = [-(-x // PS) for x in LENS]
    table = (torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32),
             torch.randperm(sum(n), generator=g).to(torch.int32),
             torch.tensor([x - (c - 1) * PS for x, c in zip(LENS, n)], dtype=torch.int32))
    pages = sum(n)
    return dict(table=table, pages=pages, q=torch.randn(4, HQ, D, generator=g).bfloat16().to(cuda),
                codes=torch.randint(0, 256, (pages, 2, H, PS, D // 2), generator=g, dtype=torch.uint8).to(cuda),
                scales=torch.randint(120, 128, (pages, 2, H, PS, D // 32), generator=g, dtype=torch.uint8).to(cuda),
                kv=torch.randn(pages, 2, H, PS, D, generator=g).bfloat16().to(cuda),
                scores=torch.rand(pages, H, PS, generator=g).to(cuda), lse=torch.full((4, HQ), 5.0, device=cuda))


def _plan(kind, s):
    t, n = s["table"], s["pages"]
    if kind == "decode_fp4":
        return bskv.bskv_plan_decode_fp4(*t, n, PS, HQ, H, D, max_workers=9)
    if kind == "weights":
        return bskv.bskv_plan_attn_weights(None, *t, n, PS, HQ, H, D)
    if kind == "evict":
        return bskv.bskv_plan_evict(*t, [300, 129, 1, 20], 2, 8, n, PS, H, D)
    return bskv.bskv_plan_decode(*t, n, PS, HQ, H, D, torch.bfloat16, max_workers=9)


def _run(kind, p, s):
    """The run's outputs; inputs that it changes are copies made on the current stream."""
    if kind == "decode_fp4":
        return bskv.bskv_run_decode_fp4(p, s["q"], s["codes"], s["scales"], return_lse=True)
    if kind == "weights":
        return (bskv.bskv_run_attn_weights(p, s["q"], s["kv"], s["lse"], s["scores"].clone()),)
    if kind == "evict":
        pool, scores = s["kv"].clone(), s["scores"].clone()
        return bskv.bskv_run_evict(p, scores, pool), pool, scores
    return bskv.bskv_run_decode(p, s["q"], s["kv"], return_lse=True)


def _busy():
    """Some tens of milliseconds of work on the current stream."""
    a = torch.ones(8192, 8192, device="cuda", dtype=torch.bfloat16)
    for _ in range(40):
        a = a @ a * 2.0 ** -13
    return a


KINDS = ["decode_fp4", "weights", "evict", "decode"]


@pytest.mark.parametrize("kind", KINDS)
def test_a_run_waits_for_an_upload_on_another_stream(cuda, kind):
    s = _inputs(cuda)
    want = _run(kind, _plan(kind, s).upload(cuda), s)
    _busy()
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    p = _plan(kind, s)
    with torch.cuda.stream(one):
        busy = _busy()
        p.upload(cuda)
        again = torch.cuda.Event()
        again.record()
    with torch.cuda.stream(two):
        got = _run(kind, p, s)
        done = two.query()
        assert again.query() or not done  # not done before the upload
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    del busy


@pytest.mark.parametrize("kind", KINDS)
def test_a_plan_dropped_after_a_run_on_another_stream(cuda, kind):
    s = _inputs(cuda)
    want = _run(kind, _plan(kind, s).upload(cuda), s)
    _busy()
    p = _plan(kind, s).upload(cuda)
    torch.cuda.synchronize()
    gc.collect()
    side = torch.cuda.Stream()
    sizes = [(w.data_ptr(), w.numel()) for w in (p.int_ws, p.float_ws) if w is not None]
    with torch.cuda.stream(side):
        busy = _busy()
        got = _run(kind, p, s)
        done = torch.cuda.Event()
        done.record()
    del p
    later = [torch.full((n,), 255, dtype=torch.uint8, device=cuda) for _, n in sizes for _ in range(3)]
    if not done.query():
        assert not {x.data_ptr() for x in later} & {at for at, _ in sizes}
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    del busy


def test_a_graph_on_a_stream_of_its_own(cuda):
    """A capture takes a plan that was uploaded, and has run, on other streams."""
    s = _inputs(cuda)
    p = _plan("decode_fp4", s).upload(cuda)
    want = _run("decode_fp4", p, s)
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bskv.bskv_run_decode_fp4(p, s["q"], s["codes"], s["scales"], out=out, lse=lse)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
