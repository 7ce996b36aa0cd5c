"""The block-sparse decode step as a server runs it: one captured graph over batches that grow, other streams, caches
whose offsets pass 32 bits, chunks of many queries, and refusals of the binding."""

import math

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
from blocks_util import batch, lists, pages_of, to64
from oracle import blocks as ob

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


class Server:
    """A paged cache whose requests grow by rows of an already projected q, k and v; every buffer of a step is made once."""

    def __init__(self, cuda, rows, requests, most, ps, hq, hkv, d, top, sink, recent, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        self.g, self.shape = g, (hq, hkv, d)
        pool = requests * most + 2
        i32 = dict(dtype=torch.int32, device=cuda)
        self.ps, self.dtype, self.cuda = ps, dtype, cuda
        self.lens, self.new = torch.zeros(requests, **i32), torch.zeros(requests, **i32)
        self.block_table = torch.full((requests, most), -1, **i32)
        self.free_pages = torch.randperm(pool, generator=g).to(**i32)
        self.free_count = torch.full((1,), pool, **i32)
        self.table = bskv.PageTable(torch.zeros(requests + 1, **i32), torch.zeros(requests * most, **i32), torch.zeros(requests, **i32),
                                    torch.zeros(requests + 1, **i32), torch.zeros(rows, **i32), torch.zeros(rows, **i32),
                                    torch.zeros(rows, dtype=torch.int64, device=cuda), torch.zeros(1, **i32))
        kw = dict(dtype=dtype, device=cuda)
        self.kv = torch.full((pool, 2, hkv, ps, d), float("nan"), **kw)
        self.bounds = torch.full((pool, hkv, 2, d), float("nan"), **kw)
        self.q, self.k, self.v = torch.zeros(rows, hq, d, **kw), torch.zeros(rows, hkv, d, **kw), torch.zeros(rows, hkv, d, **kw)
        self.q_out, self.out = torch.zeros(rows, hq, d, **kw), torch.zeros(rows, hq, d, **kw)
        self.lse = torch.zeros(rows, hq, device=cuda)
        self.blocks = torch.zeros(rows, hkv, top, **i32)
        self.wq, self.wk = (1 + 0.1 * torch.randn(d, generator=g)).to(**kw), (1 + 0.1 * torch.randn(d, generator=g)).to(**kw)
        angle = torch.arange(most * ps)[:, None] / 10000 ** (torch.arange(d // 2)[None] / (d // 2))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(cuda)
        self.plan = bskv.bskv_plan_decode_blocks(rows, most, pool, ps, hq, hkv, d, top, sink, recent, dtype).upload(cuda)
        self.pick = (top, sink, recent)

    def step(self):
        t = self.table
        bskv.bskv_build_page_table(self.lens, self.block_table, self.ps, self.kv.shape[0], new_lens=self.new,
                                   free_pages=self.free_pages, free_count=self.free_count, out=t)
        self.free_count.copy_(t.free_left)
        where = t.batch_indices, t.positions, t.kv_indptr, t.kv_indices
        bskv.bskv_norm_rope_append_paged(self.q, self.k, self.v, self.cos_sin, *where, self.kv, q_weight=self.wq,
                                         k_weight=self.wk, q_out=self.q_out)
        bskv.bskv_block_bounds_paged(self.kv, self.bounds, *where, t.kv_last_page_len)
        bskv.bskv_run_select_blocks(self.plan, self.q_out, self.bounds, *where, blocks=self.blocks)
        bskv.bskv_run_decode_blocks(self.plan, self.q_out, self.kv, self.blocks, *where, out=self.out, lse=self.lse)

    def feed(self, new):
        """The next step's inputs."""
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.lens.add_(self.new)
        for x in (self.q, self.k, self.v):
            x.copy_(torch.randn(x.shape, generator=self.g).to(x.dtype))
        for x in (self.q_out, self.out):
            x.fill_(7.0)
        self.blocks.fill_(-9)

    def check(self):
        """Every output of the step from what the operator before it in the chain wrote."""
        top, sink, recent = self.pick
        hq, hkv, d = self.shape
        n = int(self.new.sum())
        req, pos = self.table.batch_indices.tolist(), self.table.positions.tolist()
        assert req[n:] == [-1] * (len(req) - n) and (self.out[n:] == 7.0).all() and (self.blocks[n:] == -9).all()
        q, kv, bounds = to64(self.q_out), to64(self.kv), to64(self.bounds)
        table, half = self.block_table.tolist(), torch.finfo(self.dtype).eps / 2
        lens = self.lens.tolist()
        for t in range(n):
            b, p = req[t], pos[t]
            assert p == lens[b] - int(self.new[b]) + (t - req.index(b))
            cs = to64(self.cos_sin[p])
            for name, w, got in (("q", self.wq, q[t]), ("k", self.wk, kv[table[b][p // self.ps], 0, :, p % self.ps])):
                ref, size = ob.norm_rope(to64(getattr(self, name)[t]), to64(w), 1e-6, cs, d, True)
                assert (np.abs(got - ref) <= half * np.abs(ref) + 33 * 2.0 ** -24 * size + 2.0 ** -25).all()
            assert torch.equal(self.kv[table[b][p // self.ps], 1, :, p % self.ps], self.v[t])
        for b in range(len(lens)):  # pages that hold new tokens
            for j in range((lens[b] - int(self.new[b])) // self.ps, -(-lens[b] // self.ps)):
                fill = min(self.ps, lens[b] - j * self.ps)
                if int(self.new[b]):
                    assert (bounds[table[b][j]] == ob.block_bounds(kv, table[b][j], fill)).all()
        for t in range(n):
            b, p = req[t], pos[t]
            pages = np.array(table[b][:p // self.ps + 1])
            for h in range(hkv):
                g = slice(h * hq // hkv, (h + 1) * hq // hkv)
                want = ob.select(ob.block_scores(q[t, g], bounds[pages, h]), top, sink, recent)
                assert self.blocks[t, h].tolist() == want
                at = np.array([x for j in want if j >= 0 for x in range(j * self.ps, min(p + 1, (j + 1) * self.ps))])
                ref, z, size = ob.attend(q[t, g], kv[pages[at // self.ps], 0, h, at % self.ps], kv[pages[at // self.ps], 1, h, at % self.ps],
                                         d ** -0.5)
                # rows of K have a norm of about 11, logits are below 2^4 and off by 136 roundings at most
                tol = half * np.abs(ref) + (half * 1.01 + 2.0 ** -11) * size + 2.0 ** -24
                assert (np.abs(to64(self.out[t, g]) - ref) <= tol).all()
                assert (np.abs(to64(self.lse[t, g]) - z) <= 2.0 ** -11).all()
        assert bskv.bskv_get_device_status() == 0


@pytest.mark.parametrize("dtype,hq,hkv,d,ps", [(BF, 8, 2, 128, 16), (FP, 6, 1, 64, 8)])
def test_one_graph_serves_a_growing_batch(cuda, dtype, hq, hkv, d, ps):
    s = Server(cuda, 160, 4, 24, ps, hq, hkv, d, 5, 1, 2, dtype, 1)
    s.feed([70, 0, 33, 1])  # prompts, and a request that is not there yet
    s.step()
    s.check()
    count = s.free_count.clone()
    s.feed([1, 0, 1, 1])
    saved = [x.clone() for x in (s.block_table, s.free_count, s.kv, s.bounds)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    for x, y in zip((s.block_table, s.free_count, s.kv, s.bounds), saved):  # a capture runs nothing
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert torch.equal(count, s.free_count)
    graph.replay()
    s.check()
    for new in ([1, 12, 1, 0], [4, 4, 4, 4], [0, 0, 0, 0], [1, 1, 1, 1], [90, 1, 1, 30]):
        s.feed(new)
        graph.replay()
        s.check()


def test_a_step_on_another_stream(cuda):
    """The same bits from a stream of its own, and from two plans at once on two streams."""
    made = []
    for _ in range(3):
        s = Server(cuda, 64, 3, 40, 16, 16, 4, 128, 6, 1, 2, BF, 5)
        s.feed([30, 20, 14])
        made.append(s)
    torch.cuda.synchronize()
    made[0].step()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for x, st in zip(made[1:], streams):
        with torch.cuda.stream(st):
            for _ in range(3):  # again, into the same pages: they are the requests' own
                x.step()
                x.free_count.add_(x.table.kv_indptr[-1])
    torch.cuda.synchronize()
    for x in made[1:]:
        for name in ("out", "lse", "blocks", "q_out"):
            assert torch.equal(getattr(x, name), getattr(made[0], name)), name


def test_offsets_past_32_bits(cuda):
    """Pages behind 2^31 elements of a cache, and bounds behind 2^31 bytes."""
    ps, hq, hkv, d, pages = 16, 4, 1, 64, (1 << 20) + 40
    kv = torch.empty(pages, 2, hkv, ps, d, dtype=BF, device=cuda)  # 4.3 GB
    bounds = torch.empty(pages, hkv, 16, d, dtype=BF, device=cuda)[:, :, :2]
    g = torch.Generator().manual_seed(0)
    s = batch([300, 40], [300, 40], ps, 0)
    s["pages"] = pages
    s["indices"] = (pages - 1 - torch.randperm(s["indices"].numel(), generator=g)).to(torch.int32)
    n = 340
    q, k, v = (torch.randn(n, h, d, generator=g).to(BF).to(cuda) for h in (hq, hkv, hkv))
    where = lists(s, cuda)
    q_out = bskv.bskv_norm_rope_append_paged(q, k, v, None, *where, kv)
    assert torch.equal(q_out, q)
    bskv.bskv_block_bounds_paged(kv, bounds, *where, s["last"].to(cuda))
    p = bskv.bskv_plan_decode_blocks(n, 19, pages, ps, hq, hkv, d, 4, 0, 1, BF)
    blocks = bskv.bskv_run_select_blocks(p, q, bounds, *where)
    out = bskv.bskv_run_decode_blocks(p, q, kv, blocks, *where)
    assert bskv.bskv_get_device_status() == 0
    # the same with a pool of its own pages alone
    low = dict(s, pages=40, indices=(s["indices"] - (pages - 40)).to(torch.int32))
    small = bskv.bskv_plan_decode_blocks(n, 19, 40, ps, hq, hkv, d, 4, 0, 1, BF)
    where = lists(low, cuda)
    kv2, bounds2 = kv[-40:].clone(), bounds[-40:].clone()
    assert torch.equal(bskv.bskv_run_select_blocks(small, q, bounds2, *where), blocks)
    assert torch.equal(bskv.bskv_run_decode_blocks(small, q, kv2, blocks, *where), out)
    i = [0, 299, 339]
    for t in i:
        page = int(low["indices"][int(low["indptr"][int(low["req"][t])]) + int(low["pos"][t]) // ps])
        assert torch.equal(kv2[page, 0, :, int(low["pos"][t]) % ps], k[t])


def test_a_chunk_of_more_queries_than_a_slice(cuda):
    """2100 queries of a prompt, each with blocks of its own."""
    ps, hq, hkv, d, top, n = 8, 2, 1, 64, 6, 2100
    s = batch([n], [n], ps, 1)
    g = torch.Generator().manual_seed(1)
    kv = torch.randn(s["pages"], 2, hkv, ps, d, generator=g).to(FP).to(cuda)
    q = torch.randn(n, hq, d, generator=g).to(FP).to(cuda)
    bounds = torch.zeros(s["pages"], hkv, 2, d, dtype=FP, device=cuda)
    where = lists(s, cuda)
    bskv.bskv_block_bounds_paged(kv, bounds, *where, s["last"].to(cuda))
    p = bskv.bskv_plan_decode_blocks(n, 263, s["pages"], ps, hq, hkv, d, top, 1, 1, FP)
    blocks = bskv.bskv_run_select_blocks(p, q, bounds, *where)
    out = bskv.bskv_run_decode_blocks(p, q, kv, blocks, *where)
    b64, q64, kv64 = to64(bounds), to64(q), to64(kv)
    pages = pages_of(s, 0)
    for t in list(range(0, 60)) + list(range(60, n, 97)) + [2047, 2048, 2099]:
        want = ob.select(ob.block_scores(q64[t], b64[pages[:t // ps + 1], 0]), top, 1, 1)
        assert blocks[t, 0].tolist() == want
        at = np.array([x for j in want if j >= 0 for x in range(j * ps, min(t + 1, (j + 1) * ps))])
        ref, _, size = ob.attend(q64[t], kv64[pages[at // ps], 0, 0, at % ps], kv64[pages[at // ps], 1, 0, at % ps], d ** -0.5)
        assert (np.abs(to64(out[t]) - ref) <= 2.0 ** -11 * (np.abs(ref) + 1.01 * size) + 2.0 ** -11 * size + 2.0 ** -24).all()


@pytest.mark.parametrize("sms", [1, 3, 5, 40, 152])
@pytest.mark.parametrize("ps,top", [(16, 40), (64, 9), (8, 30)])
def test_runs_and_teams_of_any_size(cuda, sms, ps, top):
    """Plans for few and many SMs cut the rows in other places and share them among other numbers of warps."""
    lens, new, hq, hkv, d = [700, 3, 0, 641, 90], [2, 1, 0, 1, 2], 6, 2, 128
    s = batch(lens, new, ps, 2)
    g = torch.Generator().manual_seed(2)
    kv = torch.randn(s["pages"], 2, hkv, ps, d, generator=g).to(BF)
    q = torch.randn(sum(new), hq, d, generator=g).to(BF)
    rng = np.random.default_rng(2)
    blocks = np.full((sum(new), hkv, top), -1, dtype=np.int32)
    for t in range(sum(new)):
        seen = int(s["pos"][t]) // ps + 1
        for h in range(hkv):
            blocks[t, h, :min(top, seen)] = np.sort(rng.permutation(seen)[:min(top, seen)])
    p = bskv.bskv_plan_decode_blocks(sum(new), 100, s["pages"], ps, hq, hkv, d, top, dtype=BF, num_sms=sms)
    out, lse = bskv.bskv_run_decode_blocks(p, q.to(cuda), kv.to(cuda), torch.tensor(blocks).to(cuda), *lists(s, cuda), return_lse=True)
    k64, q64 = to64(kv), to64(q)
    for t in range(sum(new)):
        pages, pos = pages_of(s, int(s["req"][t])), int(s["pos"][t])
        for h in range(hkv):
            at = np.array([x for j in blocks[t, h] if j >= 0 for x in range(j * ps, min(pos + 1, (j + 1) * ps))])
            c = slice(3 * h, 3 * h + 3)
            ref, z, size = ob.attend(q64[t, c], k64[pages[at // ps], 0, h, at % ps], k64[pages[at // ps], 1, h, at % ps], 1 / math.sqrt(d))
            assert (np.abs(to64(out[t, c]) - ref) <= 2.0 ** -8 * (np.abs(ref) + 1.01 * size) + 2.0 ** -11 * size).all()
            assert (np.abs(to64(lse[t, c]) - z) <= 2.0 ** -11).all()
    assert bskv.bskv_get_device_status() == 0


def test_requests_that_share_pages_and_repeated_queries(cuda):
    """A prefix listed by two requests, and the same query row twice."""
    ps, hq, hkv, d, top = 16, 4, 2, 64, 3
    s = batch([100], [1], ps, 3)
    table = s["indices"].tolist()
    s["indptr"] = torch.tensor([0, 7, 14], dtype=torch.int32)
    s["indices"] = torch.tensor(table + table, dtype=torch.int32)
    s["req"], s["pos"] = torch.tensor([0, 1, 0], dtype=torch.int32), torch.tensor([99, 99, 99], dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    kv = torch.randn(s["pages"], 2, hkv, ps, d, generator=g).to(BF).to(cuda)
    q = torch.randn(1, hq, d, generator=g).to(BF).to(cuda).expand(3, -1, -1)
    bounds = torch.stack([kv[:, 0].amin(2), kv[:, 0].amax(2)], 2).contiguous()
    p = bskv.bskv_plan_decode_blocks(3, 7, s["pages"], ps, hq, hkv, d, top, dtype=BF)
    where = lists(s, cuda)
    blocks = bskv.bskv_run_select_blocks(p, q, bounds, *where)
    out = bskv.bskv_run_decode_blocks(p, q, kv, blocks, *where)
    for t in (1, 2):
        assert torch.equal(blocks[t], blocks[0]) and torch.equal(out[t], out[0])


def test_plans_without_queries(cuda):
    e = torch.empty(0, dtype=torch.int32, device=cuda)
    ptr = torch.zeros(1, dtype=torch.int32, device=cuda)
    p = bskv.bskv_plan_decode_blocks(0, 5, 9, 16, 4, 2, 64, 3)
    q, kv = torch.empty(0, 4, 64, dtype=BF, device=cuda), torch.zeros(9, 2, 2, 16, 64, dtype=BF, device=cuda)
    bounds = torch.zeros(9, 2, 2, 64, dtype=BF, device=cuda)
    blocks = bskv.bskv_run_select_blocks(p, q, bounds, e, e, ptr, e)
    assert blocks.shape == (0, 2, 3) and bskv.bskv_run_decode_blocks(p, q, kv, blocks, e, e, ptr, e).shape == (0, 4, 64)
    bskv.bskv_block_bounds_paged(kv, bounds, e, e, ptr, e, e)


def test_binding_refusals(cuda):
    ps, hq, hkv, d, top = 16, 4, 2, 64, 3
    s = batch([100, 20], [1, 1], ps, 3)
    kv = torch.zeros(s["pages"], 2, hkv, ps, d, dtype=BF, device=cuda)
    bounds = torch.zeros(s["pages"], hkv, 2, d, dtype=BF, device=cuda)
    q = torch.zeros(2, hq, d, dtype=BF, device=cuda)
    p = bskv.bskv_plan_decode_blocks(2, 7, s["pages"], ps, hq, hkv, d, top, dtype=BF)
    req, pos, indptr, indices = where = lists(s, cuda)
    last = s["last"].to(cuda)
    blocks = torch.zeros(2, hkv, top, dtype=torch.int32, device=cuda)
    sel, att = bskv.bskv_run_select_blocks, bskv.bskv_run_decode_blocks
    app, bnd, tab = bskv.bskv_norm_rope_append_paged, bskv.bskv_block_bounds_paged, bskv.bskv_build_page_table
    k = torch.zeros(2, hkv, d, dtype=BF, device=cuda)
    lens = torch.ones(2, dtype=torch.int32, device=cuda)
    bt = torch.zeros(2, 3, dtype=torch.int32, device=cuda)
    table = tab(lens, bt, ps, 9)
    for call in [
        lambda: sel(p, q.half(), bounds, *where), lambda: sel(p, q[:1], bounds, *where), lambda: sel(p, q, bounds[:-1], *where),
        lambda: sel(p, q, bounds.transpose(2, 3).contiguous().transpose(2, 3), *where), lambda: sel(p, q, bounds, req[:1], pos, indptr, indices),
        lambda: sel(p, q, bounds, req.long(), pos, indptr, indices), lambda: sel(p, q, bounds, req, pos, indptr[:0], indices),
        lambda: sel(p, q, bounds, *where, blocks=blocks[:, :, :2]), lambda: sel(p, q, bounds, *where, blocks=blocks.transpose(0, 1).contiguous().transpose(0, 1)),
        lambda: att(p, q, kv[:-1], blocks, *where), lambda: att(p, q, kv.half(), blocks, *where), lambda: att(p, q, kv, blocks[:1], *where),
        lambda: att(p, q, kv, blocks, *where, out=q[:, :, :1].expand(-1, -1, d)), lambda: att(p, q, kv, blocks, *where, lse=torch.zeros(2, hq, device=cuda).t().contiguous().t()),
        lambda: app(q, k, k, None, req, pos, indptr, indices, kv.float()), lambda: app(q, k, k[:1], None, req, pos, indptr, indices, kv),
        lambda: app(q, k, k, torch.zeros(9, 64, device=cuda).half(), req, pos, indptr, indices, kv),
        lambda: app(q, k, k, None, req, pos, indptr, indices, kv, q_weight=q[0, 0, :8]), lambda: app(None, None, None, None, req, pos, None, None, None),
        lambda: app(None, k, k, None, req, pos, indptr, indices, kv, q_weight=q[0, 0]), lambda: app(q, k, k, None, req, pos, indptr, indices, kv[:1].expand(9, -1, -1, -1, -1)),
        lambda: bnd(kv, bounds.half(), *where, last), lambda: bnd(kv, bounds, *where, last[:1]), lambda: bnd(kv, bounds[:1].expand(s["pages"], -1, -1, -1), *where, last),
        lambda: tab(lens, bt[:1], ps, 9), lambda: tab(lens, bt, ps, 9, new_lens=lens), lambda: tab(lens, bt, ps, 9, free_pages=lens),
        lambda: tab(lens, bt, ps, 9, out=bskv.PageTable(table.kv_indptr, table.kv_indices[:5], table.kv_last_page_len, table.qo_indptr, table.batch_indices, table.positions)),
        lambda: tab(lens, bt, ps, 9, free_pages=lens, free_count=lens[:1], out=table), lambda: tab(lens, bt, ps, 9, max_tokens=-1),
        lambda: bskv.PageTable(table.kv_indptr, table.kv_indices, table.kv_last_page_len, table.kv_indptr[:1], table.batch_indices, table.positions),
    ]:
        with pytest.raises(ValueError):
            call()
    for call in [lambda: att(p, q, kv, None, *where), lambda: tab(lens, bt, ps, 9, out=(1, 2)), lambda: sel(p, None, bounds, *where)]:
        with pytest.raises(TypeError):
            call()
    with pytest.raises(AttributeError):
        table.positions = pos
    with pytest.raises(bskv.BskvError, match="multiple of 16"):
        app(q, k, k, torch.zeros(9, 24, device=cuda), req, pos, indptr, indices, kv)
    with pytest.raises(bskv.BskvError, match="aligned"):
        sel(p, torch.zeros(2 * hq * d + 8, dtype=BF, device=cuda)[4:-4].view(2, hq, d), bounds, *where)
    assert bskv.bskv_get_device_status() == 0
