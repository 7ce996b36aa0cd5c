"""What the operators of a block-sparse decode step over a growing paged cache are measured on.

A serving step with long contexts goes through five operators, all of them driven by tensors on the
GPU, so that one captured step serves a batch whose requests grow: the page table and the token map
are made from the requests' lengths; queries and keys are normalised per head and rotated, and keys
and values appended to the paged cache; the channelwise bounds (least and greatest key value) of the
touched pages are brought up to date; each query chooses its best blocks (pages) by an upper bound of
its logits over them; attention runs over the chosen blocks alone. The cases here run these
operators in two forms that take the same inputs: with `own` false in elementary torch operations,
with `own` true through the package.

`op` of a case: "tables", "append", "bounds", "select", "attend", or "step" (all in order but the append,
whose rounding would decide between blocks that are nearly as good; its queries and rows are in place).
`queries` is the number of newest tokens of each request that are queries (1: plain decode, more:
drafted tokens that are verified together).
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of the paged decode benchmark's batch: a few requests need a new page
        dict(name="tables step", op="tables", batch=64, lo=512, hi=4096, queries=1, page=16),
        # a batch of prompts comes in whole: all its pages are handed out, a million tokens mapped
        dict(name="tables prompts", op="tables", batch=256, lo=512, hi=8192, queries=0, page=16),
        # the decode step's new tokens of the same batch, normalised queries and keys
        dict(name="append step", op="append", batch=64, lo=512, hi=4096, queries=1, page=16, hq=32,
             hkv=8, d=128, rot=128, neox=True, norm=True, dtype="bf16"),
        # short ragged prompts of a model with interleaved rotation of half of each head, no norms
        dict(name="append ragged d64", op="append", batch=37, lo=1, hi=999, queries=0, page=8, hq=24,
             hkv=4, d=64, rot=32, neox=False, norm=False, dtype="fp16"),
        # long prompts entering the cache
        dict(name="append prompts", op="append", batch=16, lo=1000, hi=3000, queries=0, page=16, hq=32,
             hkv=8, d=128, rot=128, neox=True, norm=True, dtype="bf16"),
        # after a decode step with large pages: one page of each request has changed
        dict(name="bounds step", op="bounds", batch=64, lo=512, hi=4096, queries=1, page=64, hkv=8,
             d=128, dtype="bf16"),
        # after those prompts: every page is new
        dict(name="bounds prompts", op="bounds", batch=16, lo=1000, hi=3000, queries=0, page=16, hkv=8,
             d=128, dtype="bf16"),
        # one long chat: 8192 blocks to choose from, latency counts
        dict(name="select one", op="select", batch=1, lo=131072, hi=131072, queries=1, page=16, hq=32,
             hkv=8, d=128, top=64, sink=1, recent=8, dtype="bf16"),
        # a batch of medium contexts
        dict(name="select batch", op="select", batch=64, lo=2048, hi=16384, queries=1, page=16, hq=32,
             hkv=8, d=128, top=64, sink=1, recent=8, dtype="bf16"),
        # the benchmark's batch, a quarter to all of each context attended to
        dict(name="attend batch", op="attend", batch=64, lo=1024, hi=4096, queries=1, page=16, hq=32,
             hkv=8, d=128, top=64, dtype="bf16"),
        # drafted tokens of short ragged requests, small pages and heads, six query heads to a kv head
        dict(name="attend drafts d64", op="attend", batch=37, lo=4, hi=999, queries=4, page=8, hq=24,
             hkv=4, d=64, top=32, dtype="fp16"),
        # the step of a long-context batch from the lengths to the output, eight query heads to a kv head
        dict(name="step long", op="step", batch=8, lo=16384, hi=16384, queries=1, page=64, hq=64, hkv=8,
             d=128, top=32, sink=1, recent=4, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tables", "append", "append", "bounds", "select", "select", "attend", "attend", "step"))
    page = rng.choice((8, 16, 16, 32, 48, 64))
    c = dict(op=op, page=page)
    if op == "tables":
        batch = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, (1 << 20) // batch)
        lo = rng.randint(max(1, hi // 8), hi)
        c.update(batch=batch, lo=lo, hi=hi, queries=rng.choice((0, 1, 1, rng.randint(1, min(8, lo)))))
        return c
    hkv = rng.choice((1, 2, 4, 8, 8))
    d = rng.choice((64, 128, 128))
    c.update(hkv=hkv, d=d, dtype=rng.choice(("bf16", "bf16", "fp16")))
    if op != "bounds":
        c.update(hq=hkv * rng.choice((1, 2, 3, 4, 4, 6, 8, 16)))
    if op == "append":
        c.update(rot=rng.choice((d, d, d // 2, 16)), neox=rng.random() < 0.6, norm=rng.random() < 0.7)
    if op in ("append", "bounds"):
        batch = _log_int(rng, 1, 128)
        # at most half of the long prompts' rows of heads
        rows = (1 << 15) * 24 // (c.get("hq", hkv) + 2 * hkv)
        hi = _log_int(rng, 1, max(1, min(8192, rows // batch)))
        lo = rng.randint(max(1, hi // 4), hi)
        c.update(batch=batch, lo=lo, hi=hi, queries=rng.choice((0, 1, rng.randint(1, lo))))
        return c
    batch = _log_int(rng, 1, 64)
    # at most 2^18 blocks of kv heads to choose from, and 2^20 cached tokens of kv heads
    most = (1 << 18) * page if op == "select" else (1 << 20)
    # where blocks are chosen, the longest requests have some to choose from
    least = 1 if op == "attend" else 32 * page
    hi = _log_int(rng, least, max(least, min(131072, most // (batch * hkv))))
    lo = rng.randint(max(1, hi // 8), hi)
    queries = rng.choice((1, 1, rng.randint(1, min(6, lo))))
    top = _log_int(rng, 3, 128)
    top = max(3, min(top, (1 << 18) // (page * batch * queries * hkv)))
    if op != "attend":
        top = min(top, (lo + hi) // 2 // page * 3 // 4)
    c.update(batch=batch, lo=lo, hi=hi, queries=queries, top=top)
    if op != "attend":
        sink = rng.randint(0, min(2, top - 2))
        c.update(sink=sink, recent=rng.randint(1, max(1, (top - sink) // 2)))
    return c


def _lens(case):
    """The requests' lengths: spread over [lo, hi], the same for every seed."""
    lo, hi = case["lo"], case["hi"]
    return [lo + int((hi - lo + 1) * ((0.5 + 0.6180339887 * i) % 1.0)) for i in range(case["batch"])]


def _new(case):
    """New tokens of each request: its last `queries`, all of them for 0."""
    return [min(n, case["queries"]) if case["queries"] else n for n in _lens(case)]


def _touched(case):
    """Pages that hold a new token."""
    page = case["page"]
    return sum(-(-n // page) - (n - m) // page for n, m in zip(_lens(case), _new(case)))


def _seen(case):
    """Blocks that each query sees, query by query."""
    return [[(n - m + i) // case["page"] + 1 for i in range(m)] for n, m in zip(_lens(case), _new(case))]


def work(case):
    op, page = case["op"], case["page"]
    new, pages = sum(_new(case)), sum(-(-n // page) for n in _lens(case))
    parts = {"tables": (16 * case["batch"] + 8 * pages + 16 * new, 8 * new)}
    if op != "tables":
        hkv, d = case["hkv"], case["d"]
        hq = case.get("hq", 0)
        if op == "append":
            parts["append"] = (new * ((hq + 2 * hkv) * d * 4 + case["rot"] * 4),
                               new * (hq + hkv) * (4 * d + 3 * case["rot"]))
        if op in ("bounds", "step"):
            rows = sum(n - (n - m) // page * page for n, m in zip(_lens(case), _new(case)))
            parts["bounds"] = ((rows + 2 * _touched(case)) * hkv * d * 2, 2 * rows * hkv * d)
        if op in ("select", "step"):
            n = sum(max([b for b in row if b > case["top"]], default=0) for row in _seen(case))
            every = sum(b for row in _seen(case) for b in row if b > case["top"])
            parts["select"] = (n * hkv * 4 * d + new * (hq * d * 2 + hkv * case["top"] * 4), every * hkv * 4 * d)
        if op in ("attend", "step"):
            chosen = [[min(b, case["top"]) for b in row] for row in _seen(case)]
            # what the queries of a request choose is theirs; no more than the whole request is read
            read = sum(min(sum(row), seen[-1]) for row, seen in zip(chosen, _seen(case)) if row)
            parts["attend"] = (read * page * hkv * 4 * d + new * hq * (4 * d + 4) + new * hkv * case["top"] * 4,
                               4 * d * page * hq * sum(sum(row) for row in chosen))
    use = parts.values() if op == "step" else [parts[op]]
    return {"bytes": sum(x[0] for x in use), "flops": sum(x[1] for x in use)}


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------

def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import block_sparse_kv_gb300 as bskv
        if "table" in s:
            s["own_table"] = bskv.PageTable(**s["table"])
        if "top" in case:
            c = case
            s["plan"] = bskv.bskv_plan_decode_blocks(
                s["q"].shape[0], s["max_pages"], s["pool"], c["page"], c["hq"], c["hkv"], c["d"], c["top"],
                sink=c.get("sink", 0), recent=c.get("recent", 1), dtype=DTYPES[c["dtype"]]).upload("cuda")
    return s


def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, page, batch = case["op"], case["page"], case["batch"]
    lens, new = _lens(case), _new(case)
    counts = [-(-n // page) for n in lens]
    before = [-(-(n - m) // page) for n, m in zip(lens, new)]
    most, pool, total = max(counts), sum(counts) + 8, sum(new)
    i32 = dict(dtype=torch.int32, device=dev)
    order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    at = torch.arange(most, device=dev)[None, :]
    held, has = torch.tensor(counts, device=dev)[:, None], torch.tensor(before, device=dev)[:, None]
    first = torch.cumsum(held, 0) - held
    s = dict(case=case, pool=pool, max_pages=most, total=total,
             lens=torch.tensor(lens, **i32), new=torch.tensor(new, **i32))
    # the token map, and the page table in compressed form
    b = torch.arange(batch, **i32).repeat_interleave(s["new"].long())
    start = torch.cumsum(s["new"], 0) - s["new"]
    pos = torch.arange(total, **i32) - start[b.long()].int() + (s["lens"] - s["new"])[b.long()]
    s.update(batch_indices=b, positions=pos,
             indptr=torch.cat([torch.zeros(1, **i32), torch.cumsum(held[:, 0], 0).to(torch.int32)]),
             indices=order[:sum(counts)].contiguous(),
             last=(s["lens"] - (held[:, 0] - 1).int() * page).contiguous())
    if op in ("tables", "step"):
        # the table that the server kept before the new tokens; pages of its free list come next
        pages = order[(first + at).clamp(max=pool - 1)]
        s["block_table"] = torch.where(at < has, pages, -1).to(torch.int32).contiguous()
        fresh = (at >= has) & (at < held)
        free = pages[fresh]  # in the order in which they will be handed out
        s["free_pages"] = torch.cat([order[sum(counts):], free.flip(0)]).contiguous()
        s["free_count"] = torch.tensor([s["free_pages"].numel()], **i32)
        rows = total + 3  # a fixed number of rows, some of them without a token
        s["table"] = dict(
            kv_indptr=torch.empty(batch + 1, **i32), kv_indices=torch.full((batch * most,), -1, **i32),
            kv_last_page_len=torch.empty(batch, **i32), qo_indptr=torch.empty(batch + 1, **i32),
            batch_indices=torch.empty(rows, **i32), positions=torch.empty(rows, **i32),
            slots=torch.empty(rows, dtype=torch.int64, device=dev), free_left=torch.empty(1, **i32))
        if op == "tables":
            return s
    else:
        rows = total
    hkv, d, dtype = case["hkv"], case["d"], DTYPES[case["dtype"]]
    hq = case.get("hq", hkv)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * scale).to(dtype)

    channel = torch.randn((hkv, 1, d), generator=gen, device=dev)  # keys share a part per channel
    if op != "select":
        s["kv"] = normal(pool, 2, hkv, page, d)
        s["kv"][:, 0] += channel.to(dtype)
    if op != "bounds":
        s["q"] = normal(rows, hq, d)
    if op == "append":
        s["k"], s["v"] = normal(rows, hkv, d, scale=2.0), normal(rows, hkv, d)
        s["q_out"] = torch.zeros_like(s["q"])
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device=dev)).to(dtype)
            s["k_weight"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device=dev)).to(dtype)
        # a table with positions stretched by four, as for contexts beyond the trained length
        half = case["rot"] // 2
        angle = (torch.arange(max(lens), dtype=torch.float64)[:, None] / 4.0
                 * 1e4 ** (-torch.arange(half, dtype=torch.float64)[None, :] / half))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().to(dev)
    if op in ("bounds", "select", "step"):
        s["bounds"] = _random_bounds(case, s, gen, channel, dtype)
    if op == "attend":
        s["blocks"] = _random_blocks(case, s, gen)
    if op in ("attend", "step"):
        s["out"] = torch.zeros((rows, hq, d), dtype=dtype, device=dev)
        s["lse"] = torch.zeros((rows, hq), device=dev)
    if op in ("select", "step"):
        s["chosen"] = torch.full((rows, hkv, case["top"]), -2, **i32)
    return s


def _random_bounds(case, s, gen, channel, dtype):
    """Bounds of every page as normal keys give them: for a step those of its cache, else drawn."""
    dev = channel.device
    if "kv" in s:
        k = s["kv"][:, 0]
        return torch.stack([k.amin(2), k.amax(2)], 2).contiguous()
    shape = (s["pool"], case["hkv"], case["d"])
    spread = math.sqrt(2.0 * math.log(case["page"]))
    lo = channel[:, 0] - spread * (0.75 + 0.5 * torch.rand(shape, generator=gen, device=dev))
    hi = channel[:, 0] + spread * (0.75 + 0.5 * torch.rand(shape, generator=gen, device=dev))
    return torch.stack([lo.to(dtype), hi.to(dtype)], 2).contiguous()


def _random_blocks(case, s, gen):
    """Per query and kv head `top` of the blocks it sees, its last one among them, in ascending order."""
    seen = s["positions"].long() // case["page"] + 1
    most = int(seen.max())
    at = torch.arange(most, device=seen.device)[None, None, :]
    key = torch.rand((seen.numel(), case["hkv"], most), generator=gen, device=seen.device)
    key = key.masked_fill(at == seen[:, None, None] - 1, 2.0).masked_fill(at >= seen[:, None, None], -1.0)
    top = min(case["top"], most)
    val, idx = key.topk(top, dim=-1)
    idx = torch.where(val >= 0, idx, most).sort(-1).values
    blocks = torch.full(key.shape[:2] + (case["top"],), -1, dtype=torch.int32, device=seen.device)
    blocks[..., :top] = torch.where(idx < most, idx, -1).to(torch.int32)
    return blocks


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    parts = dict(tables=_own_tables, append=_own_append, bounds=_own_bounds, select=_own_select,
                 attend=_own_attend) if own else dict(tables=_tables, append=_append, bounds=_bounds,
                                                      select=_select, attend=_attend)
    if op != "step":
        return parts[op](s, _given(s))
    t = parts["tables"](s, None)
    got = dict(parts["bounds"](s, t), **parts["select"](s, t))
    s["blocks"] = got["blocks"]
    return dict(t, **got, **parts["attend"](s, t))


def _given(s):
    return dict(kv_indptr=s["indptr"], kv_indices=s["indices"], kv_last_page_len=s["last"],
                batch_indices=s["batch_indices"], positions=s["positions"])


def _own_tables(s, _):
    import block_sparse_kv_gb300 as bskv
    bskv.bskv_build_page_table(s["lens"], s["block_table"], s["case"]["page"], s["pool"], new_lens=s["new"],
                               free_pages=s["free_pages"], free_count=s["free_count"], out=s["own_table"])
    return dict(s["table"], block_table=s["block_table"])


def _own_append(s, t):
    import block_sparse_kv_gb300 as bskv
    q = bskv.bskv_norm_rope_append_paged(
        s["q"], s["k"], s["v"], s["cos_sin"], t["batch_indices"], t["positions"], t["kv_indptr"], t["kv_indices"],
        s["kv"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, is_neox=s["case"]["neox"], q_out=s["q_out"])
    return {"q": q, "kv": s["kv"]}


def _own_bounds(s, t):
    import block_sparse_kv_gb300 as bskv
    return {"bounds": bskv.bskv_block_bounds_paged(s["kv"], s["bounds"], t["batch_indices"], t["positions"],
                                                   t["kv_indptr"], t["kv_indices"], t["kv_last_page_len"])}


def _own_select(s, t):
    import block_sparse_kv_gb300 as bskv
    return {"blocks": bskv.bskv_run_select_blocks(s["plan"], s["q"], s["bounds"], t["batch_indices"], t["positions"],
                                                  t["kv_indptr"], t["kv_indices"], blocks=s["chosen"])}


def _own_attend(s, t):
    import block_sparse_kv_gb300 as bskv
    out, lse = bskv.bskv_run_decode_blocks(s["plan"], s["q"], s["kv"], s["blocks"], t["batch_indices"], t["positions"],
                                           t["kv_indptr"], t["kv_indices"], out=s["out"], lse=s["lse"], return_lse=True)
    return {"out": out, "lse": lse}


# ---- the plain forms ------------------------------------------------------------------

def _tables(s, _):
    page, dev, t = s["case"]["page"], s["lens"].device, s["table"]
    lens, new, batch = s["lens"].long(), s["new"].long(), s["lens"].numel()
    pages, before = (lens + page - 1) // page, (lens - new + page - 1) // page
    at = torch.arange(s["max_pages"], device=dev)[None, :]
    # new pages come from the end of the free list, request by request
    taken = torch.cumsum(pages - before, 0) - (pages - before)
    nth = taken[:, None] + at - before[:, None]
    fresh = (at >= before[:, None]) & (at < pages[:, None])
    handed = s["free_pages"][(s["free_count"].long() - 1 - nth).clamp(min=0, max=s["free_pages"].numel() - 1)]
    s["block_table"].copy_(torch.where(fresh, handed, s["block_table"]))
    t["free_left"].copy_(s["free_count"] - (pages - before).sum())
    t["kv_indptr"][0] = 0
    t["kv_indptr"][1:] = torch.cumsum(pages, 0)
    t["qo_indptr"][0] = 0
    t["qo_indptr"][1:] = torch.cumsum(new, 0)
    listed_pages = s["block_table"][at < pages[:, None]]
    t["kv_indices"][:listed_pages.numel()] = listed_pages
    t["kv_last_page_len"].copy_(torch.where(pages > 0, lens - (pages - 1) * page, 0))
    b = torch.arange(batch, device=dev).repeat_interleave(new)
    n = b.numel()
    pos = torch.arange(n, device=dev) - t["qo_indptr"].long()[b] + (lens - new)[b]
    for name, x in (("batch_indices", b), ("positions", pos),
                    ("slots", s["block_table"][b, pos // page].long() * page + pos % page)):
        t[name][:n] = x.to(t[name].dtype)
        t[name][n:] = -1
    return dict(t, block_table=s["block_table"])


def _live(t):
    """The rows that hold a token, their request and position."""
    rows = (t["batch_indices"] >= 0).nonzero()[:, 0]
    return rows, t["batch_indices"].long()[rows], t["positions"].long()[rows]


def _page_of(t, b, block):
    return t["kv_indices"].long()[t["kv_indptr"].long()[b] + block]


def _rotated(x, weight, cos_sin, pos, rot, neox):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    half = rot // 2
    cos, sin = cos_sin[pos, None, :half], cos_sin[pos, None, half:]
    y = x.clone()
    one, two = (slice(0, half), slice(half, rot)) if neox else (slice(0, rot, 2), slice(1, rot, 2))
    y[..., one] = x[..., one] * cos - x[..., two] * sin
    y[..., two] = x[..., two] * cos + x[..., one] * sin
    return y


def _append(s, t):
    c = s["case"]
    rows, b, pos = _live(t)
    dtype = s["q"].dtype
    s["q_out"][rows] = _rotated(s["q"][rows], s["q_weight"], s["cos_sin"], pos, c["rot"], c["neox"]).to(dtype)
    k = _rotated(s["k"][rows], s["k_weight"], s["cos_sin"], pos, c["rot"], c["neox"]).to(dtype)
    page = _page_of(t, b, pos // c["page"])
    s["kv"][page, 0, :, pos % c["page"]] = k
    s["kv"][page, 1, :, pos % c["page"]] = s["v"][rows]
    return {"q": s["q_out"], "kv": s["kv"]}


def _bounds(s, t):
    c = s["case"]
    _, b, pos = _live(t)
    block = pos // c["page"]
    page = _page_of(t, b, block)
    count = (t["kv_indptr"][1:] - t["kv_indptr"][:-1]).long()[b]
    fill = torch.where(block == count - 1, t["kv_last_page_len"].long()[b], c["page"])
    first = torch.ones_like(page, dtype=torch.bool)  # rows of a page come one after another
    first[1:] = page[1:] != page[:-1]
    page, fill = page[first], fill[first]
    there = (torch.arange(c["page"], device=page.device)[None, :] < fill[:, None])[:, None, :, None]
    k = s["kv"][page, 0].float()
    s["bounds"][page, :, 0] = k.masked_fill(~there, math.inf).amin(2).to(s["bounds"].dtype)
    s["bounds"][page, :, 1] = k.masked_fill(~there, -math.inf).amax(2).to(s["bounds"].dtype)
    return {"bounds": s["bounds"]}


def _select(s, t):
    c = s["case"]
    rows, b, pos = _live(t)
    top = c["top"]
    seen = pos // c["page"] + 1
    most = max(s["max_pages"], top)
    at = torch.arange(most, device=pos.device)[None, :]
    page = _page_of(t, b[:, None], torch.where(at < seen[:, None], at, 0))
    q = s["q"][rows].double().unflatten(1, (c["hkv"], -1))
    plus, minus = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)  # over the heads of a group
    x = s["bounds"][page].double()  # [rows, blocks, kv heads, 2, dims]
    score = torch.einsum("rnhd,rhd->rhn", x[..., 1, :], plus) + torch.einsum("rnhd,rhd->rhn", x[..., 0, :], minus)
    n = seen[:, None, None]
    at = at[None]
    score = score.masked_fill((at < c["sink"]) | (at >= n - c["recent"]), math.inf).masked_fill(at >= n, -math.inf)
    order = score.argsort(dim=-1, descending=True, stable=True)[..., :top]
    order = torch.where(order < n, order, most).sort(-1).values
    s["chosen"][rows] = torch.where(order < most, order, -1).to(torch.int32)
    return {"blocks": s["chosen"]}


def _attend(s, t):
    c = s["case"]
    page, hkv, d = c["page"], c["hkv"], c["d"]
    rows, b, pos = _live(t)
    block = s["blocks"][rows].long()  # [rows, kv heads, top]
    there = block >= 0
    pg = _page_of(t, b[:, None, None], block.clamp(min=0))
    h = torch.arange(hkv, device=pos.device)[None, :, None]
    at = block[..., None] * page + torch.arange(page, device=pos.device)
    seen = (there[..., None] & (at <= pos[:, None, None, None])).flatten(2)  # [rows, kv heads, tokens]
    q = s["q"][rows].float().unflatten(1, (hkv, -1))
    x = torch.einsum("rhgd,rhnd->rhgn", q, s["kv"][pg, 0, h].flatten(2, 3).float()) / math.sqrt(d)
    x = x.masked_fill(~seen[:, :, None, :], -math.inf)
    best = x.amax(-1, keepdim=True)
    e = (x - best).exp()
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("rhgn,rhnd->rhgd", e / total, s["kv"][pg, 1, h].flatten(2, 3).float())
    s["out"][rows] = o.flatten(1, 2).to(s["out"].dtype)
    s["lse"][rows] = (best + total.log()).flatten(1)
    return {"out": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------------------------
# from the definitions, in 64 bits, request by request
# --------------------------------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "tables":
        return None  # whole numbers
    page, d, hkv = case["page"], case["d"], case["hkv"]
    lens, new = _lens(case), _new(case)
    dev = s["lens"].device
    pages = [s["indices"][int(i):int(j)].long() for i, j in zip(s["indptr"][:-1], s["indptr"][1:])]
    rows, at = [], 0
    for m in new:
        rows.append(slice(at, at + m))
        at += m
    if op == "append":
        kv, half = s["kv"].double(), case["rot"] // 2
        turn = torch.complex(s["cos_sin"][:, :half].double(), s["cos_sin"][:, half:].double())

        def rotate(x, w, pos):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS) * w.double()
            r = x[..., :case["rot"]]
            pairs = r.unflatten(-1, (2, half)).transpose(-1, -2) if case["neox"] else r.unflatten(-1, (half, 2))
            z = torch.view_as_complex(pairs.contiguous()) * turn[pos][:, None, :]
            r = torch.view_as_real(z)
            r = (r.transpose(-1, -2) if case["neox"] else r).flatten(-2)
            return torch.cat([r, x[..., case["rot"]:]], -1)

        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
        for b, (n, m) in enumerate(zip(lens, new)):
            pos = torch.arange(n - m, n, device=dev)
            out[rows[b]] = rotate(s["q"][rows[b]], s["q_weight"], pos)
            kv[pages[b][pos // page], 0, :, pos % page] = rotate(s["k"][rows[b]], s["k_weight"], pos)
            kv[pages[b][pos // page], 1, :, pos % page] = s["v"][rows[b]].double()
        return {"q": out, "kv": kv}
    got = {}
    if op == "step":  # the table and the token map are whole numbers
        got = dict.fromkeys(list(s["table"]) + ["block_table"])
    if op in ("bounds", "step"):
        lo_hi = s["bounds"].double()
        for b, (n, m) in enumerate(zip(lens, new)):
            for j in range((n - m) // page, -(-n // page)):
                k = s["kv"][pages[b][j], 0, :, :min(page, n - j * page)].double()
                lo_hi[pages[b][j], :, 0], lo_hi[pages[b][j], :, 1] = k.min(1).values, k.max(1).values
        got["bounds"] = lo_hi
        if op == "bounds":
            return got
        s["bounds"].copy_(lo_hi)
    q = s["q"].double()
    if op in ("select", "step"):
        blocks = s["chosen"].clone()
        for b, (n, m) in enumerate(zip(lens, new)):
            x = s["bounds"][pages[b]].double()
            for i in range(m):
                seen = (n - m + i) // page + 1
                each = q[rows[b]][i].view(hkv, -1, d)
                for h in range(hkv):
                    # a block's greatest possible logit of each head, summed over the heads
                    bound = torch.maximum(each[h][:, None, :] * x[None, :seen, h, 0],
                                          each[h][:, None, :] * x[None, :seen, h, 1]).sum(-1).sum(0)
                    bound[:case["sink"]] = math.inf
                    bound[max(0, seen - case["recent"]):] = math.inf
                    best = bound.argsort(descending=True, stable=True)[:case["top"]].sort().values
                    blocks[rows[b].start + i, h] = -1
                    blocks[rows[b].start + i, h, :best.numel()] = best.to(torch.int32)
        got["blocks"] = s["blocks"] = blocks
        if op == "select":
            return got
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=dev)
    group = case["hq"] // hkv
    chosen = s["blocks"].cpu()
    for b, (n, m) in enumerate(zip(lens, new)):
        k, v = s["kv"][pages[b], 0].double(), s["kv"][pages[b], 1].double()
        for i in range(m):
            r, p = rows[b].start + i, n - m + i
            for h in range(hkv):
                at = [j for j in chosen[r, h].tolist() if j >= 0]
                slots = torch.cat([torch.arange(j * page, min(p + 1, (j + 1) * page)) for j in at]).to(dev)
                kk, vv = k[slots // page, h, slots % page], v[slots // page, h, slots % page]
                x = q[r, h * group:(h + 1) * group] @ kk.T * d ** -0.5
                z = torch.logsumexp(x, -1)
                out[r, h * group:(h + 1) * group] = torch.exp(x - z[:, None]) @ vv
                lse[r, h * group:(h + 1) * group] = z
    return {"out": out, "lse": lse}
