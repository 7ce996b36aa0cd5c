"""The operators of a bounded cache together, as a server runs them: append a prompt, then step by
step append, decode, add up the attention weights, and evict when a request reaches its bound. The
cache's contents after every eviction follow from the definitions exactly; outputs and scores are
within their operators' tolerances. Also the calls around them: graphs, streams, time-outs."""

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
from oracle import cache as oc
from gpu_util import to64
from test_gpu_graph import _graph_equal

pytestmark = pytest.mark.gpu
PS, H, G, D = 16, 2, 4, 128


def _table(lens, pages_per):
    """Page table of requests that own pages_per pages each, b * pages_per onwards."""
    n = [-(-x // PS) for x in lens]
    return (torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32),
            torch.tensor([b * pages_per + i for b, c in enumerate(n) for i in range(c)], dtype=torch.int32),
            torch.tensor([x - (c - 1) * PS if c else 0 for x, c in zip(lens, n)], dtype=torch.int32))


@pytest.mark.parametrize("four", [False, True])
def test_bounded_cache_serving_loop(cuda, four):
    torch.manual_seed(5)
    lens, bound, keep, sink, recent = [40, 57, 3], 64, 40, 4, 16
    B, per = len(lens), bound // PS
    pages = B * per
    gen = torch.Generator().manual_seed(6)
    codes = torch.zeros(pages, 2, H, PS, D // 2, dtype=torch.uint8, device=cuda)
    scales = torch.full((pages, 2, H, PS, D // 32), 255, dtype=torch.uint8, device=cuda)
    kv = torch.full((pages, 2, H, PS, D), float("nan"), dtype=torch.bfloat16, device=cuda)
    scores = torch.full((pages, H, PS), float("nan"), device=cuda)

    def append(lens, new):
        """The new tokens' K and V behind lens tokens: through the 4-bit append, or by indexing."""
        table = _table([a + b for a, b in zip(lens, new)], per)
        k, v = (torch.randn(sum(new), H, D, generator=gen).bfloat16().to(cuda) for _ in range(2))
        b = torch.tensor([i for i, n in enumerate(new) for _ in range(n)], dtype=torch.int32, device=cuda)
        pos = torch.tensor([a + i for a, n in zip(lens, new) for i in range(n)], dtype=torch.int32, device=cuda)
        if four:
            bskv.bskv_quantize_fp4_append_paged(k, v, b, pos, table[0].to(cuda), table[1].to(cuda), codes, scales)
        else:
            page = b.long() * per + pos.long() // PS
            kv[page, 0, :, pos.long() % PS], kv[page, 1, :, pos.long() % PS] = k, v

    def values():
        if four:
            return oc.fp4_decode(codes.cpu().numpy(), scales.cpu().numpy())
        return to64(kv)

    append([0] * B, lens)
    for step in range(30):
        append(lens, [1] * B)
        lens = [x + 1 for x in lens]
        table = _table(lens, per)
        q = torch.randn(B, H * G, D, generator=gen).bfloat16()
        if four:
            p = bskv.bskv_plan_decode_fp4(*table, pages, PS, H * G, H, D)
            out, lse = bskv.bskv_run_decode_fp4(p, q.to(cuda), codes, scales, return_lse=True)
        else:
            p = bskv.bskv_plan_decode(*table, pages, PS, H * G, H, D, torch.bfloat16)
            out, lse = bskv.bskv_run_decode(p, q.to(cuda), kv, return_lse=True)
        w = bskv.bskv_plan_attn_weights(None, *table, pages, PS, H * G, H, D)
        before = scores.cpu().double().numpy()
        decay = 0.875 if step else 0.0  # the prompt's scores start with the first step
        if four:
            bskv.bskv_run_attn_weights_fp4(w, q.to(cuda), codes, scales, lse, scores, decay=decay)
        else:
            bskv.bskv_run_attn_weights(w, q.to(cuda), kv, lse, scores, decay=decay)

        x = values()
        a = [t.numpy() for t in table]
        ref, ref_lse = oc.paged_decode(to64(q), x, *a, PS, D ** -0.5)
        size, _ = oc.paged_decode(to64(q), np.concatenate([x[:, :1], np.abs(x[:, 1:])], 1), *a, PS, D ** -0.5)
        # weights rounded to 16 bits (half a step of bf16 at worst) and the output's own rounding
        assert (np.abs(to64(out) - ref) <= 2.0 ** -8 * (size + np.abs(ref)) + 2.0 ** -12 * size).all()
        assert np.abs(lse.cpu().numpy() - ref_lse).max() <= 2.0 ** -17 * (1 + np.abs(ref_lse).max())
        want = oc.attn_weights(to64(q), x[:, 0], lse.cpu().double().numpy(), before, np.arange(B + 1), *a, PS,
                               D ** -0.5, True, decay)
        got = scores.cpu().double().numpy()
        used = ~np.isnan(want)
        assert (np.isnan(got) == ~used).all()
        # 2^-22 (A D / 16 + 2 |s| + 4) as the operator's own test derives, with scale |q| |k| and
        # exponents of at most 25 in size
        assert (np.abs(got - want)[used] <= 2.0 ** -14 * want[used] + 1e-30).all()

        if max(lens) == bound:
            target = [keep if n == bound else n for n in lens]
            e = bskv.bskv_plan_evict(*table, target, sink, recent, pages, PS, H, D)
            pools = [codes, scales] if four else [kv]
            old = [p.clone() for p in pools] + [scores.clone()]
            kept = (bskv.bskv_run_evict_fp4 if four else bskv.bskv_run_evict)(e, scores, *pools).cpu().tolist()
            for b in range(B):
                for h in range(H):
                    s = oc.request_rows(old[-1].cpu().numpy(), a[0], a[1], b, lens[b])[h]
                    stay = oc.evict_kept(s, lens[b], target[b], sink, recent)
                    at = e.info["kept_indptr"]
                    assert kept[h][at[b]:at[b + 1]] == stay
                    to, frm = np.arange(len(stay)), np.array(stay)
                    for o, n in zip(old[:-1], pools):
                        o, n = (t.view(torch.int16) if t.dtype == torch.bfloat16 else t for t in (o, n))
                        assert torch.equal(n[b * per + to // PS, :, h, to % PS], o[b * per + frm // PS, :, h, frm % PS])
                    assert torch.equal(scores[b * per + to // PS, h, to % PS], old[-1][b * per + frm // PS, h, frm % PS])
            lens = target
    assert bskv.bskv_get_device_status() == 0


# ---- graphs, streams, time-outs ---------------------------------------------------------

def _case(cuda, lens=(700, 129, 1, 40), four=True, hq=16, seed=0):
    g = torch.Generator().manual_seed(seed)
    per = -(-max(lens) // PS)
    pages = len(lens) * per
    s = dict(table=_table(list(lens), per), pages=pages,
             q=torch.randn(len(lens), hq, D, generator=g).bfloat16().to(cuda),
             codes=torch.randint(0, 256, (pages, 2, H, PS, D // 2), generator=g, dtype=torch.uint8).to(cuda),
             scales=torch.randint(120, 128, (pages, 2, H, PS, D // 32), generator=g, dtype=torch.uint8).to(cuda),
             kv=torch.randn(pages, 2, H, PS, D, generator=g).bfloat16().to(cuda),
             scores=torch.rand(pages, H, PS, generator=g).to(cuda))
    return s


def test_graphs_of_the_cache_operators(cuda):
    s = _case(cuda)
    p = bskv.bskv_plan_decode_fp4(*s["table"], s["pages"], PS, 16, H, D).upload(cuda)
    w = bskv.bskv_plan_attn_weights(None, *s["table"], s["pages"], PS, 16, H, D).upload(cuda)
    e = bskv.bskv_plan_evict(*s["table"], [300, 129, 1, 20], 2, 8, s["pages"], PS, H, D).upload(cuda)
    out, lse = torch.empty_like(s["q"]), torch.empty(4, 16, device=cuda)
    kept = torch.empty(H, 450, dtype=torch.int32, device=cuda)
    got = [torch.empty_like(s[n]) for n in ("scores", "codes", "scales")]
    rows = [torch.empty(3, H, D, dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    new = torch.randn(2, 3, H, D, device=cuda).bfloat16()
    at = [torch.tensor(x, dtype=torch.int32, device=cuda) for x in ([0, 1, 3], [5, 128, 39])]
    dev_table = [t.to(cuda) for t in s["table"][:2]]

    def run():
        for x, n in zip(got, ("scores", "codes", "scales")):
            x.copy_(s[n])
        bskv.bskv_quantize_fp4_append_paged(new[0], new[1], *at, *dev_table, got[1], got[2])
        bskv.bskv_dequantize_fp4_paged(got[1], got[2], *at, *dev_table, k_out=rows[0], v_out=rows[1])
        bskv.bskv_run_decode_fp4(p, s["q"], got[1], got[2], out=out, lse=lse)
        bskv.bskv_run_attn_weights_fp4(w, s["q"], got[1], got[2], lse, got[0])
        bskv.bskv_run_evict_fp4(e, got[0], got[1], got[2], kept=kept)

    _graph_equal(run, [out, lse, kept] + got + rows)


def test_graph_of_windows_and_halves(cuda):
    """The window form of the weights and the eviction of a 16-bit cache into other pages."""
    s = _case(cuda, lens=(300, 40))
    spare = torch.tensor([0, 9, 11], dtype=torch.int32), torch.arange(11, dtype=torch.int32) + s["pages"]
    kv = torch.cat([s["kv"], s["kv"][:11]])
    scores = torch.cat([s["scores"], s["scores"][:11]])
    q = torch.randn(70, 16, D, device=cuda).bfloat16()
    lse = torch.full((70, 16), 6.0, device=cuda)
    w = bskv.bskv_plan_attn_weights(torch.tensor([0, 50, 70], dtype=torch.int32), *s["table"], len(kv), PS, 16, H,
                                    D).upload(cuda)
    e = bskv.bskv_plan_evict(*s["table"], [140, 25], 0, 0, len(kv), PS, H, D, *spare).upload(cuda)
    got, pool = torch.empty_like(scores), torch.empty_like(kv)
    kept = torch.empty(H, 165, dtype=torch.int32, device=cuda)

    def run():
        got.copy_(scores)
        pool.copy_(kv)
        bskv.bskv_run_attn_weights(w, q, pool, lse, got, decay=0.5)
        bskv.bskv_run_evict(e, got, pool, kept=kept)

    _graph_equal(run, [got, pool, kept])


@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
def test_plans_are_not_uploaded_by_a_capture(cuda):
    """A graph must not copy the plan's host memory at every replay."""
    s = _case(cuda)
    p = bskv.bskv_plan_decode_fp4(*s["table"], s["pages"], PS, 16, H, D)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="upload"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            bskv.bskv_run_decode_fp4(p, s["q"], s["codes"], s["scales"])
    torch.cuda.synchronize()
    out = bskv.bskv_run_decode_fp4(p, s["q"], s["codes"], s["scales"])
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all()


def test_a_query_that_is_not_finite_stays_in_its_head(cuda):
    s = _case(cuda)
    p = bskv.bskv_plan_decode_fp4(*s["table"], s["pages"], PS, 16, H, D)
    w = bskv.bskv_plan_attn_weights(None, *s["table"], s["pages"], PS, 16, H, D)
    out, lse = bskv.bskv_run_decode_fp4(p, s["q"], s["codes"], s["scales"], return_lse=True)
    want = bskv.bskv_run_attn_weights_fp4(w, s["q"], s["codes"], s["scales"], lse, s["scores"].clone())
    for bad in (float("nan"), float("inf")):
        q = s["q"].clone()
        q[1, 3, 5] = bad  # of kv head 0
        got, z = bskv.bskv_run_decode_fp4(p, q, s["codes"], s["scales"], return_lse=True)
        assert torch.isnan(got[1, 3].float()).all()
        keep = torch.ones(4, 16, dtype=torch.bool, device=cuda)
        keep[1, 3] = False
        assert torch.equal(got[keep], out[keep]) and torch.equal(z[keep], lse[keep])
        sc = bskv.bskv_run_attn_weights_fp4(w, q, s["codes"], s["scales"], z, s["scores"].clone())
        assert torch.equal(sc[:, 1], want[:, 1])
        pages = s["table"][1][s["table"][0][1]:s["table"][0][2]].to(cuda).long()
        other = torch.ones(s["pages"], dtype=torch.bool, device=cuda)
        other[pages] = False
        assert torch.equal(sc[other], want[other])


def test_offsets_past_32_bits(cuda):
    """Pages 2 GiB apart, in bytes, in every pool that takes strides."""
    step, pages, lens = 2 ** 31 + 4096, 4, [30, 25]
    s = _case(cuda, lens=(30, 25))
    assert s["pages"] == pages

    def spread(x):
        n = step // x.element_size()
        far = torch.empty(n * (pages - 1) + x[0].numel(), dtype=x.dtype, device=cuda).as_strided(
            x.shape, (n,) + x[0].contiguous().stride())
        return far.copy_(x)

    far = {n: spread(s[n]) for n in ("codes", "scales", "kv", "scores")}
    t = (*s["table"], pages, PS, 16, H, D)
    p, w = bskv.bskv_plan_decode_fp4(*t), bskv.bskv_plan_attn_weights(None, *t)
    qo = torch.tensor([0, 20, 40], dtype=torch.int32)
    tile = bskv.bskv_plan_attn_weights(qo, *t)
    e = bskv.bskv_plan_evict(*s["table"], [17, 9], 1, 2, pages, PS, H, D)
    rows = torch.randn(2, 2, H, D, device=cuda).bfloat16()
    at = [torch.tensor(x, dtype=torch.int32, device=cuda) for x in ([0, 1], [29, 24])] + [x.to(cuda) for x in s["table"][:2]]
    qs = torch.randn(40, 16, D, device=cuda).bfloat16()
    zs = torch.full((40, 16), 5.0, device=cuda)
    got = []
    for x in (s, far):
        bskv.bskv_quantize_fp4_append_paged(rows[0], rows[1], *at, x["codes"], x["scales"])
        k, v = bskv.bskv_dequantize_fp4_paged(x["codes"], x["scales"], *at)
        out, lse = bskv.bskv_run_decode_fp4(p, s["q"], x["codes"], x["scales"], return_lse=True)
        bskv.bskv_run_attn_weights_fp4(w, s["q"], x["codes"], x["scales"], lse, x["scores"])
        bskv.bskv_run_attn_weights(w, s["q"], x["kv"], lse, x["scores"])
        bskv.bskv_run_attn_weights_fp4(tile, qs, x["codes"], x["scales"], zs, x["scores"])
        bskv.bskv_run_attn_weights(tile, qs, x["kv"], zs, x["scores"])
        a = bskv.bskv_run_evict_fp4(e, x["scores"], x["codes"], x["scales"], compact_scores=False)
        b = bskv.bskv_run_evict(e, x["scores"], x["kv"])
        got.append([k, v, out, lse, a, b] + [x[n].contiguous() for n in ("codes", "scales", "kv", "scores")])
    for u, v in zip(*got):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def test_calls_run_on_the_current_stream(cuda):
    """Two plans' runs on two streams at once give what each gives alone."""
    a, b = _case(cuda, seed=1), _case(cuda, lens=(1500, 2), seed=2)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def run(s, p, w):
        sc = s["scores"].clone()
        out, lse = bskv.bskv_run_decode_fp4(p, s["q"], s["codes"], s["scales"], return_lse=True)
        return out, lse, bskv.bskv_run_attn_weights_fp4(w, s["q"], s["codes"], s["scales"], lse, sc)

    plans = []
    for s in (a, b):
        t = (*s["table"], s["pages"], PS, 16, H, D)
        plans.append((bskv.bskv_plan_decode_fp4(*t).upload(cuda), bskv.bskv_plan_attn_weights(None, *t).upload(cuda)))
    alone = [run(s, *p) for s, p in zip((a, b), plans)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i] = run(s, *plans[i])
    torch.cuda.synchronize()
    for x, y in zip(alone, got):
        for u, v in zip(x, y):
            assert torch.equal(u, v)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("nq", [20, 90])
def test_weights_windows_report_a_wait_that_gives_up(cuda, four, nq):
    s = _case(cuda, lens=(300, 400))
    w = bskv.bskv_plan_attn_weights(torch.tensor([0, nq, 2 * nq], dtype=torch.int32), *s["table"], s["pages"], PS,
                                    16, H, D).upload(cuda)
    q, lse = torch.randn(2 * nq, 16, D, device=cuda).bfloat16(), torch.zeros(2 * nq, 16, device=cuda)

    def run(scores):
        if four:
            return bskv.bskv_run_attn_weights_fp4(w, q, s["codes"], s["scales"], lse, scores)
        return bskv.bskv_run_attn_weights(w, q, s["kv"], lse, scores)

    want = run(s["scores"].clone())
    torch.cuda.synchronize()
    assert bskv.bskv_get_device_status() == 0
    bskv.bskv_set_debug_force_timeout(True)
    try:
        run(s["scores"].clone())
        torch.cuda.synchronize()
        assert bskv.bskv_get_device_status() == 5
    finally:
        bskv.bskv_set_debug_force_timeout(False)
    assert torch.equal(run(s["scores"].clone()), want)
    torch.cuda.synchronize()
    assert bskv.bskv_get_device_status() == 0


def test_layouts_are_checked_again_when_they_change(cuda):
    """A call that passed its checks does not let another layout through."""
    s = _case(cuda)
    p = bskv.bskv_plan_decode_fp4(*s["table"], s["pages"], PS, 16, H, D)
    e = bskv.bskv_plan_evict(*s["table"], [300, 129, 1, 20], 2, 8, s["pages"], PS, H, D)
    out = torch.empty_like(s["q"])
    bskv.bskv_run_decode_fp4(p, s["q"], s["codes"], s["scales"], out=out)
    for q, c, x, o in ((s["q"][:3], s["codes"], s["scales"], None), (s["q"].half(), s["codes"], s["scales"], None),
                       (s["q"], s["codes"][:-1], s["scales"], None), (s["q"], s["codes"], s["scales"].float(), None),
                       (s["q"], s["codes"].transpose(3, 4).contiguous().transpose(3, 4), s["scales"], None),
                       (s["q"], s["codes"], s["scales"].transpose(2, 3).contiguous().transpose(2, 3), None),
                       (s["q"].cpu(), s["codes"], s["scales"], None), (s["q"], s["codes"].cpu(), s["scales"], None),
                       (s["q"], s["codes"], s["scales"], out[:, :1].expand_as(out)),
                       (s["q"], s["codes"], s["scales"], out.float())):
        with pytest.raises(ValueError):
            bskv.bskv_run_decode_fp4(p, q, c, x, out=o)
    for scores in (s["scores"].half(), s["scores"][:, :1].expand_as(s["scores"]), s["scores"][..., ::2], s["scores"].cpu()):
        with pytest.raises(ValueError):
            bskv.bskv_run_evict(e, scores, s["kv"])
    with pytest.raises(ValueError):
        bskv.bskv_run_evict(e, s["scores"], s["kv"][:, :, :1].expand_as(s["kv"]))
    with pytest.raises(ValueError):
        bskv.bskv_run_evict(e, s["scores"], s["kv"], kept=torch.empty(H, 1, dtype=torch.int32, device=cuda))
    with pytest.raises(bskv.BskvError):  # 8-byte aligned
        flat = torch.empty(s["scores"].numel() + 2, device=cuda)
        bskv.bskv_run_evict(e, flat[2:].view(s["scores"].shape), s["kv"])
    torch.cuda.synchronize()
    assert bskv.bskv_get_device_status() == 0


def test_weights_without_queries_fade(cuda):
    s = _case(cuda, lens=(40, 17))
    w = bskv.bskv_plan_attn_weights(torch.zeros(3, dtype=torch.int32), *s["table"], s["pages"], PS, 16, H, D)
    q, lse = torch.zeros(0, 16, D, dtype=torch.bfloat16, device=cuda), torch.zeros(0, 16, device=cuda)
    want = s["scores"].clone()
    for b, n in enumerate((40, 17)):
        for j in range(n):
            want[int(s["table"][1][int(s["table"][0][b]) + j // PS]), :, j % PS] *= 0.5
    for four in (True, False):
        got = s["scores"].clone()
        if four:
            bskv.bskv_run_attn_weights_fp4(w, q, s["codes"], s["scales"], lse, got, decay=0.5)
        else:
            bskv.bskv_run_attn_weights(w, q, s["kv"], lse, got, decay=0.5)
        assert torch.equal(got, want)


def test_runs_of_nothing(cuda):
    """Requests without tokens: outputs of zeros and -inf, nothing else touched."""
    lens = [0, 0]
    table = (torch.zeros(3, dtype=torch.int32), torch.zeros(0, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    s = _case(cuda, lens=(40, 40))
    n = s["pages"]
    out, lse = bskv.bskv_run_decode_fp4(bskv.bskv_plan_decode_fp4(*table, n, PS, 16, H, D), s["q"], s["codes"],
                                        s["scales"], return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    before = s["scores"].clone()
    for qo in (None, [0, 30, 60]):
        w = bskv.bskv_plan_attn_weights(None if qo is None else torch.tensor(qo, dtype=torch.int32), *table, n, PS,
                                        16, H, D)
        rows = 2 if qo is None else 60
        bskv.bskv_run_attn_weights(w, torch.zeros(rows, 16, D, device=cuda).bfloat16(), s["kv"],
                                   torch.zeros(rows, 16, device=cuda), s["scores"])
    e = bskv.bskv_plan_evict(*table, [5, 0], 2, 2, n, PS, H, D)
    assert bskv.bskv_run_evict(e, s["scores"], s["kv"]).shape == (H, 0)
    assert torch.equal(s["scores"], before)
    empty = torch.zeros(0, dtype=torch.int32, device=cuda)
    rows = torch.zeros(0, H, D, dtype=torch.bfloat16, device=cuda)
    bskv.bskv_quantize_fp4_append_paged(rows, rows, empty, empty, table[0].to(cuda), empty, s["codes"], s["scales"])
    k, _ = bskv.bskv_dequantize_fp4_paged(s["codes"], s["scales"], empty, empty, table[0].to(cuda), empty)
    assert k.shape == (0, H, D)
    torch.cuda.synchronize()
    assert bskv.bskv_get_device_status() == 0
