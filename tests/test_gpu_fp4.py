"""The 4-bit paged cache on the GPU: quantised append, reading back, and decode over it.

Quantisation and reading back are exact operations (one defined rounding), so they are compared
bit for bit. Decode gate, from the arithmetic: codes, scales and products are exact, sums are
fp32; each softmax weight times scale is rounded once to f16 (half a step, 2^-11 relative) and the
output once to its type (half a step: 2^-8 of the value in bf16, 2^-11 in fp16). With
A = sum_j w_j |v_j| that is |error| <= 2^-11 A + half |o|, plus fp32 sums and ex2 of a few 2^-22
(covered by 2^-12 A). A product of weight and scale below 2^-14 is an f16 subnormal, off by up to
2^-25; the kernel keeps the largest one M of a head at 2^10 or more, so each of the L
products is off by 2^-35 M at most and its value's code is at most 6: + 6 L 2^-35 M (it matters
where the tokens of large weight hold the code 0). The lse carries the fp32 rounding of logits of its size: 2^-18 (1 + |lse|).
"""

import numpy as np
import pytest
import torch

import block_sparse_kv_gb300 as bskv
import synth
from oracle import cache as oc
from oracle.numerics import bits_to_f64
from gpu_util import bits, to64

pytestmark = pytest.mark.gpu
DT = {torch.bfloat16: "bf16", torch.float16: "fp16"}


def _f64(t):
    return bits_to_f64(bits(t), DT[t.dtype])


def _cache(seed, d, device, lo=120, hi=130):
    """Random codes and scales for the page table of `d`; pages and slots that hold no token get
    NaN scales, so a read of one shows."""
    g = torch.Generator().manual_seed(seed)
    P, H, ps, D = d["num_pages"], d["num_kv_heads"], d["page_size"], d["head_dim"]
    codes = torch.randint(0, 256, (P, 2, H, ps, D // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(lo, hi, (P, 2, H, ps, D // 32), generator=g, dtype=torch.uint8)
    used = torch.zeros(P, ps, dtype=torch.bool)
    for b in range(d["batch"]):
        for i in range(int(d["kv_lens"][b])):
            used[int(d["kv_indices"][int(d["kv_indptr"][b]) + i // ps]), i % ps] = True
    scales[~used[:, None, None, :].expand(P, 2, H, ps)] = 255
    return codes.to(device), scales.to(device)


def _reference(d, codes, scales):
    """(out, lse, tolerance of out without its own rounding) in float64."""
    q = _f64(d["q"])
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    cache = oc.fp4_decode(codes, scales)
    a = (d["kv_indptr"].numpy(), d["kv_indices"].numpy(), d["kv_last_page_len"].numpy(), d["page_size"],
         d["sm_scale"])
    ref, ref_lse = oc.paged_decode(q, cache, *a)
    size, _ = oc.paged_decode(q, np.concatenate([cache[:, :1], np.abs(cache[:, 1:])], 1), *a)
    # values of code 6 everywhere: the largest weighted sum of a head is at least 6 M
    six, _ = oc.paged_decode(q, np.concatenate(
        [cache[:, :1], oc.fp4_decode(np.full_like(codes[:, 1:], 0x77), scales[:, 1:])], 1), *a)
    n = d["kv_lens"].numpy()[:, None, None].astype(np.float64)
    return ref, ref_lse, (2.0 ** -11 + 2.0 ** -12) * size + n * 2.0 ** -35 * six.max(-1, keepdims=True)


def _check_decode(d, dtype, codes, scales, out, lse):
    ref, ref_lse, tol = _reference(d, codes, scales)
    half = 2.0 ** (-8 if dtype == torch.bfloat16 else -11)
    tol = tol + half * np.abs(ref) + (2.0 ** -25 if dtype == torch.float16 else 1e-30)
    fits = np.abs(ref) < (6e4 if dtype == torch.float16 else 1e30)  # larger ones are infinite in fp16
    with np.errstate(invalid="ignore"):
        err = np.where(fits, np.abs(to64(out) - ref), 0.0)
    assert (err <= tol).all(), (err / tol).max()
    empty = np.isneginf(ref_lse)
    got = lse.cpu().double().numpy()
    assert (np.isneginf(got) == empty).all()
    err = np.abs(got[~empty] - ref_lse[~empty])
    assert (err <= 2.0 ** -18 * (1 + np.abs(ref_lse[~empty]))).all(), err.max()


# ---- quantisation -----------------------------------------------------------------------

def _table(lens, ps, seed, spare=3):
    g = torch.Generator().manual_seed(seed)
    n = [-(-x // ps) for x in lens]
    indptr = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32)
    pages = int(indptr[-1]) + spare
    return indptr, torch.randperm(pages, generator=g)[:int(indptr[-1])].to(torch.int32), pages


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,D,ps", [(8, 128, 16), (1, 64, 8), (3, 128, 48), (5, 64, 64)])
def test_append_codes_and_scales(cuda, dtype, H, D, ps):
    """Codes, scales and untouched bytes equal the definition's, over magnitudes from subnormal
    to the type's largest, exact ties, zeros of both signs, and blocks with NaN or infinity."""
    lens = [ps + 1, 1, 3 * ps, 0, 2 * ps - 1]
    indptr, indices, pages = _table(lens, ps, 5)
    rows = [(b, i) for b, n in enumerate(lens) for i in range(n)]
    g = torch.Generator().manual_seed(6)
    order = torch.randperm(len(rows), generator=g)[:len(rows) - 2]  # two tokens are not written
    rows = [rows[i] for i in order.tolist()]
    n = len(rows)
    top = 120 if dtype == torch.bfloat16 else 15
    k = torch.randn(n, H, D, generator=g) * 2.0 ** torch.randint(-top, top, (n, H, D // 32, 1), generator=g).expand(
        n, H, D // 32, 32).reshape(n, H, D)
    v = torch.randint(-24, 25, (n, H, D), generator=g) * 0.25  # exact ties at many scales
    k, v = k.to(dtype), v.to(dtype)
    k[0, 0, :32] = 0.0
    k[0, 0, 3] = -0.0
    v[1, 0, 5] = float("inf")
    v[2, 0, 40] = float("nan")
    k[3, 0, :32] = torch.finfo(dtype).max
    k[4, 0, :32] = torch.finfo(dtype).smallest_normal / 2 ** (torch.arange(32) % 7).float()
    codes = torch.full((pages, 2, H, ps, D // 2), 0xA5, dtype=torch.uint8, device=cuda)
    scales = torch.full((pages, 2, H, ps, D // 32), 0x5A, dtype=torch.uint8, device=cuda)
    want_c, want_s = codes.cpu().numpy(), scales.cpu().numpy()
    bi = torch.tensor([r[0] for r in rows], dtype=torch.int32)
    pos = torch.tensor([r[1] for r in rows], dtype=torch.int32)
    bskv.bskv_quantize_fp4_append_paged(k.to(cuda), v.to(cuda), bi.to(cuda), pos.to(cuda),
                                        indptr.to(cuda), indices.to(cuda), codes, scales)
    torch.cuda.synchronize()
    assert bskv.bskv_get_device_status() == 0
    nan = np.zeros(want_s.shape, dtype=bool)
    for which, x in ((0, k), (1, v)):
        nib, sc = oc.fp4_encode(_f64(x))
        for i, (b, t) in enumerate(rows):
            at = (int(indices[int(indptr[b]) + t // ps]), which, slice(None), t % ps)
            want_c[at] = nib[i, :, 0::2] | (nib[i, :, 1::2] << 4)
            want_s[at] = sc[i]
            nan[at] = sc[i] == 255
    assert (scales.cpu().numpy() == want_s).all()
    same = (codes.cpu().numpy() == want_c) | np.repeat(nan, 16, axis=-1)  # a NaN block's codes say nothing
    assert same.all()
    # and back: exact in bf16 and fp32, one rounding in fp16
    for back in (torch.bfloat16, torch.float32, torch.float16):
        ko, vo = bskv.bskv_dequantize_fp4_paged(codes, scales, bi.to(cuda), pos.to(cuda),
                                                indptr.to(cuda), indices.to(cuda), dtype=back)
        for which, x in ((0, ko), (1, vo)):
            ref = np.stack([oc.fp4_decode(want_c[int(indices[int(indptr[b]) + t // ps]), which, :, t % ps],
                                          want_s[int(indices[int(indptr[b]) + t // ps]), which, :, t % ps])
                            for b, t in rows])
            want = torch.from_numpy(ref).to(back)
            assert torch.equal(torch.nan_to_num(x.cpu(), 7e4, 8e4, -8e4), torch.nan_to_num(want, 7e4, 8e4, -8e4))


def test_append_out_of_range_rows(cuda):
    """Rows of an unknown request, a negative position, a position past the pages or a page
    outside the pool are not written and raise the device status; the others are."""
    indptr = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=cuda)
    indices = torch.tensor([1, 9, -1], dtype=torch.int32, device=cuda)  # pages 9 and -1 do not exist
    codes = torch.zeros((3, 2, 2, 16, 64), dtype=torch.uint8, device=cuda)
    scales = torch.zeros((3, 2, 2, 16, 4), dtype=torch.uint8, device=cuda)
    bi = torch.tensor([0, -1, 3, 0, 0, 1, 2], dtype=torch.int32, device=cuda)
    pos = torch.tensor([4, 0, 0, -1, 16, 0, 0], dtype=torch.int32, device=cuda)
    x = torch.full((7, 2, 128), 3.0, dtype=torch.bfloat16, device=cuda)
    bskv.bskv_quantize_fp4_append_paged(x, x, bi, pos, indptr, indices, codes, scales)
    torch.cuda.synchronize()
    assert bskv.bskv_get_device_status() == 6
    assert int((scales != 0).sum()) == 2 * 2 * 4 and bool((scales[1, :, :, 4] == 126).all())
    out = torch.full((7, 2, 128), -1.0, dtype=torch.float32, device=cuda)
    out2 = out.clone()
    bskv.bskv_dequantize_fp4_paged(codes, scales, bi, pos, indptr, indices, k_out=out, v_out=out2)
    torch.cuda.synchronize()
    assert bskv.bskv_get_device_status() == 6
    assert bool((out[0] == 3).all()) and bool((out[1:] == -1).all()) and torch.equal(out, out2)


def test_append_strided_rows_and_cache(cuda):
    """K / V as slices of one projection, codes in a token-major layout, scales in a larger pool."""
    H, D, ps, n = 4, 128, 16, 40
    indptr = torch.tensor([0, 3], dtype=torch.int32, device=cuda)
    indices = torch.tensor([2, 0, 1], dtype=torch.int32, device=cuda)
    qkv = torch.randn(n, 3 * H, D, dtype=torch.bfloat16, device=cuda)
    k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    codes = torch.zeros((3, 2, ps, H, D // 2), dtype=torch.uint8, device=cuda).transpose(2, 3)
    scales = torch.zeros((3, 2, 2 * H, ps, D // 32), dtype=torch.uint8, device=cuda)[:, :, ::2]
    bi = torch.zeros(n, dtype=torch.int32, device=cuda)
    pos = torch.arange(n, dtype=torch.int32, device=cuda)
    bskv.bskv_quantize_fp4_append_paged(k, v, bi, pos, indptr, indices, codes, scales)
    dense_c, dense_s = torch.zeros_like(codes.contiguous()), torch.zeros_like(scales.contiguous())
    bskv.bskv_quantize_fp4_append_paged(k.contiguous(), v.contiguous(), bi, pos, indptr, indices,
                                        dense_c, dense_s)
    assert torch.equal(codes.contiguous(), dense_c) and torch.equal(scales.contiguous(), dense_s)
    out = torch.zeros((n, 4 * H, D), dtype=torch.bfloat16, device=cuda)
    bskv.bskv_dequantize_fp4_paged(codes, scales, bi, pos, indptr, indices, k_out=out[:, H:2 * H],
                                   v_out=out[:, 3 * H:])
    a, b = bskv.bskv_dequantize_fp4_paged(dense_c, dense_s, bi, pos, indptr, indices)
    assert torch.equal(out[:, H:2 * H], a) and torch.equal(out[:, 3 * H:], b)
    assert bool((out[:, :H] == 0).all()) and bool((out[:, 2 * H:3 * H] == 0).all())


# ---- decode -----------------------------------------------------------------------------

CASES = [
    # batch, Hq, Hkv, D, page_size, len_lo, len_hi, dtype, max_workers
    (4, 8, 2, 128, 16, 1, 200, torch.bfloat16, 0),
    (4, 8, 2, 128, 16, 1, 200, torch.bfloat16, 7),
    (3, 32, 8, 128, 64, 100, 700, torch.bfloat16, 5),
    (5, 16, 1, 64, 16, 3, 300, torch.float16, 9),      # 16 query heads per kv head
    (6, 4, 4, 128, 8, 1, 90, torch.bfloat16, 4),       # 1
    (2, 12, 4, 64, 32, 33, 97, torch.float16, 3),      # 3
    (3, 36, 4, 128, 48, 20, 300, torch.float16, 6),    # 9, pages of 48
    (2, 16, 2, 128, 16, 900, 1000, torch.bfloat16, 20),  # many pieces
    (1, 8, 2, 128, 64, 5000, 5000, torch.bfloat16, 150),  # more than 64: merged by a kernel of their own
    (3, 10, 5, 128, 8, 1, 300, torch.float16, 0),      # 5 kv heads: 15 of 16 warps
    (2, 24, 12, 64, 32, 40, 200, torch.bfloat16, 5),   # 12 kv heads: two groups of 6
    (2, 22, 2, 128, 8, 30, 700, torch.bfloat16, 9),    # 11 query heads per kv head, pages of 8
    (1, 8, 8, 64, 8, 1, 1, torch.bfloat16, 0),         # one token
    (2, 13, 1, 64, 8, 600, 900, torch.bfloat16, 2),    # windows of 256 tokens turn over
]


@pytest.mark.parametrize("case", CASES)
def test_decode(cuda, case):
    B, Hq, Hkv, D, ps, lo, hi, dtype, mw = case
    d = synth.paged_decode_inputs(700 + B + Hq + ps, B, Hq, Hkv, D, ps, lo, hi, dtype=dtype)
    codes, scales = _cache(701, d, cuda)
    p = bskv.bskv_plan_decode_fp4(d["kv_indptr"], d["kv_indices"], d["kv_last_page_len"],
                                  d["num_pages"], ps, Hq, Hkv, D, dtype, max_workers=mw)
    out, lse = bskv.bskv_run_decode_fp4(p, d["q"].to(cuda), codes, scales, return_lse=True)
    again = bskv.bskv_run_decode_fp4(p, d["q"].to(cuda), codes, scales)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    _check_decode(d, dtype, codes, scales, out, lse)


def test_decode_empty_requests(cuda):
    d = synth.paged_decode_inputs(711, 5, 8, 2, 128, 16, 0, 0, lengths=[0, 37, 0, 1, 300])
    codes, scales = _cache(712, d, cuda)
    for mw in (0, 3):
        p = bskv.bskv_plan_decode_fp4(d["kv_indptr"], d["kv_indices"], d["kv_last_page_len"],
                                      d["num_pages"], 16, 8, 2, 128, torch.bfloat16, max_workers=mw)
        out, lse = bskv.bskv_run_decode_fp4(p, d["q"].to(cuda), codes, scales, return_lse=True)
        _check_decode(d, torch.bfloat16, codes, scales, out, lse)
    none = bskv.bskv_plan_decode_fp4(torch.zeros(4, dtype=torch.int32), [], torch.zeros(3), 0, 16, 8,
                                     2, 128)
    out, lse = bskv.bskv_run_decode_fp4(none, d["q"][:3].to(cuda), codes[:0], scales[:0], return_lse=True)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_decode_scales_of_any_magnitude(cuda, dtype):
    """Blocks of very different scale, growing and shrinking along the sequence and between the
    blocks of a row. The few tokens whose keys align with a query make the largest products of
    weight and scale small ones of the scales."""
    D, L = 128, 500
    d = synth.paged_decode_inputs(721, 2, 16, 2, D, 16, 0, 0, lengths=[L, 77], dtype=dtype)
    codes, scales = _cache(722, d, cuda, 121, 123)
    g = torch.Generator().manual_seed(723)
    s = scales.cpu()
    wild = torch.randint(60, 140, s[:, 1].shape, generator=g, dtype=torch.uint8)
    wild[..., 1] = torch.randint(20, 30, wild[..., 1].shape, generator=g, dtype=torch.uint8)
    wild[..., 2] = torch.randint(1, 3, wild[..., 2].shape, generator=g, dtype=torch.uint8) + 118
    first = int(d["kv_indices"][0])
    wild[first, :, 0, :] = 150  # the first token's values are the largest by far
    s[:, 1] = torch.where(s[:, 1] == 255, s[:, 1], wild)
    scales = s.to(cuda)
    for sharp in (1.0, 16.0):
        d["q"] = (d["q"].float() * sharp).to(dtype)
        p = bskv.bskv_plan_decode_fp4(d["kv_indptr"], d["kv_indices"], d["kv_last_page_len"],
                                      d["num_pages"], 16, 16, 2, D, dtype, max_workers=3)
        out, lse = bskv.bskv_run_decode_fp4(p, d["q"].to(cuda), codes, scales, return_lse=True)
        _check_decode(d, dtype, codes, scales, out, lse)


def test_decode_nan_scales(cuda):
    """A NaN key makes its head's outputs NaN, a NaN value block those 32 values of its head's."""
    d = synth.paged_decode_inputs(731, 2, 8, 2, 128, 16, 0, 0, lengths=[90, 40])
    codes, scales = _cache(732, d, cuda)
    page = int(d["kv_indices"][2])
    scales[page, 0, 0, 3, 1] = 255   # request 0, head 0: K of token 35
    scales[page, 1, 1, 4, 2] = 255   # request 0, head 1: V of token 36, values 64..95
    for mw in (1, 4):
        p = bskv.bskv_plan_decode_fp4(d["kv_indptr"], d["kv_indices"], d["kv_last_page_len"],
                                      d["num_pages"], 16, 8, 2, 128, torch.bfloat16, max_workers=mw)
        out, lse = bskv.bskv_run_decode_fp4(p, d["q"].to(cuda), codes, scales, return_lse=True)
        bad = torch.isnan(out)
        want = torch.zeros_like(bad)
        want[0, :4] = True
        want[0, 4:, 64:96] = True
        assert torch.equal(bad, want)
        assert torch.equal(torch.isnan(lse), want[:, :, 0])


@pytest.mark.parametrize("size", [1e-38, 1e-3, 300.0])
def test_decode_query_magnitudes(cuda, size):
    """bf16 queries from near the type's smallest to large: the f16 copies are exact."""
    d = synth.paged_decode_inputs(741, 3, 8, 2, 64, 16, 5, 100)
    d["q"] = (d["q"].float() * size).to(torch.bfloat16)
    d["q"][0, 0] = 0.0
    codes, scales = _cache(742, d, cuda, 118, 121)
    p = bskv.bskv_plan_decode_fp4(d["kv_indptr"], d["kv_indices"], d["kv_last_page_len"],
                                  d["num_pages"], 16, 8, 2, 64)
    out, lse = bskv.bskv_run_decode_fp4(p, d["q"].to(cuda), codes, scales, return_lse=True)
    _check_decode(d, torch.bfloat16, codes, scales, out, lse)


def test_decode_strides_and_scale(cuda):
    """q and out as slices, a token-major cache view, an explicit sm_scale."""
    d = synth.paged_decode_inputs(751, 3, 8, 2, 128, 16, 10, 100)
    d["sm_scale"] = 0.05
    codes, scales = _cache(752, d, cuda)
    tok = codes.transpose(2, 3).contiguous().transpose(2, 3)
    big = torch.zeros((3, 16, 128), dtype=torch.bfloat16, device=cuda)
    big[:, ::2] = d["q"].to(cuda)
    out = torch.full((3, 24, 128), -7.0, dtype=torch.bfloat16, device=cuda)
    lse = torch.empty((3, 8), device=cuda)
    p = bskv.bskv_plan_decode_fp4(d["kv_indptr"], d["kv_indices"], d["kv_last_page_len"],
                                  d["num_pages"], 16, 8, 2, 128, max_workers=4)
    bskv.bskv_run_decode_fp4(p, big[:, ::2], tok, scales, out=out[:, 1::3], lse=lse, sm_scale=0.05)
    _check_decode(d, torch.bfloat16, codes, scales, out[:, 1::3], lse)
    assert bool((out[:, 0::3] == -7).all()) and bool((out[:, 2::3] == -7).all())


@pytest.mark.parametrize("n, H, D", [(6001, 8, 128), (40003, 8, 128), (30011, 3, 64)])
def test_append_and_read_of_many_rows(cuda, n, H, D):
    """Spans of several passes per CTA give the bytes and values that short calls give."""
    ps, pages = 16, -(-n // 16)
    g = torch.Generator(device=cuda).manual_seed(61)
    indptr = torch.tensor([0, pages], dtype=torch.int32, device=cuda)
    indices = torch.randperm(pages, generator=g, device=cuda).to(torch.int32)
    k, v = (torch.randn(n, H, D, generator=g, device=cuda).to(torch.bfloat16) for _ in range(2))
    bi = torch.zeros(n, dtype=torch.int32, device=cuda)
    pos = torch.randperm(n, generator=g, device=cuda).to(torch.int32)
    got = []
    for step in (n, 777):
        codes = torch.zeros((pages, 2, H, ps, D // 2), dtype=torch.uint8, device=cuda)
        scales = torch.zeros((pages, 2, H, ps, D // 32), dtype=torch.uint8, device=cuda)
        rows = []
        for i in range(0, n, step):
            at = slice(i, i + step)
            bskv.bskv_quantize_fp4_append_paged(k[at], v[at], bi[at].clone(), pos[at].clone(), indptr, indices, codes,
                                                scales)
        for i in range(0, n, step):
            at = slice(i, i + step)
            rows.append(bskv.bskv_dequantize_fp4_paged(codes, scales, bi[at].clone(), pos[at].clone(), indptr, indices))
        got.append((codes, scales, torch.cat([r[0] for r in rows]), torch.cat([r[1] for r in rows])))
    torch.cuda.synchronize()
    assert bskv.bskv_get_device_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
