"""The 4-bit paged cache, token scores and eviction, as plain definitions in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Format: OCP Microscaling Formats (MX) specification, MXFP4: E2M1 elements and one E8M0 scale
2^(code - 127) (255 = NaN) per block of 32; conversion by shared exponent floor(log2 max) - 2,
elements rounded to nearest even and clamped to the largest magnitude 6.
"""

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def fp4_decode(codes, scales):
    """codes uint8 [..., D / 2] (low nibble first), scales uint8 [..., D / 32] -> float64 [..., D]."""
    c = np.asarray(codes, dtype=np.uint8)
    nib = np.stack([c & 15, c >> 4], -1).reshape(c.shape[:-1] + (-1,)).astype(np.int64)
    val = np.where(nib & 8, -1.0, 1.0) * E2M1[nib & 7]
    s = np.asarray(scales, dtype=np.uint8).astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return val * np.repeat(f, 32, axis=-1)


def fp4_encode(x):
    """float64 [..., D] -> (E2M1 nibbles [..., D], scale codes [..., D / 32]); blocks with an
    infinity or a NaN get code 255 (nibbles 0)."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(b).all(-1)
    top = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1))
    _, e = np.frexp(top)  # top = m * 2^e with m in [0.5, 1): floor(log2) = e - 1
    code = np.where(top > 0, np.clip(e - 1 - 2 + 127, 0, 254), 0)
    y = np.where(bad[..., None], 0.0, b) / np.ldexp(1.0, code - 127)[..., None]
    a = np.minimum(np.abs(y), 6.0)
    # nearest of the eight magnitudes; between two equally near, the one with an even code
    dist = np.abs(a[..., None] - E2M1)
    near = dist == dist.min(-1, keepdims=True)
    pick = np.where(near, np.arange(8) + 8 * (np.arange(8) & 1), 99).argmin(-1)
    nib = pick + 8 * (np.signbit(y))
    return nib.reshape(x.shape).astype(np.uint8), np.where(bad, 255, code).astype(np.uint8)


def lengths(kv_indptr, kv_last, page_size):
    n = np.diff(np.asarray(kv_indptr))
    return np.where(n > 0, (n - 1) * page_size + np.asarray(kv_last), 0)


def request_rows(pool, kv_indptr, kv_indices, b, length):
    """pool [pages, heads, page_size, ...] -> [heads, length, ...] of request b."""
    pages = np.asarray(kv_indices)[kv_indptr[b]:kv_indptr[b + 1]]
    x = np.moveaxis(pool[pages], 1, 0)
    return x.reshape((x.shape[0], -1) + x.shape[3:])[:, :length]


def paged_decode(q, cache, kv_indptr, kv_indices, kv_last, page_size, sm_scale):
    """q [B, Hq, D] and cache [pages, 2, Hkv, page_size, D] in float64 -> (out, lse)."""
    B, Hq, D = q.shape
    Hkv = cache.shape[2]
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    for b, L in enumerate(lengths(kv_indptr, kv_last, page_size)):
        if L == 0:
            continue
        k = request_rows(cache[:, 0], kv_indptr, kv_indices, b, L)
        v = request_rows(cache[:, 1], kv_indptr, kv_indices, b, L)
        for h in range(Hq):
            s = sm_scale * (k[h // (Hq // Hkv)] @ q[b, h])
            m = s.max()
            e = np.exp(s - m)
            out[b, h] = (e / e.sum()) @ v[h // (Hq // Hkv)]
            lse[b, h] = m + np.log(e.sum())
    return out, lse


def attn_weights(q, keys, lse, scores, qo_indptr, kv_indptr, kv_indices, kv_last, page_size,
                 sm_scale, causal, decay):
    """scores after one accumulation: q [Tq, Hq, D], keys [pages, Hkv, page_size, D], lse
    [Tq, Hq], scores [pages, Hkv, page_size] in float64."""
    out = np.array(scores, dtype=np.float64)
    Hq, Hkv = q.shape[1], keys.shape[1]
    g = Hq // Hkv
    for b, L in enumerate(lengths(kv_indptr, kv_last, page_size)):
        L = int(L)
        nq = int(qo_indptr[b + 1] - qo_indptr[b])
        k = request_rows(keys, kv_indptr, kv_indices, b, L)
        see = np.ones((L, nq), dtype=bool)
        if causal:
            see = np.arange(L)[:, None] <= np.arange(nq)[None, :] + L - nq
        rows = slice(int(qo_indptr[b]), int(qo_indptr[b]) + nq)
        fresh = (decay == 0) | (np.arange(L) >= L - nq)
        pages = np.asarray(kv_indices)[kv_indptr[b] + np.arange(L) // page_size]
        for h in range(Hkv):
            w = np.zeros(L)
            for r in range(h * g, (h + 1) * g):
                z = lse[rows, r][None, :]
                live = see & ~np.isneginf(z)
                with np.errstate(invalid="ignore", over="ignore"):
                    e = np.exp(sm_scale * (k[h] @ q[rows, r].T) - z)
                w += np.where(live, e, 0.0).sum(1)
            slots = (pages, h, np.arange(L) % page_size)
            with np.errstate(invalid="ignore"):
                out[slots] = np.where(fresh, w, decay * out[slots] + w)
    return out


def evict_kept(score, length, keep, sink, recent):
    """Old slots of the kept tokens of one request and head, in order (score [length])."""
    if length <= keep:
        return list(range(length))
    sure = [j for j in range(length) if j < sink or j >= length - recent]
    rest = [j for j in range(length) if sink <= j < length - recent]
    # highest score first (NaN above everything), the lowest slot among equals
    rest.sort(key=lambda j: (not np.isnan(score[j]), -score[j] if not np.isnan(score[j]) else 0.0, j))
    return sorted(sure + rest[:keep - len(sure)])
