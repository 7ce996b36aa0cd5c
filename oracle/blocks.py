"""The block-sparse decode step over a paged cache, as plain definitions in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Page tables and token maps from lengths, normalised and rotated rows, the bounds of a cache's
blocks, the choice of blocks by them, and attention over the chosen blocks; request by request and
head by head.
"""

import numpy as np


def page_table(lens, new, table, page_size, free=None):
    """table [B, max_pages] lists, changed in place where `free` (a list that is popped) gives pages ->
    (kv_indptr, kv_indices, kv_last_page_len, qo_indptr, batch_indices, positions, slots)."""
    indptr, indices, last, qo = [0], [], [], [0]
    req, pos, slots = [], [], []
    for b, (n, m) in enumerate(zip(lens, new)):
        pages = -(-n // page_size)
        if free is not None:
            for j in range(-(-(n - m) // page_size), pages):
                table[b][j] = free.pop()
        indices += [int(x) for x in table[b][:pages]]
        indptr.append(len(indices))
        last.append(n - (pages - 1) * page_size if pages else 0)
        for p in range(n - m, n):
            req.append(b)
            pos.append(p)
            slots.append(int(table[b][p // page_size]) * page_size + p % page_size)
        qo.append(len(req))
    return indptr, indices, last, qo, req, pos, slots


def norm_rope(x, weight, eps, cos_sin, rot, is_neox):
    """Rows x [heads, D] of one token at the table's row cos_sin [rot] -> (values, sizes), the sizes being what
    the values' terms add up to without their signs."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    y, size = x.copy(), np.abs(x)
    half = rot // 2
    for i in range(half):
        a, b = (i, i + half) if is_neox else (2 * i, 2 * i + 1)
        c, s = cos_sin[i], cos_sin[half + i]
        y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
        size[:, a] = np.abs(x[:, a] * c) + np.abs(x[:, b] * s)
        size[:, b] = np.abs(x[:, b] * c) + np.abs(x[:, a] * s)
    return y, size


def block_bounds(cache, page, fill):
    """Bounds [heads, 2, D] of the first `fill` slots of a page of cache [pages, 2, heads, page_size, D]."""
    k = cache[page, 0, :, :fill]
    return np.stack([k.min(1), k.max(1)], 1)


def block_scores(q, bounds):
    """q [group, D] and bounds [blocks, 2, D] -> scores [blocks]: each head's greatest possible logit, summed over the
    heads, term by term max(q lo, q hi) of bounds in order. Out of order the sign of q says which is meant; zero times an
    infinite bound is NaN, and a bound that is NaN stays NaN."""
    q, lo, hi = np.asarray(q, dtype=np.float64)[:, None, :], bounds[None, :, 0], bounds[None, :, 1]
    with np.errstate(invalid="ignore"):
        term = np.where(q > 0, q * hi, np.where(q < 0, q * lo, q * lo + q * hi))
        return np.where(np.isnan(lo) | np.isnan(hi), np.nan, term).sum((0, 2))


def select(scores, top_k, sink, recent):
    """The chosen blocks of one query and kv head, ascending, padded with -1."""
    n = len(scores)
    if n <= top_k:
        return list(range(n)) + [-1] * (top_k - n)
    key = np.where(np.isnan(scores), np.inf, scores).astype(np.float64)
    nan = np.isnan(scores).astype(int)
    forced = np.zeros(n, dtype=int)
    forced[:sink] = 1
    forced[n - recent:] = 1
    # last key of lexsort counts most: forced, NaN, score, then the lowest index
    order = np.lexsort((np.arange(n), -key, -nan, -forced))
    return sorted(order[:top_k].tolist())


def attend(q, k, v, scale):
    """q [group, D] over keys and values [tokens, D] -> (out, lse, sizes): sizes [group, D] are the sums of weights
    times |v|."""
    if not len(k):
        return np.zeros_like(q), np.full(len(q), -np.inf), np.zeros_like(q)
    x = q @ k.T * scale
    top = x.max(-1, keepdims=True)
    e = np.exp(x - top)
    w = e / e.sum(-1, keepdims=True)
    return w @ v, (top + np.log(e.sum(-1, keepdims=True)))[:, 0], w @ np.abs(v)
