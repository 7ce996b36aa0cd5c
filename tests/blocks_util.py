"""Inputs of the block-sparse step's tests: batches with permuted pages, made on the CPU."""

import numpy as np
import torch


def batch(lens, new, ps, seed, spare=3):
    """Page table, token map and pool size of requests of these lengths; int32 CPU tensors."""
    g = torch.Generator().manual_seed(seed)
    n = [-(-x // ps) for x in lens]
    pages = sum(n) + spare
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    req = np.repeat(np.arange(len(lens)), new)
    pos = np.concatenate([np.arange(a - m, a) for a, m in zip(lens, new)]) if len(lens) else np.zeros(0)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32)  # noqa: E731
    return dict(lens=lens, new=new, ps=ps, pages=pages, indptr=i32([0] + list(np.cumsum(n))), indices=perm[:sum(n)].clone(),
                last=i32([x - (c - 1) * ps if c else 0 for x, c in zip(lens, n)]), req=i32(req), pos=i32(pos))


def lists(s, dev):
    """(batch_indices, positions, kv_indptr, kv_indices) on the device."""
    return tuple(s[k].to(dev) for k in ("req", "pos", "indptr", "indices"))


def pages_of(s, b):
    return s["indices"][int(s["indptr"][b]):int(s["indptr"][b + 1])].long().numpy()


def to64(t):
    return t.detach().cpu().double().numpy()
