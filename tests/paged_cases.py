"""Seeded caches and batches for the paged-cache tests (no operator arithmetic)."""
from __future__ import annotations

import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
# Half a step of each type, relative, and its smallest (subnormal) step.
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def make_cache(lens, Hkv, d, page, dtype, seed, spare=3, width=None, layers=None, unused=None):
    """(kpool, vpool, table, refs) on the CPU, every sequence's pages scattered.

    unused: value of everything that no sequence holds (pages, and rows behind a
    sequence's last token); default: random like the rest.
    """
    g = torch.Generator().manual_seed(seed)
    n = [-(-int(l) // page) for l in lens]
    P = sum(n) + spare
    width = width or max(n + [1]) + 1
    shape = ([layers] if layers else []) + [P, Hkv, page, d]
    kp = torch.randn(shape, generator=g).to(dtype)
    vp = torch.randn(shape, generator=g).to(dtype)
    ids = torch.randperm(P, generator=g).tolist()
    table = torch.full((len(n), width), -1, dtype=torch.int32)
    refs = torch.zeros(P, dtype=torch.int32)
    at = 0
    for b, k in enumerate(n):
        table[b, :k] = torch.tensor(ids[at:at + k], dtype=torch.int32)
        refs[table[b, :k].long()] = 1
        at += k
    if unused is not None:
        held = torch.zeros(P, page, dtype=torch.bool)
        for b, l in enumerate(lens):
            for t in range(0, int(l), page):
                held[int(table[b, t // page]), :min(page, int(l) - t)] = True
        for pool in (kp, vp):
            mask = ~held[:, None, :, None].expand(P, Hkv, page, d)
            pool.masked_fill_(mask if not layers else mask.expand(layers, *mask.shape), unused)
    return kp, vp, table, refs


def cu(T):
    return torch.tensor(np.concatenate([[0], np.cumsum(T)]), dtype=torch.int32)


def randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)
