"""Inputs shared by the tests of the operators on drafted token trees."""
from __future__ import annotations

import numpy as np
import torch

DEV = "cuda:0"


def parents_of(kind: str, n: int, rng) -> list:
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1) if n else []
    if kind == "branches":
        return [-1 if i == 0 else 0 if i <= 4 else i - 4 for i in range(n)]
    return [-1 if i == 0 else int(rng.integers(0, i)) for i in range(n)]  # "random"


def forest(kind: str, counts, rng):
    """(parents [T], node_start [B + 1]) as int32 arrays."""
    par = [p for n in counts for p in parents_of(kind, n, rng)]
    return np.array(par, dtype=np.int32), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def tables(lengths, page_size: int, extra_pages: int, spare: int, rng):
    """(block_table [B, max_pages] int32 with -1 behind the owned, owned pages, free pages, number)."""
    owned = [-(-x // page_size) for x in lengths]
    width = max(1, max(owned) + extra_pages)
    total = sum(owned) + spare
    ids = rng.permutation(total).astype(np.int32)
    table = np.full((len(lengths), width), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(owned):
        table[b, :k] = ids[at:at + k]
        at += k
    return table, np.array(owned, dtype=np.int32), ids[at:].copy(), max(total, 1)


def dev(a) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to("cpu").to(torch.float64).numpy()
