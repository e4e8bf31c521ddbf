"""Inputs and checks shared by the tests of the operators around a verification step."""
from __future__ import annotations

import numpy as np
import torch

from device_draft_verification_specverify_amd import serving
from oracle import serving as ora
from tree_helpers import DEV, dev, host64, tables

F = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def starts(counts) -> np.ndarray:
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def laid_out(t, layout):
    """The same values with heads in front of a page's tokens in memory."""
    return t if layout == "token" else t.transpose(-3, -2).contiguous().transpose(-3, -2)


# ---------------------------------------------------------------- chunk attention
def chunk_case(seed, lengths, counts, Hq, Hkv, D, page_size, dtype=torch.bfloat16, layout="token",
               max_chunk=None, sharp=1.0, garbage=True, spare_pages=2):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    held = [a + n for a, n in zip(lengths, counts)]
    table, _, _, total = tables(held, page_size, spare_pages, 2, rng)
    caches = [torch.randn((total, page_size, Hkv, D), generator=g) for _ in "kv"]
    if garbage:  # slots behind a chunk and free pages hold anything
        used = torch.zeros(total, page_size, dtype=torch.bool)
        for b, n in enumerate(held):
            at = torch.arange(n)
            used[torch.from_numpy(table[b])[at // page_size].long(), at % page_size] = True
        for t in caches:
            t[~used] = float("nan")
    k, v = (laid_out(t.to(dtype).to(DEV), layout) for t in caches)
    T = sum(counts)
    q = (torch.randn((T, Hq + 3, D), generator=g) * sharp).to(dtype).to(DEV)[:, :Hq]
    return dict(q=q, k_cache=k, v_cache=v, table=table, lengths=np.array(lengths, np.int32),
                start=starts(counts), max_chunk=max_chunk or max(max(counts), 1), scale=None)


def chunk_run(c, **kw):
    err = word()
    out, lse = serving.specverify_chunk_attention(
        c["q"], c["k_cache"], c["v_cache"], dev(c["table"]), dev(c["lengths"]), dev(c["start"]),
        max_chunk=c["max_chunk"], scale=c["scale"], want_lse=True, device_error=err, **kw)
    torch.cuda.synchronize()
    return out, lse, int(err.item())


def chunk_reference(c):
    return ora.attention(*(host64(c[k]) for k in ("q", "k_cache", "v_cache")), c["table"],
                         c["lengths"], c["start"], max_chunk=c["max_chunk"],
                         scale=c["scale"] or c["q"].shape[2] ** -0.5)


def chunk_tolerance(ref, ref_lse, weight, spread, dtype, keys):
    """(out, lse). From the arithmetic (e half a step of the type, f = 2^-24): softmax weights
    rounded for the product, e W with W = sum p |v|, and the output once, e |out|; scores are float32
    sums of D products, (D + 2) f S with S = max sum |q k| scale, scaled and taken from the maximum,
    4 f S, then exp2, 2 f: a factor exp(+-c) in sum and denominator, 2 c W; sums over the keys and
    rescalings, 4 N f W; the quotient, 3 f |out|. lse: c + 4 N f and the logarithm, 4 f (|lse| + 1)."""
    D, e = ref.shape[2], HALF_STEP[dtype]
    c = (D + 2) * F * spread + 4 * F * spread + 2 * F
    tol = e * (weight + np.abs(ref)) * (1 + e) + (2 * c[:, :, None] + 4 * keys * F) * weight + 3 * F * np.abs(ref)
    return tol + torch.finfo(dtype).smallest_normal * e, c + 4 * keys * F + 4 * F * (np.abs(ref_lse) + 1)


def chunk_check(c, error=0, **kw):
    """Runs a case and holds it to the oracle; rows that belong to no chunk keep their NaN."""
    out = torch.full(c["q"].shape, float("nan"), dtype=c["q"].dtype, device=DEV)
    out, lse, err = chunk_run(c, out=out, **kw)
    assert err == error, err
    ref, ref_lse, weight, spread = chunk_reference(c)
    keys = int(c["lengths"].clip(0).max(initial=0)) + c["max_chunk"]
    tol, tol_lse = chunk_tolerance(ref, ref_lse, weight, spread, out.dtype, keys)
    got, got_lse = host64(out), host64(lse)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), np.argwhere(np.isnan(got) != np.isnan(ref))[:5]
    there = ~np.isnan(ref)
    bad = np.abs(got - ref)[there] > tol[there]
    assert not bad.any(), (np.argwhere(there)[bad][:5].tolist(), np.abs(got - ref)[there].max())
    rows = ~np.isnan(ref_lse)
    assert np.all(np.abs(got_lse - ref_lse)[rows] <= tol_lse[rows])
    return out, lse


# ---------------------------------------------------------------- pages
def pages_case(seed, lengths, counts, page_size, *, extra=0, spare=None, shared=(), ended=()):
    """A batch in the pages: `lengths` cached tokens, `counts` new ones to come, `extra` pages owned
    beyond the cached, shared = (request, the one it began as, full pages), requests that end."""
    rng = np.random.default_rng(seed)
    B = len(lengths)
    owned = [-(-a // page_size) + extra for a in lengths]
    need = [-(-(a + n) // page_size) for a, n in zip(lengths, counts)]
    total = sum(owned) + (sum(need) if spare is None else spare)
    ids = rng.permutation(total)
    table = np.full((B, max(owned + need) + 1), -1, np.int64)
    at = 0
    for b, k in enumerate(owned):
        table[b, :k] = ids[at:at + k]
        at += k
    shares = np.zeros(total, np.int64)
    for b, other, n in shared:
        table[b, :n] = table[other, :n]
        shares[table[b, :n]] += 1
    used = {int(table[b, j]) for b in range(B) for j in range(owned[b])}
    free = [int(p) for p in ids if int(p) not in used]
    prefix = np.array([0 if b in ended else a for b, a in enumerate(lengths)])
    return dict(prefix_len=prefix, pages=np.array(owned), block_table=table,
                free_pages=np.array([-7] * (total - len(free)) + free), free_head=total - len(free),
                page_size=page_size, num_pages=total,
                chunk_start=starts([0 if b in ended else n for b, n in enumerate(counts)]),
                rows=int(sum(0 if b in ended else n for b, n in enumerate(counts))), shares=shares)


def i32(a):
    return None if a is None else dev(np.asarray(a, dtype=np.int32).reshape(-1) if np.ndim(a) < 2 else
                                      np.asarray(a, dtype=np.int32))


def resize_run(c, **kw):
    """(outputs as the oracle's dict, error)."""
    err, table, free = word(), i32(c["block_table"]), i32(c["free_pages"])
    o = serving.specverify_pages_resize(
        i32(c["prefix_len"]), i32(c["pages"]), table, free, i32(c["free_head"]),
        page_size=c["page_size"], num_pages=c["num_pages"], chunk_start=i32(c["chunk_start"]),
        rows=c["rows"], shares=i32(c["shares"]), device_error=err, **kw)
    torch.cuda.synchronize()
    h = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    return dict(pages=h(o.pages), free_head=int(o.free_head.item()), shares=h(o.shares),
                position=h(o.position), slots=h(o.slots), block_table=h(table), free_pages=h(free),
                error=int(err.item()))


def same(got, want):
    for k, x in want.items():
        if x is None or got[k] is None:
            assert got[k] is None or k in ("position", "slots"), k
        else:
            assert np.array_equal(got[k], x), (k, got[k], x)


def resize_check(c, error=0):
    want = ora.resize(**c)
    assert want["error"] == error, want["error"]
    got = resize_run(c)
    same(got, want)
    return got
