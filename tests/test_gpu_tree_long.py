"""GPU: attention where each of the 256 workgroups has a share of many tiles: page ids are fetched
in several batches, a share goes over the ends of items, and each tile rescales the ones before.

Values are indicators: column (j / 64) % D of key j is 1, the others 0. So all sums are of
non-negative numbers, the bounds below are relative, and a block of 64 keys that is lost, taken
twice or read in another's place moves a column by about 1 / (keys / (64 D)), 3 to 40 per cent.

Tolerance, as for short prefixes, from the arithmetic (e = half a step of the type, f = 2^-24): the
weights' rounding and the output's, e each; scores off by d = (D + 2) f S and 4 f S more, 2 f for
the exponential, in the sum and in the denominator; sums of at most N terms one after the other and
as many rescalings, 4 N f, where N is a share's keys and the shares of an item; 3 f for the quotient.
Below a type's smallest normal number its step no longer shrinks, and half a step is t = e times that
number (f16: 2^-11 2^-14 = 2^-25). So an output is off by up to t, and so is each weight, where the
largest is 1: t sum v / sum p.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import test_gpu_tree_attention as att
from tree_helpers import DEV, dev, forest

pytestmark = pytest.mark.gpu

F = att.F
WORKERS = 256


def case(seed, kind, lengths, counts, Hq, Hkv, D, page_size, dtype):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    owned = [-(-n // page_size) for n in lengths]
    total = sum(owned) + 3
    ids = rng.permutation(total).astype(np.int32)
    table = np.full((len(lengths), max(owned) + 1), -1, dtype=np.int32)
    shape = (total, page_size, Hkv, D)
    k_cache = torch.full(shape, float("nan"), dtype=dtype, device=DEV)
    v_cache = torch.full(shape, float("nan"), dtype=dtype, device=DEV)
    at = 0
    for b, n in enumerate(lengths):
        table[b, :owned[b]] = ids[at:at + owned[b]]
        at += owned[b]
        pages = dev(table[b, :owned[b]].astype(np.int64))
        j = torch.arange(owned[b] * page_size, device=DEV)
        k = torch.randn((len(j), Hkv, D), generator=g, device=DEV)
        if kind == "rising":  # scores from 0 to 8 along the prefix
            k.zero_()
            k[:, :, 0] = (j / max(n, 1) * D ** 0.5)[:, None]
        v = ((j // 64 % D)[:, None, None] == torch.arange(D, device=DEV)).float()
        v = v.expand(-1, Hkv, -1).clone()
        k[n:], v[n:] = float("nan"), float("nan")
        k_cache[pages] = k.to(dtype).view(-1, page_size, Hkv, D)
        v_cache[pages] = v.to(dtype).view(-1, page_size, Hkv, D)
    parents, start = forest("random", counts, rng)
    T = int(start[-1])
    q = torch.randn((T, Hq, D), generator=g, device=DEV)
    if kind == "flat":
        q.zero_()
    elif kind == "rising":
        q.zero_()
        q[:, :, 0] = 8.0
    k_tree = torch.randn((T, Hkv, D), generator=g, device=DEV)
    v_tree = torch.rand((T, Hkv, D), generator=g, device=DEV)
    anc = np.concatenate([att.ora.ancestor_words(parents[start[b]:start[b + 1]], max(counts))
                          for b in range(len(counts))])
    return dict(q=q.to(dtype), k_tree=k_tree.to(dtype), v_tree=v_tree.to(dtype), k_cache=k_cache,
                v_cache=v_cache, table=table, lengths=np.array(lengths, dtype=np.int32),
                start=start, anc=anc, max_nodes=max(counts), scale=None)


def check(c, chain):
    """Against float64, one product per request and key head; `chain` is N above."""
    out, lse, err = att.run(c)
    assert err == 0
    T, Hq, D = out.shape
    Hkv = c["k_tree"].shape[1]
    G, e, scale = Hq // Hkv, att.HALF_STEP[out.dtype], D ** -0.5
    tiny = torch.finfo(out.dtype).smallest_normal * e
    for b, n in enumerate(c["lengths"].tolist()):
        lo, hi = int(c["start"][b]), int(c["start"][b + 1])
        if lo == hi:
            continue
        size = c["k_cache"].shape[1]
        pages = dev(c["table"][b, :-(-n // size)].astype(np.int64))
        nodes = torch.arange(hi - lo, device=DEV)
        words = dev(c["anc"][lo:hi].view(np.int64))
        see = (words[:, nodes // 64] >> (nodes % 64)) & 1 == 1
        see = torch.cat([torch.ones((hi - lo, n), dtype=torch.bool, device=DEV), see], 1)
        see = see.repeat_interleave(G, 0)
        for h in range(Hkv):
            kk = torch.cat([c["k_cache"][pages, :, h].reshape(-1, D)[:n], c["k_tree"][lo:hi, h]]).double()
            vv = torch.cat([c["v_cache"][pages, :, h].reshape(-1, D)[:n], c["v_tree"][lo:hi, h]]).double()
            q = c["q"][lo:hi, h * G:(h + 1) * G].reshape(-1, D).double()
            s = (q @ kk.t().contiguous() * scale).masked_fill(~see, -float("inf"))
            top = s.max(1, keepdim=True).values
            p = torch.exp(s - top)
            sums = p.sum(1, keepdim=True)
            ref, ref_lse = p @ vv / sums, (top + torch.log(sums))[:, 0]
            spread = (q.abs() @ kk.abs().t().contiguous()).max(1).values * scale
            cc = (D + 6) * F * spread + 2 * F
            rel = 2 * e * (1 + e) + 2 * cc + 4 * chain * F + 3 * F
            got = out[lo:hi, h * G:(h + 1) * G].reshape(-1, D).double()
            bad = (got - ref).abs() > rel[:, None] * ref + tiny * (1 + vv.sum(0) / sums)
            assert not bool(bad.any()), (b, h, bad.nonzero()[:5].tolist())
            got_lse = lse[lo:hi, h * G:(h + 1) * G].reshape(-1).double()
            tol = cc + 4 * chain * F + 4 * F * (ref_lse.abs() + 1)
            assert bool(((got_lse - ref_lse).abs() <= tol).all()), (b, h)
    return out, lse


# rows of a key head (nodes x 4) that choose each kernel, and the keys of a tile and the tiles of a
# batch of page ids there
KERNELS = [(64, 5, 128, 32), (64, 30, 128, 32), (64, 50, 64, 64), (128, 5, 128, 16),
           (128, 30, 128, 16), (128, 50, 64, 32), (256, 5, 64, 8), (256, 30, 32, 16)]


def lengths_of(tile, batch, heads):
    """A long, some short, two long requests: 2.4 batches of tiles a worker in all."""
    keys = int(2.4 * batch * tile * WORKERS / heads)
    return [int(0.45 * keys) + 7, 3, 0, tile, int(0.25 * keys) + 1, int(0.3 * keys)]


@pytest.mark.parametrize("kind", ["flat", "random", "rising"])
@pytest.mark.parametrize("D,nodes,tile,batch", KERNELS)
def test_shares_of_many_tiles(kind, D, nodes, tile, batch):
    lengths = lengths_of(tile, batch, 8)
    c = case(D + nodes, kind, lengths, [nodes, 1, nodes, 2, nodes, 3], 32, 8, D, 16, torch.bfloat16)
    check(c, int(2.5 * batch) * tile + WORKERS)


@pytest.mark.parametrize("page_size", [2, 512])
@pytest.mark.parametrize("D,nodes,tile,batch", [KERNELS[0], KERNELS[4], KERNELS[6]])
def test_shares_of_many_tiles_in_other_pages(page_size, D, nodes, tile, batch):
    # pages of fewer rows than a wavefront loads at once, and of several tiles
    lengths = lengths_of(tile, batch, 8)
    c = case(D, "random", lengths, [nodes, 1, nodes, 2, nodes, 3], 32, 8, D, page_size, torch.float16)
    check(c, int(2.5 * batch) * tile + WORKERS)


def test_long_shares_of_heads_narrower_than_their_tiles():
    c = case(5, "random", lengths_of(128, 16, 8), [5, 1, 4, 2, 5, 3], 32, 8, 80, 16, torch.bfloat16)
    check(c, 40 * 128 + WORKERS)


def test_many_items_of_a_worker():
    # 320 requests of 8 heads, 10 items a worker, with a long one between them
    rng = np.random.default_rng(2)
    lengths = [int(x) for x in rng.integers(0, 200, 320)]
    lengths[150] = 9000
    counts = [int(x) for x in rng.integers(0, 6, 320)]
    check(case(6, "random", lengths, counts, 32, 8, 64, 16, torch.bfloat16), 9006)


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("D,nodes,tile,batch", [KERNELS[0], KERNELS[5], KERNELS[6]])
def test_wild_values_behind_shares_of_many_tiles(what, D, nodes, tile, batch):
    c = case(9, "random", lengths_of(tile, batch, 8), [nodes, 1, nodes, 2, nodes, 3], 32, 8, D, 16,
             torch.bfloat16)
    c["anc"] = np.zeros_like(c["anc"])
    for b in range(6):
        for i in range(int(c["start"][b]), int(c["start"][b + 1])):  # a node sees itself
            m = i - int(c["start"][b])
            c["anc"][i, m // 64] = np.uint64(1) << np.uint64(m % 64)
    out, lse, _ = att.run(c)
    wild = nodes - 1
    c["v_tree"][wild, :, 5] = what
    got, got_lse, _ = att.run(c)
    assert torch.equal(got_lse, lse)
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[wild, :, 5] = False
    assert torch.equal(got[rest], out[rest])
    x = got[wild, :, 5].float()
    assert torch.all(torch.isnan(x)) if what != what else torch.all(x == what)
