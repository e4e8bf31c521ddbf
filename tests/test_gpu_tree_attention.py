"""GPU: attention of drafted trees over a paged cache against the oracle in float64.

Tolerance, from the arithmetic (e = half a step of the storage type, f = 2^-24):
  softmax weights are rounded to the type for the product with the values: e * W with
    W = sum_j p_j |v_j|; the output is rounded once: e * |out|;
  scores: a float32 sum of D exact products, each partial sum off by at most f of its size, so
    d = (D + 2) f * S with S = max_j scale sum |q k_j|, and one rounding each of the scaled
    score and its difference from the maximum: 2 f * 2 S; exp2 in float32 (2 f). A weight is then
    off by a factor exp(+-c), c = d + 4 f S + 2 f, in the sum and in the denominator: 2 c W;
  sums over N keys in float32, and at most N rescalings of either sum: 4 N f W;
  the quotient: 3 f |out|.
lse: the same scores and sums, c + 4 N f, and the logarithm and its sum with the maximum: 4 f (|lse| + 1).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import device_draft_verification_specverify_amd as sv
from device_draft_verification_specverify_amd import tree
from oracle import tree as ora
from tree_helpers import DEV, dev, forest, host64, tables

pytestmark = pytest.mark.gpu

F = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def case(seed, lengths, counts, Hq, Hkv, D, page_size, dtype=torch.bfloat16, kind="random",
         layout="token", max_nodes=None, sharp=1.0, garbage=True, mask="tree"):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    max_nodes = max_nodes or max(max(counts), 1)
    parents, start = forest(kind, counts, rng)
    T = int(start[-1])
    table, owned, _, total = tables(lengths, page_size, 2, 2, rng)
    shape = (total, page_size, Hkv, D) if layout == "token" else (total, Hkv, page_size, D)
    caches = [torch.randn(shape, generator=g) for _ in "kv"]
    if layout == "head":
        caches = [t.transpose(1, 2) for t in caches]
    if garbage:  # slots behind a prefix and free pages hold anything
        used = torch.zeros(total, page_size, dtype=torch.bool)
        for b, n in enumerate(lengths):
            for j in range(n):
                used[table[b, j // page_size], j % page_size] = True
        for t in caches:
            t[~used] = float("nan")
    caches = [t.to(dtype).to(DEV) for t in caches]
    if layout == "head":
        caches = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in caches]
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g)
    qkv[:, :Hq] *= sharp
    qkv = qkv.to(dtype).to(DEV)
    q, k, v = qkv.split([Hq, Hkv, Hkv], dim=1)
    anc = None
    if mask != "chain":
        anc = np.concatenate([ora.ancestor_words(parents[start[b]:start[b + 1]], max_nodes)
                              for b in range(len(counts))] or [np.zeros((0, 1), np.uint64)])
    return dict(q=q, k_tree=k, v_tree=v, k_cache=caches[0], v_cache=caches[1], table=table,
                lengths=np.array(lengths, dtype=np.int32), start=start, anc=anc,
                max_nodes=max_nodes, scale=None)


def run(c, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    anc = None if c["anc"] is None else dev(c["anc"].view(np.int64))
    out, lse = tree.specverify_tree_attention(
        c["q"], c["k_tree"], c["v_tree"], c["k_cache"], c["v_cache"], dev(c["table"]),
        dev(c["lengths"]), dev(c["start"]), anc, max_nodes=c["max_nodes"], scale=c["scale"],
        want_lse=True, device_error=err, **kw)
    torch.cuda.synchronize()
    return out, lse, int(err.item())


def reference(c):
    D = c["q"].shape[2]
    return ora.attention(*(host64(c[k]) for k in ("q", "k_tree", "v_tree", "k_cache", "v_cache")),
                         c["table"], c["lengths"], c["start"], c["anc"], max_nodes=c["max_nodes"],
                         scale=c["scale"] or D ** -0.5)


def check(c, error=0, **kw):
    out, lse, err = run(c, **kw)
    assert err == error
    ref, ref_lse, weight, spread = reference(c)
    D = ref.shape[2]
    e = HALF_STEP[out.dtype]
    keys = int(c["lengths"].clip(0).max(initial=0)) + c["max_nodes"]
    cc = ((D + 2) * F * spread + 4 * F * spread + 2 * F)[:, :, None]
    tol = e * (weight + np.abs(ref)) * (1 + e) + (2 * cc + 4 * keys * F) * weight + 3 * F * np.abs(ref)
    got, got_lse = host64(out), host64(lse)
    rows = ~np.isnan(ref_lse)
    if not np.isnan(ref).any():
        tiny = torch.finfo(out.dtype).smallest_normal * e
        bad = np.abs(got - ref) > tol + tiny
        assert not bad.any(), (np.argwhere(bad)[:5].tolist(), np.abs(got - ref).max())
        fin = np.isfinite(ref_lse)
        assert np.array_equal(np.isneginf(got_lse), np.isneginf(ref_lse))
        tl = cc[:, :, 0] + 4 * keys * F + 4 * F * (np.abs(np.where(fin, ref_lse, 0)) + 1)
        assert np.all(np.abs(got_lse - ref_lse)[fin] <= tl[fin])
    return out, lse, ref, rows, tol


DTYPES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [8, 64, 80, 128, 200, 256])
@pytest.mark.parametrize("Hq,Hkv,most", [(4, 4, 5), (8, 2, 9), (21, 3, 12), (16, 1, 40)])
def test_widths_heads_and_rows(dtype, D, Hq, Hkv, most):
    # 5 to 640 rows of a key head: every split of a workgroup between rows and keys
    check(case(D + Hq, [37, 0, 130, 256], [most, 1, max(1, most // 2), most], Hq, Hkv, D, 16, dtype))


@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255,
                                    256, 257, 700])
@pytest.mark.parametrize("n", [1, 2, 33])
def test_lengths_around_tiles_and_pages(length, n):
    check(case(length * 5 + n, [length], [n], 8, 2, 64, 16))


@pytest.mark.parametrize("page_size", [1, 2, 8, 64, 512])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_page_sizes_and_layouts(page_size, layout):
    check(case(page_size, [300, 5, 77], [6, 7, 1], 8, 2, 128, page_size, layout=layout))


@pytest.mark.parametrize("n", [1, 9, 63, 64, 65, 100, 127, 128])
@pytest.mark.parametrize("mask", ["chain", "tree"])
def test_tree_sizes(n, mask):
    check(case(n, [40, 3], [n, 1], 4, 2, 64, 16, kind="chain" if mask == "chain" else "random",
               mask=mask, max_nodes=128 if n == 100 else None))


@pytest.mark.parametrize("dtype", DTYPES)
def test_sharp_rows(dtype):
    # scores up to about 60: the maximum moves by much from tile to tile
    check(case(4, [900, 100], [10, 3], 8, 2, 128, 32, dtype, sharp=12.0))


def test_rising_maxima():
    # later keys score higher, so every tile rescales what came before
    c = case(6, [1200], [5], 4, 1, 64, 16)
    c["k_cache"][:] = 0
    for j in range(1200):
        c["k_cache"][c["table"][0, j // 16], j % 16, 0, 0] = j / 100.0
    c["q"][:, :, 0] = 8.0
    check(c)


def test_a_long_prefix_is_split_over_the_card():
    check(case(7, [20000], [3], 2, 1, 64, 64))
    check(case(8, [9000, 0, 4000], [20, 2, 1], 16, 2, 128, 64))


def test_many_requests():
    rng = np.random.default_rng(3)
    counts = [int(x) for x in rng.integers(0, 4, 700)]
    check(case(9, [int(x) for x in rng.integers(0, 20, 700)], counts, 2, 1, 64, 8))


def test_rows_that_see_nothing():
    c = case(10, [0, 20, 0], [4, 3, 70], 4, 2, 64, 16)
    c["anc"][1] = 0                    # empty prefix and mask
    c["anc"][5] = 0                    # the prefix alone
    c["anc"][7 + 66, 0] = 0            # sees nodes 64 .. only
    out, lse, ref, _, _ = check(c)
    assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))


def test_bits_behind_a_tree_are_ignored():
    c = case(11, [5, 9], [3, 2], 4, 2, 64, 16, max_nodes=70)
    want, want_lse, _, _, _ = check(c)
    c["anc"] = c["anc"].copy()
    for i, n in ((0, 3), (1, 3), (2, 3), (3, 2), (4, 2)):
        c["anc"][i, 0] |= ~np.uint64(0) << np.uint64(n)
        c["anc"][i, 1] = ~np.uint64(0)
    got, got_lse, _ = run(c)
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("most", [6, 40, 100])
def test_wild_values_in_masked_nodes_stay_there(what, most):
    # a star: node i sees the root and itself, so a wild sibling must not reach it
    c = case(12, [33, 0], [most, 3], 4, 2, 64, 16, kind="star")
    out, lse, _, _, _ = check(c)
    wild = most - 2
    c["k_tree"][wild] = what
    c["v_tree"][wild] = what
    got, got_lse, _ = run(c)
    others = [i for i in range(most + 3) if i != wild]
    assert torch.equal(got[others], out[others]) and torch.equal(got_lse[others], lse[others])
    # only values wild: the node itself gets them, in the columns they are in
    c = case(12, [33, 0], [most, 3], 4, 2, 64, 16, kind="star")
    c["v_tree"][wild, :, 5] = what
    got, got_lse, _ = run(c)
    assert torch.equal(got[others], out[others]) and torch.equal(got_lse, lse)
    cols = [d for d in range(64) if d != 5]
    assert torch.equal(got[wild][:, cols], out[wild][:, cols])
    x = got[wild][:, 5].float()
    assert torch.all(torch.isnan(x)) if what != what else torch.all(x == what)


def test_rows_behind_the_last_request_stay():
    c = case(13, [10, 3], [4, 2], 4, 2, 64, 16)
    out = torch.full((6, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    c["start"] = np.array([0, 3, 4], dtype=np.int32)
    run(c, out=out)
    assert torch.all(out[4:] == 7.0) and not torch.any(out[:4] == 7.0)


def test_strided_output_and_single_heads():
    c = case(14, [50], [5], 1, 1, 128, 16)
    wide = torch.zeros((5, 3, 128), dtype=torch.bfloat16, device=DEV)
    out, _, _, _, _ = check(c, out=wide[:, 1:2])
    assert torch.all(wide[:, 0] == 0) and torch.all(wide[:, 2] == 0)


def test_broadcast_keys():
    # stride 0: all pages' tokens and both heads read one key
    c = case(15, [70, 31], [6, 2], 8, 2, 64, 16, garbage=False)
    one = c["k_cache"][:1, :1, :1].contiguous()
    c["k_cache"] = one.expand_as(c["k_cache"])
    c["v_cache"] = c["v_cache"][:1, :1, :1].contiguous().expand_as(c["k_cache"])
    check(c)


def test_bad_pages_count_as_zeros():
    c = case(16, [70, 40], [4, 2], 4, 2, 64, 16)
    c["table"][0, 2] = -1
    c["table"][1, 0] = c["k_cache"].shape[0]
    check(c, error=tree.SV_ERR_PAGE)


def test_lengths_outside_the_table_are_clamped():
    c = case(17, [32, 16, 5], [3, 2, 2], 4, 2, 64, 16, garbage=False)
    c["table"] = np.zeros_like(c["table"])
    c["lengths"] = np.array([1 << 30, -5, 5], dtype=np.int32)
    out, lse, err = run(c)
    assert err == tree.SV_ERR_LENGTH
    c["lengths"] = np.array([c["table"].shape[1] * 16, 0, 5], dtype=np.int32)
    check(c)
    again, _, _ = run(c)
    assert torch.equal(again, out)


def test_wrong_node_starts_leave_their_rows():
    c = case(18, [10, 20, 30], [3, 4, 5], 4, 2, 64, 16)
    good, _, _, _, _ = check(c)
    c["start"] = np.array([0, 3, 2, 12], dtype=np.int32)   # descends; 10 rows are too many
    out = torch.full((12, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    _, _, err = run(c, out=out)
    assert err == tree.SV_ERR_TREE
    assert torch.equal(out[:3], good[:3]) and torch.all(out[3:] == 7.0)


def test_results_do_not_depend_on_the_batch_around_them():
    # the same request alone and among others: within the tolerance of either
    c = case(19, [500, 64, 1000, 3], [9, 2, 17, 1], 8, 2, 128, 16)
    out, _, ref, _, tol = check(c)
    again, _, _ = run(c)
    assert torch.equal(out, again)


def test_no_nodes():
    c = case(20, [5, 6], [0, 0], 4, 2, 64, 16, max_nodes=3)
    out, lse, err = run(c)
    assert out.shape == (0, 4, 64) and err == 0


def test_refusals():
    c = case(21, [5], [3], 4, 2, 64, 16)
    with pytest.raises(sv.SpecVerifyError, match="status -1"):
        run(c | {"scale": -1.0})
    with pytest.raises(sv.SpecVerifyError, match="types differ"):
        run(c | {"q": c["q"].half()})
    with pytest.raises(sv.SpecVerifyError, match="status -3"):
        run(c, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    odd = torch.zeros(4 * 3 * 64 + 8, dtype=torch.bfloat16, device=DEV)[1:1 + 768].view(3, 4, 64)
    with pytest.raises(sv.SpecVerifyError, match="status -4"):
        run(c | {"q": odd})
