"""GPU: attention of chunks of new tokens over a paged cache against the oracle in float64 (the
tolerance is derived in serving_helpers.chunk_tolerance)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from device_draft_verification_specverify_amd import serving, tree
from serving_helpers import chunk_case, chunk_check, chunk_run, starts
from tree_helpers import DEV, dev, host64

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [8, 64, 80, 128, 200, 256])
@pytest.mark.parametrize("Hq,Hkv,most", [(4, 4, 5), (8, 2, 9), (21, 3, 19), (16, 1, 40)])
def test_widths_heads_and_rows(dtype, D, Hq, Hkv, most):
    # 5 to 640 rows of a key head: every kernel, each with full and partly filled row tiles
    chunk_check(chunk_case(D + Hq, [37, 0, 130, 256], [most, 1, max(1, most // 2), most], Hq, Hkv, D,
                           16, dtype))


@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 700])
@pytest.mark.parametrize("n", [1, 2, 33, 100])
def test_lengths_around_tiles_and_pages(length, n):
    chunk_check(chunk_case(length * 5 + n, [length], [n], 8, 2, 64, 16))


@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 1), (64, 7, 1), (256, 2, 2)])
def test_chunks_from_nothing_and_behind_a_prefix(n, D, Hq, Hkv):
    chunk_check(chunk_case(n + D, [0, 77], [n, n], Hq, Hkv, D, 16))


@pytest.mark.parametrize("page_size", [1, 2, 8, 64, 512])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("n", [7, 150])
def test_page_sizes_and_layouts(page_size, layout, n):
    chunk_check(chunk_case(page_size, [300, 5, 77], [n, 1, n - 3], 8, 2, 128, page_size, layout=layout))


@pytest.mark.parametrize("counts", [[1] * 9, [0, 0, 3, 0], [120, 1, 1, 0, 60, 1], [1, 130], [0, 1, 0]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_ragged_batches(counts, D):
    rng = np.random.default_rng(len(counts) + D)
    chunk_check(chunk_case(D, [int(x) for x in rng.integers(0, 400, len(counts))], counts, 8, 2, D, 32))


@pytest.mark.parametrize("most", [2, 40, 300, 100000])
def test_a_longer_bound_than_the_longest_chunk(most):
    # the bound picks the kernel; what it computes is the same
    chunk_check(chunk_case(3, [90, 7], [2, 1], 8, 2, 128, 16, max_chunk=most))


@pytest.mark.parametrize("heads", [65, 128, 200, 300])
@pytest.mark.parametrize("n", [1, 3])
def test_more_query_heads_than_a_workgroup_has_rows(heads, n):
    chunk_check(chunk_case(heads, [50, 0], [n, 1], heads, 1, 64, 16))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [10, 120])
def test_sharp_rows(dtype, n):
    # scores up to about 60: the maximum moves by much from tile to tile
    chunk_check(chunk_case(4, [900, 100], [n, 3], 8, 2, 128, 32, dtype, sharp=12.0))


def test_a_scale_of_ones_own():
    c = chunk_case(5, [64, 9], [70, 2], 4, 2, 64, 16)
    c["scale"] = 0.03
    chunk_check(c)


@pytest.mark.parametrize("n,D", [(1, 128), (20, 128), (90, 64), (70, 256)])
def test_many_shares_of_one_request(n, D):
    # few items, each with many tiles: shared out over the workgroups and joined
    chunk_check(chunk_case(n, [6000, 2500], [n, 1], 4, 1, D, 64))


def brute(c, rows):
    """out and lse of some rows in float64 on the device."""
    D, Hq = c["q"].shape[2], c["q"].shape[1]
    page, Hkv = c["k_cache"].shape[1:3]
    start = c["start"]
    outs, lses = [], []
    for i in rows:
        b = int(np.searchsorted(start, i, side="right")) - 1
        seen = int(c["lengths"][b]) + i - int(start[b]) + 1
        ids = dev(c["table"][b][:-(-seen // page)].astype(np.int64))
        k, v = (c[x][ids].flatten(0, 1)[:seen].double().repeat_interleave(Hq // Hkv, 1)
                for x in ("k_cache", "v_cache"))
        z = (c["q"][i].double() * k).sum(-1).T * D ** -0.5  # [Hq, seen]
        lses.append(torch.logsumexp(z, 1))
        outs.append((torch.softmax(z, 1).T[:, :, None] * v).sum(0))
    return torch.stack(outs).cpu().numpy(), torch.stack(lses).cpu().numpy()


@pytest.mark.parametrize("D,Hq,Hkv,lengths,counts", [
    (128, 8, 2, [0], [2500]), (128, 7, 1, [3000, 5], [1700, 900]), (64, 4, 4, [0, 0, 64], [1200, 1, 1300]),
    (256, 4, 2, [100], [1100]), (80, 21, 3, [1], [777])])
def test_long_chunks_by_samples(D, Hq, Hkv, lengths, counts):
    c = chunk_case(D + Hq, lengths, counts, Hq, Hkv, D, 64, garbage=False)
    out, lse, err = chunk_run(c)
    assert err == 0
    T = sum(counts)
    rows = sorted(set(np.random.default_rng(1).integers(0, T, 40)) | {0, 1, 63, 64, 65, 255, 256, T - 1})
    ref, ref_lse = brute(c, rows)
    # random values of size 1: sum p |v| <= max |v| < 6, weights and output rounded once each
    tol = 2.0 ** -8 * (6 + np.abs(ref)) * 1.02 + 1e-4
    assert np.all(np.abs(host64(out)[rows] - ref) <= tol)
    assert np.all(np.abs(host64(lse)[rows] - ref_lse) <= 1e-4)


# ------------------------------------------------------------- what is not seen
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n,D,length", [(6, 64, 20), (40, 128, 500), (150, 128, 30), (100, 64, 2500),
                                        (90, 256, 77), (300, 128, 0)])
def test_wild_values_of_later_tokens(what, n, D, length):
    c = chunk_case(n + D, [length, 33], [n, 2], 4, 2, D, 16)
    out, lse = chunk_check(c)
    token = n // 2
    at = length + token
    page, off = int(c["table"][0, at // 16]), at % 16
    before = [i for i in range(n + 2) if i < token or i >= n]
    after = list(range(token, n))
    c["v_cache"][page, off, 1, 5] = what  # of key head 1: query heads 2 and 3
    got, got_lse, _ = chunk_run(c)
    assert torch.equal(got[before], out[before]) and torch.equal(got_lse, lse)
    cols = [d for d in range(D) if d != 5]
    assert torch.equal(got[after][:, :, cols], out[after][:, :, cols])
    assert torch.equal(got[after][:, :2], out[after][:, :2])
    x = got[after][:, 2:, 5].float()
    assert torch.all(torch.isnan(x)) if what != what else torch.all(x == what)
    # its keys wild too: no row before it changes
    c["k_cache"][page, off] = what
    got, got_lse, _ = chunk_run(c)
    assert torch.equal(got[before], out[before]) and torch.equal(got_lse[before], lse[before])


def test_rows_outside_chunks_are_left_as_they_were():
    c = chunk_case(9, [40, 3], [20, 2], 4, 2, 64, 16)
    c["q"] = torch.cat([c["q"], c["q"][:5]])
    chunk_check(c)
    c["start"] = c["start"] + 3
    chunk_check(c)


@pytest.mark.parametrize("n", [3, 90])
def test_wrong_data(n):
    c = chunk_case(11, [40, 30, 50], [n, 2, n], 4, 2, 64, 16, garbage=False)
    bad = dict(c, table=c["table"].copy())
    bad["table"][0, 1], bad["table"][2, 0] = -1, 10 ** 6
    chunk_check(bad, error=16)
    chunk_check(dict(c, lengths=np.array([40, -5, 50], np.int32)), error=64)
    # a length whose chunk would end behind the table is taken as what fits
    most = c["table"].shape[1] * 16
    table = np.where(c["table"] < 0, 0, c["table"])
    chunk_check(dict(c, table=table, lengths=np.array([40, 30, most - 1], np.int32)), error=64)
    chunk_check(dict(c, start=np.array([0, n, n - 2, 2 * n + 2], np.int32)), error=8)
    chunk_check(dict(c, start=np.array([0, -1, n + 2, 2 * n + 2], np.int32)), error=8)
    chunk_check(dict(c, start=np.array([0, n, n + 2, 9 * n], np.int32)), error=8)
    if n > 3:
        chunk_check(dict(c, max_chunk=n - 1), error=8)


def test_a_chunk_longer_than_its_table():
    c = chunk_case(12, [0, 4], [40, 2], 4, 2, 64, 16, garbage=False)
    chunk_check(dict(c, table=c["table"][:, :2].copy()), error=64)


def test_offsets_beyond_32_bits():
    # pages 2^32 bytes and more into the cache
    D, Hkv, page = 128, 8, 64
    pages = (5 << 30) // (page * Hkv * D * 2)
    k = torch.zeros((pages, page, Hkv, D), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    small = chunk_case(13, [90, 10], [80, 1], 16, Hkv, D, page, garbage=False)
    n = small["k_cache"].shape[0]
    k[-n:], v[-n:] = small["k_cache"], small["v_cache"]
    want, want_lse, _ = chunk_run(small)
    table = np.where(small["table"] >= 0, small["table"] + pages - n, -1).astype(np.int32)
    got, got_lse, err = chunk_run(dict(small, k_cache=k, v_cache=v, table=table))
    assert err == 0 and torch.equal(got, want) and torch.equal(got_lse, want_lse)


def test_unusual_strides():
    c = chunk_case(14, [70, 9], [75, 3], 6, 2, 64, 16, garbage=False)
    want, want_lse, _ = chunk_run(c)
    T = c["q"].shape[0]
    heads_first = torch.empty((6, T, 64), dtype=c["q"].dtype, device=DEV).transpose(0, 1)
    heads_first.copy_(c["q"])
    wide = torch.full((T, 6, 96), float("nan"), dtype=c["q"].dtype, device=DEV)
    k, v = (torch.stack([x, x], 2)[:, :, 0] for x in (c["k_cache"], c["v_cache"]))
    table = np.full((2, c["table"].shape[1] + 5), -1, np.int32)
    table[:, :c["table"].shape[1]] = c["table"]
    got, got_lse = serving.specverify_chunk_attention(
        heads_first, k, v, dev(table)[:, :c["table"].shape[1]], dev(c["lengths"]), dev(c["start"]),
        max_chunk=c["max_chunk"], out=wide[:, :, :64], want_lse=True)
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    assert torch.isnan(wide[:, :, 64:]).all()
    # one query for all tokens
    one = c["q"][:1].expand(T, -1, -1)
    a, _, _ = chunk_run(dict(c, q=one))
    b, _, _ = chunk_run(dict(c, q=one.contiguous()))
    assert torch.equal(a, b)


@pytest.mark.parametrize("n", [1, 9, 40, 120])
def test_a_chunk_is_a_chain_of_nodes_that_was_committed(n):
    # tree attention of a chain outside the cache, and the same tokens as a chunk inside
    D, Hq, Hkv, page, length = 128, 8, 2, 16, 333
    c = chunk_case(n, [length], [n], Hq, Hkv, D, page, garbage=False)
    at = length + torch.arange(n, device=DEV)
    ids = dev(c["table"][0].astype(np.int64))[at // page]
    k, v = c["k_cache"][ids, at % page], c["v_cache"][ids, at % page]
    want, want_lse = tree.specverify_tree_attention(
        c["q"], k, v, c["k_cache"], c["v_cache"], dev(c["table"]), dev(c["lengths"]),
        dev(starts([n])), max_nodes=128, want_lse=True)
    got, got_lse, _ = chunk_run(c)
    # both are off by at most a rounding of weights and output: twice 2^-8 (sum p |v| + |out|), |v| < 6
    assert (got.float() - want.float()).abs().max() <= 2 * 2.0 ** -8 * (6 + want.float().abs().max())
    assert (got_lse - want_lse).abs().max() <= 1e-4


def test_results_do_not_change_from_call_to_call():
    c = chunk_case(15, [3000, 17, 500], [200, 1, 90], 8, 2, 128, 16)
    a = chunk_run(c)
    for _ in range(3):
        b = chunk_run(c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_rows_at_all():
    c = chunk_case(16, [10, 0], [0, 0], 4, 2, 64, 16)
    out, lse, err = chunk_run(c)
    assert out.shape == (0, 4, 64) and err == 0
