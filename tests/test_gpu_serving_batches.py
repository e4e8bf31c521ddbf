"""GPU: chunk attention of batches whose requests go to different kernels, of more requests than a
workgroup has threads, over pages and values that are not as usual in the middle of long chunks."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from serving_helpers import chunk_case, chunk_check, chunk_reference, chunk_run, chunk_tolerance
from tree_helpers import host64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 3, 1), (80, 4, 1), (256, 2, 1)])
def test_more_requests_than_threads(D, Hq, Hkv):
    rng = np.random.default_rng(D)
    counts = [0 if b % 7 == 1 else 1 for b in range(700)]
    lengths = [int(x) for x in rng.integers(0, 40, 700)]
    for b, n in ((3, 90), (511, 70), (512, 65), (699, 130)):
        counts[b], lengths[b] = n, 100 - b % 60
    chunk_check(chunk_case(D, lengths, counts, Hq, Hkv, D, 16, spare_pages=0))


@pytest.mark.parametrize("rows", [64, 65, 128, 129, 256, 257])
@pytest.mark.parametrize("others", [[], [1, 1], [0, 5]])
def test_requests_at_the_borders_between_the_kernels(rows, others):
    # one query head, so that a token is a row
    chunk_check(chunk_case(rows, [50, 7, 30][:1 + len(others)], [rows] + others, 2, 2, 64, 16))


@pytest.mark.parametrize("D", [64, 96, 128])
def test_the_same_request_alone_and_in_a_batch(D):
    # (what kernel takes it, and how it is shared out, may differ: the result only by roundings)
    both = chunk_case(D, [333, 90], [100, 1], 8, 2, D, 16, garbage=False)
    out, lse, _ = chunk_run(both)
    ref, ref_lse, weight, spread = chunk_reference(both)
    tol, tol_lse = chunk_tolerance(ref, ref_lse, weight, spread, out.dtype, 433)
    for b, (lo, hi) in enumerate(((0, 100), (100, 101))):
        one = dict(both, q=both["q"][lo:hi], table=both["table"][b:b + 1], lengths=both["lengths"][b:b + 1],
                   start=np.array([0, hi - lo], np.int32), max_chunk=hi - lo)
        got, got_lse, _ = chunk_run(one)
        assert np.all(np.abs(host64(got) - host64(out)[lo:hi]) <= 2 * tol[lo:hi])
        assert np.all(np.abs(host64(got_lse) - host64(lse)[lo:hi]) <= 2 * tol_lse[lo:hi])


@pytest.mark.parametrize("page_size", [1, 2, 4, 16, 128])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_bad_pages_amid_a_long_chunk(page_size, D):
    c = chunk_case(page_size + D, [200, 500], [150, 40], 4, 2, D, page_size, garbage=False)
    table = c["table"].copy()
    for b, keys in ((0, (3, 130, 349)), (1, (0, 300))):
        for k in keys:
            table[b, k // page_size] = -1 if k % 2 else 10 ** 9
    chunk_check(dict(c, table=table), error=16)


@pytest.mark.parametrize("n,D", [(3, 128), (60, 64), (200, 128), (150, 256)])
@pytest.mark.parametrize("what", [float("inf"), float("nan")])
def test_wild_values_in_front_of_a_chunk_stay_in_their_column(n, D, what):
    c = chunk_case(n + D, [700, 50], [n, 2], 4, 2, D, 16)
    out, lse = chunk_check(c)
    c["v_cache"][int(c["table"][0, 10]), 7, 1, 9] = what
    got, got_lse, _ = chunk_run(c)
    cols = [d for d in range(D) if d != 9]
    assert torch.equal(got_lse, lse) and torch.equal(got[:, :2], out[:, :2]) and torch.equal(got[n:], out[n:])
    assert torch.equal(got[:n][:, :, cols], out[:n][:, :, cols])
    assert not torch.isfinite(got[:n, 2:, 9]).any()


@pytest.mark.parametrize("n,D", [(3, 64), (40, 128), (200, 128), (150, 256)])
def test_wild_keys_and_queries_stay_in_their_rows(n, D):
    c = chunk_case(n * 3 + D, [300, 50], [n, 2], 4, 2, D, 16)
    out, lse = chunk_check(c)
    c["q"][n // 2, 1] = float("nan")
    got, got_lse, _ = chunk_run(c)
    same = torch.ones(n + 2, 4, dtype=torch.bool)
    same[n // 2, 1] = False
    assert torch.equal(got[same.to(got.device)], out[same.to(got.device)])
    assert torch.equal(got_lse[same.to(got.device)], lse[same.to(got.device)])
    assert torch.isnan(got[n // 2, 1]).all() and torch.isnan(got_lse[n // 2, 1])


def test_scores_that_rise_and_fall_by_much():
    # the reference of the softmax may lag behind the maximum by 2^8 and not by more: keys whose scores
    # climb by 3 a tile, then one far above all, then far below
    c = chunk_case(5, [1000], [140], 2, 1, 128, 16, dtype=torch.float16, garbage=False)
    c["q"][:] = 0
    c["q"][:, :, 0] = 16.0
    c["k_cache"][:] *= 0.01
    ids = c["table"][0]
    for j in range(1140):
        x = min(j / 64 * 0.13, 3.0) if j != 700 else 8.0
        c["k_cache"][int(ids[j // 16]), j % 16, 0, 0] = x if j < 900 else -2.0
    chunk_check(c)
