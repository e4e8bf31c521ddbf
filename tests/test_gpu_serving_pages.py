"""GPU: pages taken, given back and shared, against the oracle: whole numbers and copies, equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import device_draft_verification_specverify_amd as sv
from device_draft_verification_specverify_amd import serving
from oracle import serving as ora
from serving_helpers import i32, laid_out, pages_case, resize_check, resize_run, same, word
from tree_helpers import DEV

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- resize
@pytest.mark.parametrize("page", [1, 2, 16, 64, 512])
@pytest.mark.parametrize("lengths,counts", [([0], [1]), ([0], [700]), ([15, 16, 17], [1, 1, 1]), ([5, 0, 33], [0, 0, 0]),
                                            ([100, 0, 31, 64], [28, 65, 1, 0])])
def test_pages_for_chunks(page, lengths, counts):
    resize_check(pages_case(page, lengths, counts, page))


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("extra", [0, 2])
def test_some_end_and_some_go_on(shared, extra):
    lengths, counts = [100, 40, 7, 90, 0, 33], [5, 0, 200, 16, 17, 1]
    c = pages_case(3, lengths, counts, 16, extra=extra, ended=(0, 3),
                   shared=[(1, 0, 2), (5, 3, 2), (3, 1, 1)] if shared else ())
    if not shared:
        c["shares"] = None
    resize_check(c)


def test_a_page_comes_free_with_its_last_holder():
    c = pages_case(4, [48, 48, 48], [0, 0, 0], 16, shared=[(1, 0, 3), (2, 0, 2)])
    for ended in ((0,), (0, 1), (0, 1, 2), (1, 2)):
        resize_check(dict(c, prefix_len=np.where(np.isin(np.arange(3), ended), 0, c["prefix_len"])))


def test_what_is_given_back_can_be_taken():
    # no free page but those of the request that ends
    c = pages_case(5, [64, 32], [0, 60], 16, spare=0, ended=(0,))
    got = resize_check(c)
    assert set(got["block_table"][1][2:6]) <= set(c["block_table"][0][:4])


def test_a_list_that_does_not_reach():
    c = pages_case(6, [10, 20, 30, 40], [30, 40, 2, 30], 16, spare=3)
    got = resize_check(c, error=16)
    assert np.all(got["slots"][c["chunk_start"][1]:c["chunk_start"][2]] == -1)


def test_wrong_data_in_a_large_cache():
    # more pages than one workgroup goes through, the same mistakes
    c = pages_case(12, [40, 30, 50, 700], [5, 40, 7, 300], 16, spare=20000)
    resize_check(c)
    resize_check(dict(c, prefix_len=np.array([40, -1, 50, 700])), error=64)
    resize_check(dict(c, chunk_start=np.array([0, 5, 3, 20, 300])), error=8)
    resize_check(dict(c, chunk_start=np.array([0, 5, 45, 53, 10])), error=8)
    table = c["block_table"].copy()
    table[0, 2], table[2, 0] = -1, c["num_pages"]
    resize_check(dict(c, block_table=table, prefix_len=np.array([0, 30, 0, 0]), chunk_start=np.array([0, 0, 300, 300, 352])), error=16)
    free = c["free_pages"].copy()
    free[c["free_head"] + 3] = -1
    resize_check(dict(c, free_pages=free), error=16)
    for head in (-1, len(free) + 1):
        resize_check(dict(c, free_head=head), error=16)
    resize_check(dict(c, free_head=len(free) - 21), error=16)
    resize_check(dict(c, free_head=1, prefix_len=np.zeros(4, int), chunk_start=np.zeros(5, int), rows=0), error=16)


def test_pages_that_come_free_are_taken_in_a_large_cache():
    # takes that lie in several blocks of pages, some from what came free and some from the list
    n = [9000, 12000, 64, 0]
    c = pages_case(13, n, [0, 1000, 9500, 3000], 1, spare=5000, ended=(0,))
    resize_check(c)
    c = pages_case(14, n, [0, 100, 12500, 3000], 1, spare=4000, ended=(0,), shared=[(1, 0, 5000)])
    resize_check(c, error=16)


@pytest.mark.parametrize("B,num", [(1, 9000), (600, 40000), (65536, 70000)])
def test_large_batches_and_caches(B, num):
    rng = np.random.default_rng(B)
    lengths, counts = rng.integers(0, 60 if B > 1000 else 700, B), rng.integers(0, 2 if B > 1000 else 90, B)
    if B == 1:
        lengths, counts = np.array([70000]), np.array([5000])
    page = 64 if B > 1000 else 16
    c = pages_case(B, [int(x) for x in lengths], [int(x) for x in counts], page, ended=tuple(range(0, B, 3)) if B > 1 else (),
                   shared=[(b, b - 1, 1) for b in range(1, B, 3) if min(lengths[b], lengths[b - 1]) >= page])
    resize_check(c)


def test_without_chunks():
    c = pages_case(7, [100, 40], [0, 0], 16, extra=1, ended=(1,))
    want = ora.resize(**dict(c, chunk_start=None))
    got = resize_run(dict(c, chunk_start=None))
    same(got, dict(want, position=None, slots=None))


def test_rows_outside_every_chunk():
    c = pages_case(8, [10, 20], [5, 6], 16)
    resize_check(dict(c, rows=c["rows"] + 9))
    resize_check(dict(c, rows=c["rows"] + 9, chunk_start=c["chunk_start"] + 4))


def test_wrong_lengths_chunks_pages_and_heads():
    c = pages_case(9, [40, 30, 50], [5, 40, 7], 16)
    resize_check(dict(c, prefix_len=np.array([40, -1, 50])), error=64)
    resize_check(dict(c, prefix_len=np.array([40, 99, 50])), error=64)
    resize_check(dict(c, pages=np.array([3, 2, -1])), error=64)
    resize_check(dict(c, pages=np.array([3, 2, 100])), error=64)
    resize_check(dict(c, chunk_start=np.array([0, 5, 3, 20])), error=8)
    resize_check(dict(c, chunk_start=np.array([0, 5, 45, 53])), error=8)
    table = c["block_table"].copy()
    table[0, 2], table[2, 0] = -1, c["num_pages"]
    resize_check(dict(c, block_table=table), error=16)
    resize_check(dict(c, block_table=table, prefix_len=np.array([0, 30, 0]), chunk_start=None, rows=0), error=16)
    free = c["free_pages"].copy()
    free[c["free_head"]] = 10 ** 8
    resize_check(dict(c, free_pages=free), error=16)
    for head in (-1, len(free) + 1):
        resize_check(dict(c, free_head=head), error=16)
    # a list without room for what comes back
    resize_check(dict(c, free_head=1, prefix_len=np.array([0, 0, 0]), chunk_start=np.array([0, 0, 0, 0]), rows=0), error=16)


def test_the_same_page_given_back_twice_by_one_request():
    c = pages_case(10, [64], [0], 16, ended=(0,))
    c["block_table"][0, 2] = c["block_table"][0, 1]
    c["shares"] = None
    resize_check(c)


# ---------------------------------------------------------------- fork
def fork_case(seed, lengths, forks, *, B=None, page=16, layers=2, H=2, D=64, dtype=torch.bfloat16, layout="token", spare=None):
    """Requests of `lengths` tokens behind which the others are empty; forks = [(source, target)]."""
    B = B or max([t for _, t in forks] + [len(lengths) - 1]) + 1
    c = pages_case(seed, list(lengths) + [0] * (B - len(lengths)), [0] * B, page, spare=len(forks) + 1 if spare is None else spare)
    g = torch.Generator().manual_seed(seed)
    c["k_cache"], c["v_cache"] = (laid_out(torch.randn((layers, c["num_pages"], page, H, D), generator=g).to(dtype).to(DEV), layout)
                                  for _ in "kv")
    c["source"], c["target"] = (np.array(x) for x in (zip(*forks) if forks else ([], [])))
    return c


def host(t):
    return t.cpu().float().numpy() if t.is_floating_point() else t.cpu().numpy()


def fork_run(c, **kw):
    err, table = word(), i32(c["block_table"])
    k, v = c["k_cache"].clone(memory_format=torch.preserve_format), c["v_cache"].clone(memory_format=torch.preserve_format)
    o = serving.specverify_pages_fork(i32(c["source"]), i32(c["target"]), i32(c["prefix_len"]), i32(c["pages"]), table,
                                      i32(c["free_pages"]), i32(c["free_head"]), i32(c["shares"]), k, v, device_error=err, **kw)
    torch.cuda.synchronize()
    return dict(prefix_len=host(o.prefix_len), pages=host(o.pages), free_head=int(o.free_head.item()), shares=host(o.shares),
                block_table=host(table), k_cache=host(k), v_cache=host(v), error=int(err.item()))


def fork_check(c, error=0):
    want = ora.fork(c["source"], c["target"], c["prefix_len"], c["pages"], c["block_table"], c["free_pages"], c["free_head"],
                    c["shares"], host(c["k_cache"]), host(c["v_cache"]), num_pages=c["num_pages"])
    assert want["error"] == error, want["error"]
    got = fork_run(c)
    same(got, want)
    return got


@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 32, 100])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_one_request_four_times(length, dtype, layout):
    fork_check(fork_case(length, [length], [(0, t) for t in (1, 2, 3, 4)], dtype=dtype, layout=layout))


@pytest.mark.parametrize("page,H,D,layers", [(1, 1, 8, 3), (8, 3, 80, 1), (64, 8, 128, 5), (16, 4, 256, 2)])
def test_shapes(page, H, D, layers):
    fork_check(fork_case(page, [70, 0, 33, 5], [(0, 4), (2, 5), (3, 7), (0, 6), (1, 8)], page=page, H=H, D=D, layers=layers))


def test_many_forks():
    rng = np.random.default_rng(0)
    lengths = [int(x) for x in rng.integers(0, 200, 300)]
    fork_check(fork_case(1, lengths, [(int(rng.integers(0, 300)), 300 + t) for t in rng.permutation(700)], layers=1, H=1, D=8))


def test_a_list_that_does_not_reach_for_all_forks():
    c = fork_case(2, [20, 32, 5], [(0, 3), (1, 4), (2, 5), (0, 6), (1, 7)], spare=2)
    fork_check(c, error=16)


def test_forks_that_may_not_be():
    c = fork_case(3, [20, 40, 5], [(0, 3), (0, 0), (0, 1), (1, 3), (-1, 4), (2, 99), (99, 5), (2, 6), (1, -3), (0, 6)], B=7, spare=12)
    got = fork_check(c, error=128)
    assert got["prefix_len"].tolist() == [20, 40, 5, 20, 0, 0, 5]


def test_wrong_sources_pages_and_heads():
    c = fork_case(4, [20, 40, 5], [(0, 3), (1, 4), (2, 5)])
    fork_check(dict(c, prefix_len=np.array([20, 400, 5, 0, 0, 0])), error=64)
    fork_check(dict(c, pages=np.array([2, 3, -1, 0, 0, 0])), error=64)
    table = c["block_table"].copy()
    table[0, 1], table[1, 0] = -1, 10 ** 6
    fork_check(dict(c, block_table=table), error=16)
    free = c["free_pages"].copy()
    free[c["free_head"] + 1] = -9
    fork_check(dict(c, free_pages=free), error=16)
    fork_check(dict(c, free_head=-4), error=16)


def test_no_forks():
    got = fork_check(fork_case(5, [20, 3], []))
    assert got["prefix_len"].tolist() == [20, 3]


def test_forked_requests_end_one_after_the_other():
    c = fork_case(6, [40], [(0, 1), (0, 2)])
    f = fork_run(c)
    state = dict(c, prefix_len=f["prefix_len"], pages=f["pages"], block_table=f["block_table"], free_head=f["free_head"],
                 shares=f["shares"], chunk_start=None, rows=0)
    for name in ("source", "target", "k_cache", "v_cache"):
        state.pop(name)
    at_first = c["free_head"]
    for ended in (1, 0, 2):
        state["prefix_len"] = np.where(np.arange(3) == ended, 0, state["prefix_len"])
        got = resize_run(state)
        same(got, dict(ora.resize(**state), position=None, slots=None))
        state.update({k: got[k] for k in ("pages", "block_table", "free_pages", "free_head", "shares")})
    assert state["free_head"] == at_first - 3 and not state["shares"].any()
    assert sorted(state["free_pages"][state["free_head"]:]) == list(range(c["num_pages"]))


def test_pages_beyond_32_bits():
    D, H, page = 128, 8, 64
    pages = (5 << 30) // (page * H * D * 2)
    k = torch.zeros((1, pages, page, H, D), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    k[0, pages - 1], v[0, pages - 1] = 3.0, 4.0
    table = i32([[pages - 1, -1], [-1, -1]])
    o = serving.specverify_pages_fork(i32([0]), i32([1]), i32([40, 0]), i32([1, 0]), table, i32([pages - 2]), i32(0),
                                      torch.zeros(pages, dtype=torch.int32, device=DEV), k, v)
    assert o.pages.tolist() == [1, 1] and table.tolist() == [[pages - 1, -1], [pages - 2, -1]]
    assert torch.all(k[0, pages - 2, :40] == 3.0) and torch.all(v[0, pages - 2, :40] == 4.0)
    assert not k[0, pages - 2, 40:].any() and not k[0, pages - 3].any()


@pytest.mark.parametrize("wrong", ["free", "shares", "table", "rows"])
def test_refusals(wrong):
    c = pages_case(11, [40, 30], [5, 6], 16)
    if wrong == "free":
        c["free_pages"], c["free_head"] = c["free_pages"][1:], 0
    elif wrong == "shares":
        c["shares"] = c["shares"][1:]
    elif wrong == "rows":
        c["chunk_start"] = None
    with pytest.raises(sv.SpecVerifyError):
        if wrong == "table":
            serving.specverify_pages_resize(i32(c["prefix_len"]), i32(c["pages"]), i32(c["block_table"][:1]).expand(2, -1),
                                            i32(c["free_pages"]), i32(c["free_head"]), page_size=16, num_pages=c["num_pages"])
        else:
            resize_run(c)
