"""GPU: uses of the operators on drafted trees that their header allows, beside the plain ones:
captured and replayed with new data in the same buffers, several calls at once, the largest sizes,
broadcast and strided inputs, wrong numbers in one row or one request alone."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import test_gpu_tree_attention as att
import test_gpu_tree_cache as cache
import test_gpu_tree_long as long_
import test_gpu_tree_verify as ver
from device_draft_verification_specverify_amd import tree
from oracle import tree as ora
from tree_helpers import DEV, dev

pytestmark = pytest.mark.gpu


def attention_call(c):
    """The call with its inputs made once: (function, the tensors that may be filled anew)."""
    args = [c[n] for n in ("q", "k_tree", "v_tree", "k_cache", "v_cache")]
    lengths = dev(c["lengths"])
    args += [dev(c["table"]), lengths, dev(c["start"]), dev(c["anc"].view(np.int64))]
    return (lambda: tree.specverify_tree_attention(*args, max_nodes=c["max_nodes"], want_lse=True),
            (c["q"], lengths))


def verify_call(c):
    put = lambda a: None if a is None else dev(a)  # noqa: E731
    names = ("target", "draft", "tokens", "parents", "node_start", "u", "r")
    args = [put(c[n]) for n in names]
    return (lambda: tree.specverify_tree_verify(*args, mode=c["mode"], max_nodes=c["max_nodes"],
                                                max_path=c["max_path"]), args)


@pytest.mark.parametrize("D,most", [(64, 5), (128, 40), (256, 9)])
def test_captured_attention_of_shared_prefixes(D, most):
    c = att.case(D, [2500, 700, 90], [most, 3, 1], 8, 2, D, 16, garbage=False)
    call, (q, lengths) = attention_call(c)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call()
    for step in range(4):
        lengths.copy_(dev(np.array([2500 - 700 * step, 700 - step, 90 - 30 * step], dtype=np.int32)))
        q.mul_(0.9)
        graph.replay()
        want, want_lse = call()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse), step


@pytest.mark.parametrize("mode", ver.MODES)
def test_captured_verification_of_shared_rows(mode):
    c = ver.case(4 + mode, 5, 12, "random", 40000, mode)
    call, args = verify_call(c)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for step in range(5):
        args[-2].mul_(0.8)
        args[-1].copy_((args[-1] + 0.37) % 1.0)
        graph.replay()
        call()
        torch.cuda.synchronize()
        ref = ver.reference(c | {"u": args[-2].cpu().numpy(), "r": args[-1].cpu().numpy()})
        assert np.array_equal(got.emitted.cpu().numpy(), ref["emitted"]), step
        assert np.array_equal(got.path.cpu().numpy(), ref["path"]), step


def test_calls_on_several_streams_at_once():
    # more workgroups than fit at a time: none may need another one's to be there
    cases = [ver.case(20 + i, 30 + i, 4, "random", 60000, ora.IID) for i in range(3)]
    calls = [verify_call(c)[0] for c in cases]
    big = att.case(3, [2500, 700], [9, 3], 8, 2, 128, 16)
    side, _ = attention_call(big)
    want = [c().emitted.clone() for c in calls]
    out, lse = side()
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got, outs = [], []
    for _ in range(4):
        for i, call in enumerate(calls):
            with torch.cuda.stream(streams[i]):
                got.append((i, call().emitted))
        with torch.cuda.stream(streams[3]):
            outs.append(side())
    torch.cuda.synchronize()
    for i, g in got:
        assert torch.equal(g, want[i])
    for o, l in outs:
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("mode", ver.MODES)
def test_the_largest_vocabulary(mode):
    ver.check(ver.case(30 + mode, 2, 3, "star", 1 << 22, mode))


@pytest.mark.parametrize("mode", [ora.IID, ora.DISTINCT])
def test_a_rejection_of_each_of_the_most_nodes(mode):
    # a star of 128 nodes, no child of which is accepted: 127 passes and a draw
    c = ver.case(40 + mode, 2, 128, "star", 40000, mode)
    c["u"][:] = 1.0 - 2.0 ** -53
    ref = ver.check(c)
    assert np.all(ref["out_token"] >= 0)


def test_attention_of_the_most_rows():
    # 128 nodes x 512 query heads of one key head
    c = long_.case(3, "random", [300, 0], [128, 1], 512, 1, 64, 16, torch.bfloat16)
    long_.check(c, 700)


def test_attention_of_many_requests_most_of_them_empty():
    rng = np.random.default_rng(4)
    B = 5000
    counts, lengths = np.zeros(B, dtype=np.int64), np.zeros(B, dtype=np.int64)
    some = np.sort(rng.choice(B, 150, replace=False))
    counts[some], lengths[some] = rng.integers(1, 5, 150), rng.integers(0, 300, 150)
    lengths[rng.choice(B, 50)] = 20          # a prefix and nothing to do
    lengths[0] = counts[0] = counts[B - 1] = 3
    c = long_.case(5, "random", lengths.tolist(), counts.tolist(), 4, 2, 64, 16, torch.bfloat16)
    long_.check(c, 400)


def test_broadcast_queries_and_drafts():
    c = att.case(6, [300, 20], [6, 3], 8, 2, 64, 16)
    c["q"] = c["q"][:1, :1].expand(9, 8, 64)
    att.check(c)
    # one draft distribution for all nodes, rows of the two sides in different distances
    v = ver.case(7, 4, 9, "random", 3000, ora.IID)
    T = len(v["tokens"])
    v["draft"][:] = v["draft"][0]
    ref = ver.reference(v)
    _, args = verify_call(v)
    wide = torch.zeros((T, 3005), device=DEV)
    wide[:, :3000] = args[0]
    o = tree.specverify_tree_verify(wide[:, :3000], args[1][:1].expand(T, 3000), *args[2:],
                                    mode=ora.IID, max_nodes=9, max_path=9)
    torch.cuda.synchronize()
    assert np.array_equal(o.emitted.cpu().numpy(), ref["emitted"])


def test_block_tables_with_rows_far_apart():
    c = att.case(8, [70, 200, 3], [5, 2, 1], 4, 2, 64, 16)
    out, _, _, _, _ = att.check(c)
    B, width = c["table"].shape
    wide = torch.full((B, width + 7), 1 << 30, dtype=torch.int32, device=DEV)
    wide[:, :width] = dev(c["table"])
    got, _ = tree.specverify_tree_attention(
        *(c[n] for n in ("q", "k_tree", "v_tree", "k_cache", "v_cache")), wide[:, :width],
        dev(c["lengths"]), dev(c["start"]), dev(c["anc"].view(np.int64)), max_nodes=c["max_nodes"])
    assert torch.equal(got, out)
    p = cache.plan_case(9, 20, "random", 9, 8, 60)
    B, width = p["block_table"].shape
    wide = torch.full((B, width + 5), 77, dtype=torch.int32, device=DEV)
    wide[:, :width] = dev(p["block_table"])
    o, _, err = cache.run_plan(p, wide[:, :width])
    ref = ora.plan(**p)
    assert err == 0 and np.array_equal(o.slots.cpu().numpy(), ref["slots"])
    assert np.array_equal(wide[:, :width].cpu().numpy(), ref["block_table"])
    assert torch.all(wide[:, width:] == 77)


@pytest.mark.parametrize("lengths", [[200, 40], [3000, 700]])
@pytest.mark.parametrize("D,most", [(64, 6), (128, 40), (256, 40)])
def test_wrong_numbers_stay_in_their_rows_and_requests(lengths, D, most):
    c = att.case(10 + D, lengths, [most, 3], 4, 2, D, 16)
    out, lse, _, _, _ = att.check(c)
    T = most + 3
    # a query: its row and head alone
    q = c["q"].clone()
    q[2, 1] = float("nan")
    got, got_lse, _ = att.run(c | {"q": q})
    keep = torch.ones((T, 4), dtype=torch.bool, device=DEV)
    keep[2, 1] = False
    assert torch.equal(got[keep], out[keep]) and torch.equal(got_lse[keep], lse[keep])
    assert torch.all(torch.isnan(got[2, 1]))
    # a cached key and a cached value: the rows of its request and key head alone
    page = int(c["table"][0, 7])
    for name in ("k_cache", "v_cache"):
        for what in (float("nan"), float("inf")):
            wrong = c[name].clone()
            wrong[page, 3, 1] = what
            got, got_lse, _ = att.run(c | {name: wrong})
            keep = torch.ones((T, 4), dtype=torch.bool, device=DEV)
            keep[:most, 2:] = False
            assert torch.equal(got[keep], out[keep]) and torch.equal(got_lse[keep], lse[keep])
            if name == "v_cache":
                assert not torch.isfinite(got[:most, 2:].float()).any()


def test_what_is_not_read_may_hold_anything():
    for mode in ver.MODES:
        c = ver.case(12 + mode, 6, 7, "random", 500, mode)
        want = ver.check(c)
        roots = c["node_start"][:-1]
        c["u"][roots] = float("nan")
        c["tokens"][roots] = -5
        if mode != ora.FIXED:
            for b in range(6):
                lo, hi = int(roots[b]), int(c["node_start"][b + 1])
                for i in range(lo, hi):
                    if i - lo not in c["parents"][lo:hi]:
                        c["draft"][i] = float("nan")
        got = ver.run(c)
        assert got["error"] == 0 and np.array_equal(got["emitted"], want["emitted"])
