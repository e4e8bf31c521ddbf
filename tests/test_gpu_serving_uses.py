"""GPU: the operators around a verification step as they are used together and in the ways that their
header allows: prompts in chunks through the pages, replies forked, drafted trees with penalties on
top; captured and replayed; on several streams; with workspaces of any contents."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import test_gpu_serving_logits as log
import test_gpu_serving_pages as pag
import test_gpu_serving_rotate as rot
from device_draft_verification_specverify_amd import serving, tree
from oracle import serving as ora
from serving_helpers import HALF_STEP, chunk_case, i32, pages_case, starts, word
from tree_helpers import DEV, dev, host64

pytestmark = pytest.mark.gpu

L, HQ, HKV, D, V, PAGE, WIDTH = 2, 8, 2, 64, 700, 16, 40
FREQ = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float()


class Server:
    """Buffers and weights of a loop over at most B requests of a toy model of two layers, whose
    queries, keys and values are fixed functions of a token; the position comes in by rotation."""

    def __init__(self, B, seed):
        g = torch.Generator().manual_seed(seed)
        w = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.B, self.pages_in_all = B, B * WIDTH
        self.embed = w(V, D).to(DEV)
        self.wqkv = (w(L, D, (HQ + 2 * HKV) * D) / 8).to(DEV)
        self.head = (w(HQ * D, V) / 3).to(DEV)
        self.norm = [(1 + 0.2 * w(L, D)).bfloat16().to(DEV) for _ in "qk"]
        self.freq = FREQ.to(DEV)
        cache = lambda: torch.full((L, self.pages_in_all, PAGE, HKV, D), float("nan"), dtype=torch.bfloat16, device=DEV)  # noqa: E731
        self.k_cache, self.v_cache = cache(), cache()
        self.table = torch.full((B, WIDTH), -1, dtype=torch.int32, device=DEV)
        self.free = dev(np.random.default_rng(seed).permutation(self.pages_in_all).astype(np.int32))
        self.free_head = i32(0)
        self.shares = torch.zeros(self.pages_in_all, dtype=torch.int32, device=DEV)
        self.prefix = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.pages = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.err = word()

    def qkv(self, layer, tokens):
        x = self.embed[tokens.long()] @ self.wqkv[layer]
        return x.view(-1, HQ + 2 * HKV, D).bfloat16().split([HQ, HKV, HKV], 1)

    def room(self, counts):
        o = serving.specverify_pages_resize(
            self.prefix, self.pages, self.table, self.free, self.free_head, page_size=PAGE,
            num_pages=self.pages_in_all, chunk_start=dev(starts(counts)), rows=sum(counts), shares=self.shares,
            device_error=self.err)
        self.pages, self.free_head, self.shares = o.pages, o.free_head, o.shares
        return o

    def chunk(self, tokens, counts):
        """New tokens through all layers into the pages: attention outputs [L, T, HQ, D]."""
        o, outs = self.room(counts), []
        start = dev(starts(counts))
        for i in range(L):
            q, k, v = self.qkv(i, tokens)
            q, _ = serving.specverify_rotate(q, k, v, o.position, self.freq, q_weight=self.norm[0][i],
                                             k_weight=self.norm[1][i], slots=o.slots, k_cache=self.k_cache[i],
                                             v_cache=self.v_cache[i], device_error=self.err)
            out, _ = serving.specverify_chunk_attention(q, self.k_cache[i], self.v_cache[i], self.table, self.prefix,
                                                        start, max_chunk=max(counts), device_error=self.err)
            outs.append(out)
        self.prefix = self.prefix + i32(counts)
        return torch.stack(outs)

    def want(self, tokens, layer):
        """Attention of one request's tokens in float64 from the definitions: out and its tolerance."""
        q, k, v = self.qkv(layer, tokens)
        n = len(tokens)
        rotated = []
        for x, w in ((q, self.norm[0][layer]), (k, self.norm[1][layer])):
            y, _ = ora.rotate(host64(x), host64(w), np.arange(n), FREQ.numpy(), eps=1e-6, interleaved=False)
            rotated.append(torch.from_numpy(y).bfloat16().double().numpy())
        caches = [np.asarray(x).reshape(1, n, HKV, D) for x in (rotated[1], host64(v))]
        out, _, weight, spread = ora.attention(rotated[0], *caches, np.zeros((1, 1), np.int64), [0], [0, n], max_chunk=n,
                                               scale=D ** -0.5)
        # A query or key that lies between two bfloat16 values to 32 f may be rounded to the other one: a
        # step, 2^-7 of it. Were it all of them, scores would be off by 2 * 2^-7 S; weights by twice that.
        e = HALF_STEP[torch.bfloat16]
        return out, 1.02 * e * (weight + np.abs(out)) + 4 * 2 * e * spread[:, :, None] * weight + 1e-4


def test_prompts_in_chunks_replies_and_drafts():
    s = Server(6, 1)
    rng = np.random.default_rng(1)
    text = [rng.integers(0, V, n) for n in (75, 130, 33)]
    # prompts of three requests in chunks of uneven sizes
    got = [[], [], []]
    at = [0, 0, 0]
    for counts in ([40, 1, 33], [0, 100, 0], [35, 29, 0]):
        now = np.concatenate([text[b][at[b]:at[b] + n] for b, n in enumerate(counts)])
        out = host64(s.chunk(dev(now.astype(np.int32)), counts + [0, 0, 0]))
        for b, n in enumerate(counts):
            lo = sum(counts[:b])
            got[b].append(out[:, lo:lo + n])
            at[b] += n
    assert int(s.err.item()) == 0 and s.prefix.tolist() == [75, 130, 33, 0, 0, 0]
    for b in range(3):
        for i in range(L):
            want, tol = s.want(dev(text[b].astype(np.int32)), i)
            assert np.all(np.abs(np.concatenate([x[i] for x in got[b]]) - want) <= tol), (b, i)

    # two more replies to the first prompt, one to the second: then a token each, and the sources another one
    f = serving.specverify_pages_fork(i32([0, 0, 1]), i32([3, 4, 5]), s.prefix, s.pages, s.table, s.free, s.free_head,
                                      s.shares, s.k_cache, s.v_cache, device_error=s.err)
    s.prefix, s.pages, s.free_head, s.shares = f.prefix_len, f.pages, f.free_head, f.shares
    assert s.prefix.tolist() == [75, 130, 33, 75, 75, 130] and int(s.shares.sum().item()) == 4 + 4 + 8
    new = rng.integers(0, V, 6)
    out = host64(s.chunk(dev(new.astype(np.int32)), [1] * 6))
    whole = [np.append(text[b], new[k]) for k, b in enumerate((0, 1, 2, 0, 0, 1))]
    for k in range(6):
        for i in range(L):
            want, tol = s.want(dev(whole[k].astype(np.int32)), i)
            assert np.all(np.abs(out[i, k] - want[-1]) <= tol[-1]), (k, i)

    # a step of drafted trees on top: keys outside the cache, penalties by each node's path
    parents = [-1, 0, 0, 1, 2]
    N, T = 5, 30
    start, par = dev(starts([N] * 6)), dev(np.tile(parents, 6).astype(np.int32))
    tokens = dev(rng.integers(0, V, T).astype(np.int32))
    plan = tree.specverify_tree_plan(par, start, s.prefix, s.pages, s.table, s.free, s.free_head, page_size=PAGE,
                                     num_pages=s.pages_in_all, max_nodes=N, max_path=3, device_error=s.err)
    sums, ks, vs = 0, [], []
    for i in range(L):
        q, k, v = s.qkv(i, tokens)
        q, k = serving.specverify_rotate(q, k, None, plan.position, s.freq, q_weight=s.norm[0][i], k_weight=s.norm[1][i])
        v = v.contiguous()
        ks.append(k)
        vs.append(v)
        out, _ = tree.specverify_tree_attention(q, k, v, s.k_cache[i], s.v_cache[i], s.table, s.prefix, start,
                                                plan.ancestors, max_nodes=N, device_error=s.err)
        sums = sums + out.float()
        for b in range(6):  # each path is a text of its own
            for node, line in ((3, [0, 1, 3]), (4, [0, 2, 4])):
                text_b = np.append(whole[b], host64(tokens[b * N:][line]).astype(np.int64))
                want, tol = s.want(dev(text_b.astype(np.int32)), i)
                assert np.all(np.abs(host64(out[b * N + node]) - want[-1]) <= tol[-1]), (b, node, i)
    logits = sums.view(T, HQ * D) @ s.head
    history = np.full((6, 200), -1, np.int32)
    for b in range(6):
        history[b, :len(whole[b])] = whole[b]
    ones = torch.ones(6, device=DEV)
    x = serving.specverify_penalize(logits, tokens, start, dev(history), s.prefix, dev(np.array([75, 130, 33, 75, 75, 130], np.int32)),
                                    1.5 * ones, 0.5 * ones, 0.25 * ones, ancestors=plan.ancestors, max_nodes=N, device_error=s.err)
    ref, size, _, err = ora.penalize(host64(logits), host64(tokens).astype(int), host64(start).astype(int), history,
                                     host64(s.prefix), [75, 130, 33, 75, 75, 130], [1.5] * 6, [0.5] * 6, [0.25] * 6,
                                     paths=[[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4]] * 6, max_nodes=N)
    assert err == 0 and np.all(np.abs(host64(x) - ref) <= 9 * 2.0 ** -24 * size + 2.0 ** -24 * np.abs(ref))
    p = torch.softmax(x, 1)
    res = tree.specverify_tree_verify(p, None, tokens, par, start, torch.rand(T, dtype=torch.float64, device=DEV) * 0.01,
                                      torch.rand(6, dtype=torch.float64, device=DEV), mode=tree.DRAFT_FIXED, max_nodes=N,
                                      max_path=3, device_error=s.err)
    before = s.prefix.clone()
    s.prefix = tree.specverify_tree_commit(torch.stack(ks), torch.stack(vs), s.k_cache, s.v_cache, start, res.path,
                                           res.accept_len, plan.slots, s.prefix, max_nodes=N, device_error=s.err)
    s.pages, s.free_head = plan.pages, plan.free_head
    assert int(s.err.item()) == 0 and torch.equal(s.prefix, before + res.accept_len + 1)
    # what was committed is what the next token sees
    grown = [np.concatenate([whole[b], host64(tokens[b * N:][res.path[b, :int(res.accept_len[b]) + 1].long()]).astype(np.int64)])
             for b in range(6)]
    last = rng.integers(0, V, 6)
    out = host64(s.chunk(dev(last.astype(np.int32)), [1] * 6))
    for b in range(6):
        want, tol = s.want(dev(np.append(grown[b], last[b]).astype(np.int32)), 1)
        assert np.all(np.abs(out[1, b] - want[-1]) <= tol[-1]), b
    # and when all have ended, every page is free again
    s.prefix = torch.zeros_like(s.prefix)
    s.room([0] * 6)
    assert int(s.err.item()) == 0 and s.free_head.tolist() == [0] and not s.shares.any()
    assert sorted(s.free.tolist()) == list(range(s.pages_in_all))


def calls(seed):
    """(name, function, tensors to fill anew) of every operator, inputs made once."""
    g = torch.Generator().manual_seed(seed)
    c = chunk_case(seed, [900, 60], [90, 3], 8, 2, 128, 16, garbage=False)
    table, lengths, start = dev(c["table"]), dev(c["lengths"]), dev(c["start"])
    yield "attention", lambda: serving.specverify_chunk_attention(
        c["q"], c["k_cache"], c["v_cache"], table, lengths, start, max_chunk=90, want_lse=True), [c["q"]]
    one = chunk_case(seed, [3000, 60, 9], [1, 1, 1], 8, 2, 64, 16, garbage=False)
    args = [dev(one[k]) for k in ("table", "lengths", "start")]
    yield "single tokens", lambda: serving.specverify_chunk_attention(
        one["q"], one["k_cache"], one["v_cache"], *args, max_chunk=1, want_lse=True), [one["q"]]
    r = rot.case(seed, 20, 8, 2, 128, 128, torch.bfloat16)
    caches = [torch.zeros((3, 16, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    slots = torch.randperm(48, generator=g)[:20].to(DEV)
    yield "rotate", lambda: (serving.specverify_rotate(**r, slots=slots, k_cache=caches[0], v_cache=caches[1])[0],
                             *caches), [r["q"], r["k"]]
    p = log.case(seed, [9, 3], 40000, [600, 20], bias=3, mask=True)
    put = {k: dev(p[k]) for k in ("tokens", "start", "history", "prefix", "prompt", "rep", "pres", "freq", "bias_start",
                                  "bias_token", "bias", "mask")}
    yield "penalize", lambda: (serving.specverify_penalize(
        p["logits"], put["tokens"], put["start"], put["history"], put["prefix"], put["prompt"], put["rep"], put["pres"],
        put["freq"], max_nodes=9, bias_start=put["bias_start"], bias_token=put["bias_token"], bias=put["bias"],
        mask=put["mask"]),), [p["logits"]]
    z = pages_case(seed, [100, 40, 300], [30, 0, 50], 16, shared=[(1, 0, 2)], ended=(0,))
    held = {k: i32(z[k]) for k in ("prefix_len", "pages", "block_table", "free_pages", "free_head", "chunk_start", "shares")}

    def resize():
        o = serving.specverify_pages_resize(
            held["prefix_len"], held["pages"], held["block_table"], held["free_pages"], held["free_head"], page_size=16,
            num_pages=z["num_pages"], chunk_start=held["chunk_start"], rows=z["rows"], shares=held["shares"])
        return o.pages, o.free_head, o.shares, o.position, o.slots, held["block_table"], held["free_pages"]
    yield "resize", resize, []
    f = pag.fork_case(seed, [70, 33], [(0, 2), (1, 3), (0, 4)])
    k = {n: i32(f[n]) for n in ("source", "target", "prefix_len", "pages", "block_table", "free_pages", "free_head", "shares")}

    def fork():
        o = serving.specverify_pages_fork(*k.values(), f["k_cache"], f["v_cache"])
        return o.prefix_len, o.pages, o.free_head, o.shares, k["block_table"], f["k_cache"], f["v_cache"]
    yield "fork", fork, []


def equal(a, b):
    return len(a) == len(b) and all(x is y or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", ["attention", "single tokens", "rotate", "penalize", "resize", "fork"])
def test_captured_calls_replay(name):
    call, fill = next((f, t) for n, f, t in calls(5) if n == name)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for step in range(4):
        for t in fill:
            t.mul_(0.9)
        graph.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in got]
        want = call()  # the program's own work between the replays
        torch.cuda.synchronize()
        assert equal(mine, want), step


def test_all_of_them_on_four_streams_at_once():
    sets = [list(calls(20 + i)) for i in range(4)]
    want = [[[t.clone() for t in call()] for _, call, _ in one] for one in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[] for _ in sets]
    for _ in range(3):
        for i, (one, st) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(st):
                got[i].append([[t.clone() for t in call()] for _, call, _ in one])
    torch.cuda.synchronize()
    for i in range(4):
        for turn in got[i]:
            for (name, _, _), a, b in zip(sets[i], turn, want[i]):
                assert equal(a, b), name


def test_workspaces_of_any_contents_serve_calls_of_different_sizes():
    ws = torch.empty(160 << 20, dtype=torch.uint8, device=DEV)
    z = pages_case(3, [100, 40, 300], [30, 0, 50], 16, shared=[(1, 0, 2)], ended=(0,))
    f = pag.fork_case(3, [70, 33], [(0, 2), (1, 3), (0, 4)])
    cases = [chunk_case(i, [2000, 60], [n, 3], 8, 2, D, 16, garbage=False) for i, (n, D) in enumerate([(1, 64), (100, 128), (30, 256)])]
    from serving_helpers import chunk_run, resize_run
    want = [chunk_run(c) for c in cases], resize_run(z), pag.fork_run(f)
    for fill in (0xFF, 0x00, 0x7F):
        ws.fill_(fill)
        for c, (out, lse, _) in zip(cases, want[0]):
            got = chunk_run(c, ws=ws)
            assert torch.equal(got[0], out) and torch.equal(got[1], lse)
        for got, ref in ((resize_run(z, ws=ws), want[1]), (pag.fork_run(f, ws=ws), want[2])):
            for k, x in ref.items():
                assert np.array_equal(got[k], x), k


def test_a_call_waits_for_its_stream_alone():
    c = chunk_case(7, [500], [70], 8, 2, 64, 16, garbage=False)
    args = (c["k_cache"], c["v_cache"], dev(c["table"]), dev(c["lengths"]), dev(c["start"]))
    want, _ = serving.specverify_chunk_attention(c["q"], *args, max_chunk=70)
    q = torch.zeros_like(c["q"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        q.copy_(c["q"])  # ordered in front of the call on this stream only
        got, _ = serving.specverify_chunk_attention(q, *args, max_chunk=70)
    side.synchronize()
    assert torch.equal(got, want)
