"""GPU: penalties, biases and masks on logits against the oracle in float64.

Tolerance, from the arithmetic (f = 2^-24): 1 / repetition and the product 2 f, frequency * count +
presence and the difference 2 f, up to 4 biases of one id 4 f and their sum with the logit f: 9 f of what
was added up in absolute values, plus half a step of the result's type. Which are -inf is exact.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import device_draft_verification_specverify_amd as sv
from device_draft_verification_specverify_amd import serving
from oracle import serving as ora
from oracle import tree as ora_tree
from serving_helpers import F, HALF_STEP, word
from tree_helpers import DEV, dev, forest, host64

pytestmark = pytest.mark.gpu


def case(seed, counts, V, lengths, *, kind="chain", dtype=torch.float32, bias=0, mask=False, max_nodes=None):
    rng = np.random.default_rng(seed)
    B, max_nodes = len(counts), max_nodes or max(max(counts), 1)
    parents, start = forest(kind, counts, rng)
    T, H = int(start[-1]), max(max(lengths), 1)
    zipf = lambda *s: ((V ** rng.random(s)).astype(np.int64).clip(1, V) - 1).astype(np.int32)  # noqa: E731
    c = dict(tokens=zipf(T), start=start, history=zipf(B, H), max_nodes=max_nodes,
             prefix=np.array(lengths, np.int32), prompt=np.array([a // 3 for a in lengths], np.int32),
             rep=(0.7 + rng.random(B)).astype(np.float32), pres=rng.random(B).astype(np.float32),
             freq=(rng.random(B) - 0.2).astype(np.float32), paths=None, anc=None, bias_start=None,
             bias_token=None, bias=None, mask=None)
    c["logits"] = torch.from_numpy(rng.standard_normal((T, V)).astype(np.float32) * 4).to(dtype).to(DEV)
    c["paths"], words = [], []
    for b, n in enumerate(counts):
        par = parents[start[b]:start[b] + n]
        c["paths"] += [ora_tree.line_of(par, i) for i in range(n)]
        words.append(ora_tree.ancestor_words(par, max_nodes))
    if kind != "chain":
        c["anc"] = np.concatenate(words).view(np.int64)
    if bias:
        c["bias_start"] = np.array([b * bias for b in range(B + 1)], np.int32)
        c["bias_token"] = zipf(B * bias)
        c["bias"] = rng.standard_normal(B * bias).astype(np.float32)
    if mask:
        c["mask"] = rng.integers(-2 ** 31, 2 ** 31, (T, (V + 31) // 32)).astype(np.int32)
    return c


def run(c, **kw):
    put = lambda a: None if a is None else dev(a)  # noqa: E731
    err = word()
    out = serving.specverify_penalize(
        c["logits"], dev(c["tokens"]), dev(c["start"]), dev(c["history"]), dev(c["prefix"]), dev(c["prompt"]),
        dev(c["rep"]), dev(c["pres"]), dev(c["freq"]), ancestors=put(c["anc"]), max_nodes=c["max_nodes"],
        bias_start=put(c["bias_start"]), bias_token=put(c["bias_token"]), bias=put(c["bias"]),
        mask=put(c["mask"]), device_error=err, **kw)
    torch.cuda.synchronize()
    return out, int(err.item())


def reference(c):
    return ora.penalize(host64(c["logits"]), c["tokens"], c["start"], c["history"], c["prefix"], c["prompt"],
                        c["rep"], c["pres"], c["freq"], paths=c["paths"], max_nodes=c["max_nodes"],
                        bias_start=c["bias_start"], bias_token=c["bias_token"], bias=c["bias"], mask=c["mask"])


def check(c, error=0, out=None, **kw):
    if out is None:
        out = torch.full(c["logits"].shape, 77.0, dtype=c["logits"].dtype, device=DEV)
    ref, size, written, err = reference(c)
    assert err == error, err
    got, got_err = run(c, out=out, **kw)
    assert got_err == error, got_err
    x = host64(got)
    assert np.all(x[~written] == 77.0)
    x, ref, size = x[written], ref[written], size[written]
    assert np.array_equal(np.isnan(x), np.isnan(ref))
    fin = np.isfinite(ref)
    assert np.array_equal(x[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)])
    e = HALF_STEP[got.dtype]
    tol = 9 * F * size + e * np.abs(np.where(fin, ref, 0)) * (1 + 1e-6) + 1e-37
    bad = np.abs(np.where(fin, x - ref, 0)) > tol
    assert not bad.any(), (np.argwhere(bad)[:5].tolist(), np.abs(np.where(fin, x - ref, 0)).max())
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 7, 31, 4096, 4097, 32001, 50000])
def test_vocabularies_and_types(dtype, out_dtype, V):
    c = case(V, [3, 1, 5], V, [40, 0, 200], dtype=dtype, bias=4 if V > 300 else 0, mask=True)
    check(c, out=torch.full((9, V), 77.0, dtype=out_dtype, device=DEV))


@pytest.mark.parametrize("kind,counts", [("chain", [1]), ("chain", [9] * 7), ("random", [40, 1, 128]),
                                         ("branches", [33, 33, 0, 5]), ("star", [65, 128]), ("chain", [128, 64, 65])])
def test_trees(kind, counts):
    rng = np.random.default_rng(len(counts))
    check(case(sum(counts), counts, 9000, [int(x) for x in rng.integers(0, 300, len(counts))], kind=kind,
               max_nodes=128))


@pytest.mark.parametrize("length", [0, 1, 511, 512, 513, 2047, 2048, 2049, 20000])
def test_histories(length):
    check(case(length, [2, 3], 6000, [length, 5], dtype=torch.bfloat16))


def test_the_same_tokens_again_and_again():
    # one id emitted throughout, in the history, on the path and in the biases
    c = case(1, [9], 5000, [300], bias=4)
    c["history"][:], c["tokens"][:], c["bias_token"][:] = 4999, 4999, 4999
    got = check(c)
    assert torch.equal(got[:, :4999], c["logits"][:, :4999])


def test_more_biases_than_threads():
    c = case(2, [2, 2], 5000, [30, 40], bias=1500)
    # every id a few times at most: the tolerance counts four
    rng = np.random.default_rng(0)
    c["bias_token"] = np.concatenate([rng.permutation(np.repeat(np.arange(375) * 13, 4)) for _ in "ab"]).astype(np.int32)
    check(c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_in_place(dtype):
    c = case(3, [9, 4], 33000, [500, 60], dtype=dtype, bias=7, mask=True)
    want = check(c)
    got, _ = run(c, out=c["logits"])
    assert got is c["logits"] and torch.equal(got, want)


def test_masked_logits_and_masks_that_leave_nothing():
    c = case(4, [4], 5000, [50], mask=True)
    low = torch.finfo(torch.float32).min
    c["logits"][0, ::3] = -float("inf")
    c["logits"][1, ::3] = low
    c["mask"][2] = 0
    c["rep"][:] = 0.9  # a lowest value times less than 1 stays finite
    got = check(c)
    assert torch.all(torch.isneginf(got[2]))


def test_infinities_and_nan_stay_where_they_are():
    c = case(5, [2], 5000, [30])
    c["logits"][0, 17], c["logits"][0, 4097] = float("inf"), float("nan")
    out, err = run(c)
    assert err == 0 and torch.isposinf(out[0, 17]) and torch.isnan(out[0, 4097])
    assert torch.isfinite(out).sum() == out.numel() - 2


def test_none_of_it_leaves_the_logits_as_they_are():
    c = case(6, [9, 2], 40000, [400, 3], dtype=torch.bfloat16)
    c["rep"][:], c["pres"][:], c["freq"][:] = 1.0, 0.0, 0.0
    assert torch.equal(run(c)[0], c["logits"])


def test_strides():
    c = case(7, [3, 2], 5003, [70, 9], bias=3, mask=True)
    want = check(c)
    wide = torch.zeros((5, 5101), device=DEV)
    wide[:, 3:5006] = c["logits"]  # rows that begin anywhere: element accesses
    history = np.full((2, 100), -5, np.int32)
    history[:, :70] = c["history"]
    mask = np.zeros((5, 200), np.int32)
    mask[:, :157] = c["mask"]
    out = torch.full((5, 6000), 77.0, device=DEV)
    put = {k: dev(c[k]) for k in ("tokens", "start", "prefix", "prompt", "rep", "pres", "freq", "bias_start", "bias_token", "bias")}
    got = serving.specverify_penalize(
        wide[:, 3:5006], put["tokens"], put["start"], dev(history)[:, :70], put["prefix"], put["prompt"],
        put["rep"], put["pres"], put["freq"], max_nodes=3, bias_start=put["bias_start"], bias_token=put["bias_token"],
        bias=put["bias"], mask=dev(mask)[:, :157], out=out[:, :5003])
    assert torch.equal(got, want) and torch.all(out[:, 5003:] == 77.0)
    # one row of logits for all nodes
    one = dict(c, logits=c["logits"][:1].expand(5, -1))
    a, _ = run(one)
    b, _ = run(dict(one, logits=one["logits"].contiguous()))
    assert torch.equal(a, b)


def test_wrong_data():
    c = case(8, [3, 2, 4], 5000, [50, 60, 70], bias=2)
    check(dict(c, tokens=np.where(np.arange(9) % 4 == 1, 5000, c["tokens"])), error=1)
    check(dict(c, history=np.where(np.arange(70) % 9 == 1, -1, c["history"]).astype(np.int32)), error=1)
    check(dict(c, bias_token=np.array([0, 1, -1, 5, 9 ** 9, 7], np.int32)), error=1)
    check(dict(c, prefix=np.array([50, 71, 70], np.int32)), error=64)
    check(dict(c, prefix=np.array([50, -1, 70], np.int32)), error=64)
    check(dict(c, prompt=np.array([50, 20, 99], np.int32)), error=64)
    check(dict(c, rep=np.array([1.0, 0.0, 2.0], np.float32)), error=256)
    check(dict(c, rep=np.array([np.nan, 1.0, -2.0], np.float32)), error=256)
    check(dict(c, bias_start=np.array([0, 2, 1, 6], np.int32)), error=64)
    check(dict(c, bias_start=np.array([0, 2, 4, 7], np.int32)), error=64)
    check(dict(c, start=np.array([0, 3, 2, 9], np.int32)), error=8)
    check(dict(c, start=np.array([0, 3, 5, 10], np.int32)), error=8)


def test_rows_behind_the_last_request_are_left_as_they_were():
    c = case(9, [3, 2], 5000, [50, 60])
    c["logits"] = torch.cat([c["logits"], c["logits"][:2]])
    c["tokens"] = np.concatenate([c["tokens"], [0, 0]]).astype(np.int32)
    c["paths"] += [[], []]
    check(c)


def test_a_verification_of_penalized_logits():
    # a banned id is never emitted, and an allowed one alone always
    B, g, V = 4, 3, 33000
    c = case(10, [g + 1] * B, V, [60] * B, mask=True)
    c["mask"][:] = 0
    only = np.array([3, 4097, 32999, 20])
    for b in range(B):
        c["mask"][b * (g + 1):(b + 1) * (g + 1), only[b] // 32] = np.int32(np.uint32(1 << (only[b] % 32)).view(np.int32))
    x, err = run(c)
    assert err == 0
    draft = torch.randn((B, 1, g, V), device=DEV)
    tokens = torch.randint(0, V, (B, 1, g), device=DEV, dtype=torch.int32)
    tokens[0, 0, 0] = 3
    o = sv.specverify_step(x.view(B, g + 1, V), draft, tokens, torch.ones(B, device=DEV), 7)
    assert o.out_token[:, 0].tolist() == only.tolist() and int(o.device_error.item()) == 0


@pytest.mark.parametrize("wrong", ["bias", "out", "logits", "history", "mask", "type"])
def test_refusals(wrong):
    c = case(11, [3, 2], 5000, [50, 60], bias=2, mask=True)
    out = None
    if wrong == "bias":
        c["bias_token"] = None
    elif wrong == "out":
        out = torch.zeros((1, 5000), device=DEV).expand(5, -1)
    elif wrong == "logits":
        c["logits"] = c["logits"].half()
    elif wrong == "history":
        c["history"] = c["history"].astype(np.int64)
    elif wrong == "mask":
        c["mask"] = c["mask"][:, 1:]
    else:
        c["rep"] = c["rep"].astype(np.float64)
    with pytest.raises(sv.SpecVerifyError):
        run(c, out=out)
