"""GPU: norms and rotation of queries and keys, and their way into the cache, against the oracle in
float64.

Tolerance, from the arithmetic (f = 2^-24, e half a step of the type): the sum of squares of a head in
float32, 14 f, mean, root and quotient 4 f, two products 2 f: a normed element is off by 16 f of itself;
the angle is rounded to float32 in half turns, pi f, and cos and sin are off by 2 f more; two products and
a sum 3 f: 16 + 4 + 2 + 3 < 32 f of |a| + |b|, and e |y| of the result. At positions near 2^31 the float64
angle itself is off by 2^-22 = 4 f in the kernel, once more by the factor 1 / 2 pi, and the same in the
oracle: 64 f.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import device_draft_verification_specverify_amd as sv
from device_draft_verification_specverify_amd import serving
from oracle import serving as ora
from serving_helpers import F, HALF_STEP, laid_out, word
from tree_helpers import DEV, dev, host64

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def case(seed, T, Hq, Hkv, D, R, dtype, *, norm="type", first=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn((T, Hq + 2 * Hkv, D), generator=g) * scale).to(dtype).to(DEV)
    q, k, v = qkv.split([Hq, Hkv, Hkv], dim=1)
    weights = [None, None]
    if norm:
        weights = [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype if norm == "type" else torch.float32).to(DEV)
                   for _ in "qk"]
    freq = (10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) / (R // 2))).float()
    position = (first + torch.randperm(T, generator=g)).int()
    return dict(q=q, k=k, v=v, position=position.to(DEV), inv_freq=freq.to(DEV), q_weight=weights[0],
                k_weight=weights[1])


def want_of(c, name, interleaved, eps=1e-6):
    w = c[name + "_weight"]
    return ora.rotate(host64(c[name]), None if w is None else host64(w), host64(c["position"]),
                      c["inv_freq"].cpu().numpy(), eps=eps, interleaved=interleaved)


def hold(got, want, size, factor=32):
    e = HALF_STEP[got.dtype]
    y = host64(got)
    there = ~np.isnan(want)
    tol = factor * F * size * (1 + e) + e * np.abs(want) + torch.finfo(got.dtype).smallest_normal * e
    bad = np.abs(y - want)[there] > tol[there]
    assert not bad.any(), (np.argwhere(there)[bad][:5].tolist(), np.abs(y - want)[there].max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(8, 8), (8, 2), (64, 64), (80, 80), (80, 20), (128, 128), (128, 64),
                                 (128, 6), (200, 200), (200, 144), (256, 256), (256, 250)])
def test_widths(dtype, interleaved, D, R):
    c = case(D + R, 7, 5, 2, D, R, dtype)
    q, k = serving.specverify_rotate(**dict(c, v=None), interleaved=interleaved)
    hold(q, *want_of(c, "q", interleaved))
    hold(k, *want_of(c, "k", interleaved))


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 32, 8), (1, 1, 1), (9, 21, 3), (3, 100, 1), (130, 8, 8)])
@pytest.mark.parametrize("norm", [None, "type", "float32"])
def test_heads_and_norms(T, Hq, Hkv, norm):
    c = case(T + Hq, T, Hq, Hkv, 128, 128, torch.bfloat16, norm=norm, scale=3.0)
    q, k = serving.specverify_rotate(**dict(c, v=None), eps=0.01)
    hold(q, *want_of(c, "q", False, 0.01))
    hold(k, *want_of(c, "k", False, 0.01))


@pytest.mark.parametrize("which", ["q_weight", "k_weight"])
def test_a_norm_of_one_of_them(which):
    c = case(3, 5, 4, 2, 64, 64, torch.float16)
    c[which] = None
    q, k = serving.specverify_rotate(**dict(c, v=None))
    hold(q, *want_of(c, "q", False))
    hold(k, *want_of(c, "k", False))


@pytest.mark.parametrize("first,factor", [(131072, 32), (10 ** 7, 32), (2 ** 31 - 40, 64)])
def test_far_positions(first, factor):
    c = case(5, 33, 2, 1, 128, 128, torch.float32, first=first)
    q, k = serving.specverify_rotate(**dict(c, v=None))
    hold(q, *want_of(c, "q", False), factor)
    hold(k, *want_of(c, "k", False), factor)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("page,D,R", [(1, 64, 64), (16, 128, 128), (64, 80, 20)])
def test_into_the_cache(dtype, layout, page, D, R):
    T, Hkv = 37, 3
    c = case(page + D, T, 6, Hkv, D, R, dtype, first=100)
    pages = -(-T // page) + 3
    g = torch.Generator().manual_seed(page)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[[4, 9]] = -1
    caches = [laid_out(torch.randn((pages, page, Hkv, D), generator=g).to(dtype).to(DEV), layout) for _ in "kv"]
    before = [t.clone() for t in caches]
    q, none = serving.specverify_rotate(**c, slots=slots.to(DEV), k_cache=caches[0], v_cache=caches[1])
    assert none is None
    q2, k2 = serving.specverify_rotate(**dict(c, v=None))
    assert torch.equal(q, q2)
    for t in range(T):
        if slots[t] >= 0:
            before[0][slots[t] // page, slots[t] % page] = k2[t]
            before[1][slots[t] // page, slots[t] % page] = c["v"][t]
    assert torch.equal(caches[0], before[0]) and torch.equal(caches[1], before[1])
    # and beside it, where it is asked for
    out_k = torch.zeros_like(c["k"])
    _, k3 = serving.specverify_rotate(**c, slots=slots.to(DEV), k_cache=caches[0], v_cache=caches[1], out_k=out_k)
    assert k3 is out_k and torch.equal(k3, k2)


@pytest.mark.parametrize("D,R,interleaved", [(128, 128, False), (80, 20, False), (64, 64, True)])
def test_in_place(D, R, interleaved):
    c = case(D, 50, 9, 3, D, R, torch.bfloat16)
    q, k = serving.specverify_rotate(**dict(c, v=None), interleaved=interleaved)
    v = c["v"].clone()
    q2, k2 = serving.specverify_rotate(**dict(c, v=None), interleaved=interleaved, out_q=c["q"], out_k=c["k"])
    assert q2 is c["q"] and torch.equal(q2, q) and torch.equal(k2, k) and torch.equal(c["v"], v)


def test_rows_of_negative_positions_are_passed_by():
    c = case(7, 12, 4, 2, 64, 64, torch.bfloat16)
    c["position"][3] = -1
    c["position"][8] = -2 ** 31
    out_q, out_k = torch.full_like(c["q"], 7.0), torch.full_like(c["k"], 7.0)
    caches = [torch.full((2, 16, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    slots = torch.arange(12, device=DEV)
    serving.specverify_rotate(**c, out_q=out_q, out_k=out_k, slots=slots, k_cache=caches[0], v_cache=caches[1])
    for t in (3, 8):
        for x in (out_q[t], out_k[t], caches[0][0, t], caches[1][0, t]):
            assert torch.all(x == 7.0)
    hold(out_q, *want_of(c, "q", False))
    hold(out_k, *want_of(c, "k", False))


def test_slots_outside_the_cache_store_nothing():
    c = case(8, 6, 4, 2, 64, 64, torch.float32)
    caches = [torch.full((3, 16, 2, 64), 7.0, device=DEV) for _ in "kv"]
    slots = dev(np.array([0, 48, -2, 2 ** 62, -2 ** 62, 5], dtype=np.int64))
    err = word()
    q, _ = serving.specverify_rotate(**c, slots=slots, k_cache=caches[0], v_cache=caches[1], device_error=err)
    assert int(err.item()) == 16
    hold(q, *want_of(c, "q", False))
    flat = caches[0].flatten(0, 1)
    assert torch.all(flat[[i for i in range(48) if i not in (0, 5)]] == 7.0) and not torch.any(flat[0] == 7.0)
    err.zero_()
    serving.specverify_rotate(**c, slots=torch.full((6,), -1, device=DEV), k_cache=caches[0],
                              v_cache=caches[1], device_error=err)
    assert int(err.item()) == 0


def test_strided_and_broadcast_inputs():
    c = case(9, 10, 6, 6, 64, 64, torch.float16)
    q = torch.empty((6, 10, 64), dtype=torch.float16, device=DEV).transpose(0, 1)
    q.copy_(c["q"])
    one = dict(c, q=q, k=c["k"][:, :1].expand(-1, 6, -1), v=None)
    out = torch.full((10, 6, 96), float("nan"), dtype=torch.float16, device=DEV)
    got_q, got_k = serving.specverify_rotate(**one, out_q=out[:, :, :64])
    want_q, _ = serving.specverify_rotate(**dict(c, v=None))
    assert torch.equal(got_q, want_q) and torch.isnan(out[:, :, 64:]).all()
    hold(got_k, *want_of(dict(c, k=one["k"]), "k", False))


def test_a_row_that_is_zero_and_one_that_is_not_finite():
    c = case(10, 4, 2, 2, 64, 64, torch.bfloat16)
    c["q"][1] = 0.0
    c["q"][2, 1, 5] = float("inf")
    q, k = serving.specverify_rotate(**dict(c, v=None))
    assert torch.all(q[1] == 0.0) and torch.isnan(q[2, 1]).any()
    others = [i for i in range(4) if i != 2]
    want, size = want_of(c, "q", False)
    hold(q[others], want[others], size[others])
    hold(q[2, :1][None], want[2, :1][None], size[2, :1][None])


def test_no_rows():
    c = case(11, 0, 4, 2, 64, 64, torch.bfloat16)
    q, k = serving.specverify_rotate(**dict(c, v=None))
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)


def test_gradients_are_not_recorded():
    c = case(12, 3, 4, 2, 64, 64, torch.float32)
    q, _ = serving.specverify_rotate(**dict(c, v=None))
    assert not q.requires_grad


@pytest.mark.parametrize("wrong", ["v", "slots", "out_q", "weight", "position", "odd"])
def test_refusals(wrong):
    c = case(13, 4, 4, 2, 64, 64, torch.bfloat16)
    cache = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    slots = torch.arange(4, device=DEV)
    kw = dict(c, k_cache=cache, v_cache=cache.clone(), slots=slots)
    if wrong == "v":
        kw["v"] = None
    elif wrong == "slots":
        kw["slots"] = None
    elif wrong == "out_q":
        kw["out_q"] = c["q"][:1].expand(4, -1, -1)
    elif wrong == "weight":
        kw["q_weight"] = kw["q_weight"].half()
    elif wrong == "position":
        kw["position"] = kw["position"].long()
    else:
        kw["inv_freq"] = torch.zeros(33, device=DEV)  # wider than the head
    with pytest.raises(sv.SpecVerifyError):
        serving.specverify_rotate(**kw)
