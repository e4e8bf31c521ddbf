"""GPU: calls of more workgroups than one dimension of a grid takes, and rotations of many tokens with few heads."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from device_draft_verification_specverify_amd import serving
from oracle import serving as ora
from test_gpu_serving_rotate import case as rotate_case, hold, want_of
from tree_helpers import DEV, host64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,Hq,Hkv", [((1 << 24) + 7, 1, 1), ((1 << 22) + 5, 31, 1)])
def test_rotations_of_millions_of_tokens(T, Hq, Hkv):
    g = torch.Generator(device=DEV).manual_seed(T)
    q = torch.randn((T, Hq, 8), generator=g, device=DEV, dtype=torch.float16)
    k = torch.randn((T, Hkv, 8), generator=g, device=DEV, dtype=torch.float16)
    freq = torch.tensor([1.0, 0.25, 0.01, 0.001], device=DEV)
    position = torch.arange(T, dtype=torch.int32, device=DEV) % 131072
    q_out = torch.full_like(q, float("nan"))
    k_out = torch.full_like(k, float("nan"))
    serving.specverify_rotate(q, k, None, position, freq, out_q=q_out, out_k=k_out)
    assert not torch.isnan(q_out).any() and not torch.isnan(k_out).any()
    some = torch.tensor([0, 1, T // 2, (1 << 22) - 1, 1 << 22, (1 << 22) + 1, T - 4, T - 1], device=DEV)
    for x, y in ((q, q_out), (k, k_out)):
        want = ora.rotate(host64(x[some]), None, host64(position[some]), freq.cpu().numpy(), eps=1e-6, interleaved=False)
        hold(y[some], *want)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 63, 401])
@pytest.mark.parametrize("Hq,Hkv,D,R", [(8, 1, 64, 64), (8, 1, 64, 20), (1, 1, 256, 250), (2, 2, 80, 80), (14, 1, 128, 128),
                                        (15, 1, 128, 6), (3, 2, 8, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_few_heads(T, Hq, Hkv, D, R, interleaved):
    c = rotate_case(T + D, T, Hq, Hkv, D, R, torch.bfloat16, first=50)
    c["position"][T // 2] = -1
    q_out = torch.full_like(c["q"], 7.0)
    k_cache, v_cache = (torch.full((T + 1, 1, Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    slots = torch.arange(T, device=DEV)
    slots[T // 3] = -1
    serving.specverify_rotate(**c, interleaved=interleaved, out_q=q_out, slots=slots, k_cache=k_cache, v_cache=v_cache)
    there = torch.arange(T, device=DEV) != T // 2
    stored = there & (slots >= 0)
    (q, q_size), (k, k_size) = want_of(c, "q", interleaved), want_of(c, "k", interleaved)
    at, kept = there.cpu().numpy(), stored.cpu().numpy()
    hold(q_out[there], q[at], q_size[at])
    hold(k_cache[:T, 0][stored], k[kept], k_size[kept])
    assert torch.equal(v_cache[:T, 0][stored], c["v"][stored])
    assert torch.all(q_out[~there] == 7.0) and torch.all(k_cache[:T][~stored] == 7.0) and torch.all(v_cache[:T][~stored] == 7.0)
    assert torch.all(k_cache[T] == 7.0) and torch.all(v_cache[T] == 7.0)


def test_penalties_of_many_requests():
    B, V = 90000, 200000
    rows = [0, 45001, B - 1]
    start = np.searchsorted(rows, np.arange(B + 1)).astype(np.int32)
    rng = np.random.default_rng(0)
    put = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    logits = torch.from_numpy(rng.standard_normal((3, V)).astype(np.float32)).to(DEV)
    history = rng.integers(0, V, (B, 2)).astype(np.int32)
    tokens = rng.integers(0, V, 3).astype(np.int32)
    twos, ones = np.full(B, 2, np.int32), np.ones(B, np.int32)
    half, nothing = np.full(B, 0.5, np.float32), np.zeros(B, np.float32)
    out = serving.specverify_penalize(logits, put(tokens), put(start), put(history), put(twos), put(ones), put(half),
                                      put(half), put(nothing), max_nodes=1)
    want = logits.clone()
    for r, b in enumerate(rows):  # halves are exact, and so are differences of one
        for v, emitted in {int(history[b, 0]): False, int(history[b, 1]): True, int(tokens[r]): True}.items():
            x = float(logits[r, v])
            want[r, v] = float(np.float32(x * 2 if x > 0 else x / 2) - np.float32(0.5 if emitted else 0))
    assert torch.equal(out, want)


def test_forks_of_many_layers():
    forks, layers, page = 65535, 65, 2
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    k = torch.zeros((layers, forks + 1, page, 1, 8), dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    k[:, 0] = torch.arange(1, layers + 1, dtype=torch.float16, device=DEV).view(-1, 1, 1, 1)
    v[:, 0] = -k[:, 0]
    table = torch.full((forks + 1, 1), -1, dtype=torch.int32, device=DEV)
    table[0] = 0
    one = torch.zeros(forks + 1, dtype=torch.int32, device=DEV)
    one[0] = 1
    o = serving.specverify_pages_fork(torch.zeros(forks, dtype=torch.int32, device=DEV), i32(range(1, forks + 1)), one, one.clone(), table,
                                      i32(range(1, forks + 1)), i32([0]), one.clone(), k, v)
    assert torch.all(o.prefix_len == 1) and torch.all(o.pages == 1) and int(o.free_head) == forks
    assert torch.equal(table[:, 0], torch.arange(forks + 1, dtype=torch.int32, device=DEV))
    assert torch.equal(k[:, 1:, 0], k[:, :1, 0].expand(layers, forks, 1, 8))
    assert torch.equal(v[:, 1:, 0], v[:, :1, 0].expand(layers, forks, 1, 8))
    assert not k[:, 1:, 1].any()
