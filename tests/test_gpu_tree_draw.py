"""GPU: the token that verification draws where a row's weights are few and lie far apart, at the
ends of the uniform's range and at the borders between tokens, against the oracle.

The kernel's running sums are taken by chunk of ids and then by a doubling scan over the chunks, so
neighbouring ones may differ in their last bit although no weight lies between them; the drawn token
has to have a weight all the same."""
from __future__ import annotations

import numpy as np
import pytest

import test_gpu_tree_verify as ver
from oracle import tree as ora

pytestmark = pytest.mark.gpu

LAST = 1.0 - 2.0 ** -53


def stars(seed, B, V, support, kids, mode, dtype="f32"):
    """Requests of a root and `kids` children of one token that the target cannot emit: all are
    rejected, and what is left is a residual on `support` ids that needs all of a double's bits."""
    rng = np.random.default_rng(seed)
    n = kids + 1
    T = B * n
    target, draft = np.zeros((T, V), dtype=np.float32), np.zeros((T, V), dtype=np.float32)
    tokens = np.zeros(T, dtype=np.int32)
    for b in range(B):
        ids = rng.choice(V, support + 1, replace=False)
        tokens[b * n:(b + 1) * n] = ids[support]
        z = rng.standard_normal(support) * 1.5
        p, q = np.exp(z), np.exp(z * 0.8 + rng.standard_normal(support) * 0.7)
        target[b * n, ids[:support]] = p / p.sum()
        draft[b * n, ids[:support]] = 0.98 * q / q.sum()
        draft[b * n, ids[support]] = 0.02
    if dtype == "bf16":
        import torch
        target, draft = (torch.from_numpy(x).bfloat16().float().numpy() for x in (target, draft))
    return dict(target=target, draft=None if mode == ora.FIXED else draft, tokens=tokens,
                parents=np.tile([-1] + [0] * kids, B).astype(np.int32),
                node_start=(np.arange(B + 1) * n).astype(np.int32), u=np.full(T, 0.5),
                r=np.full(B, LAST), mode=mode, max_nodes=n, max_path=n, dtype=dtype)


# 32 chunks of 4096 ids, by 8 workgroups a request and by one; the last has more chunks than the
# wavefront that adds them up has lanes
@pytest.mark.parametrize("mode", [ora.IID, ora.DISTINCT])
@pytest.mark.parametrize("B,V,support,dtype", [
    (64, 128256, 20, "f32"), (64, 128256, 60, "f32"), (64, 128256, 20, "bf16"),
    (300, 40000, 12, "f32"), (4, 600000, 30, "f32")])
def test_the_last_uniform_draws_a_token_with_a_weight(mode, B, V, support, dtype):
    c = stars(B + support + mode, B, V, support, 2, mode, dtype)
    got, ref = ver.run(c), ver.reference(c)
    assert got["error"] == 0 and ref["error"] == 0
    assert np.all(got["out_token"] >= 0)
    assert np.all(c["target"][c["node_start"][:-1], got["out_token"]] > 0)
    assert np.array_equal(got["emitted"][:, 0], got["out_token"])
    assert np.array_equal(got["out_token"], ref["out_token"])


@pytest.mark.parametrize("stride", [None, 128261])
@pytest.mark.parametrize("B", [6, 300])
def test_borders_between_far_tokens(B, stride):
    # weights of a 64th each: every running sum is exact, so the border is met bit by bit
    V, eps = 128256, 2.0 ** -53
    rng = np.random.default_rng(B)
    target = np.zeros((B, V), dtype=np.float32)
    r, want = np.zeros(B), np.zeros(B, dtype=np.int64)
    for b in range(B):
        ids = np.sort(rng.choice(V, 64, replace=False))
        target[b, ids] = 2.0 ** -6
        k = int(rng.integers(0, 64))
        low = bool(rng.integers(0, 2)) and k > 0
        r[b] = k / 64.0 - (eps if low else 0.0)
        want[b] = ids[k - 1 if low else k]
    c = dict(target=target, draft=None, tokens=np.zeros(B, dtype=np.int32),
             parents=np.full(B, -1, dtype=np.int32), node_start=np.arange(B + 1, dtype=np.int32),
             u=np.zeros(B), r=r, mode=ora.FIXED, max_nodes=1, max_path=1, dtype="f32")
    assert np.array_equal(ver.check(c, stride=stride)["out_token"], want)
