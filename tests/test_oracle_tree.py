"""Pins of the oracle of the operators on drafted token trees: hand-worked cases, and the law of
verification (what is emitted first follows the target's distribution, whatever the draft)."""
import numpy as np
import pytest

from oracle import tree as ora


def test_ancestors_of_a_small_tree():
    # 0 - (1 - 3, 2 - (4, 5))
    assert ora.ancestor_words([-1, 0, 0, 1, 2, 2], 6)[:, 0].tolist() == [1, 3, 5, 11, 21, 37]
    far = ora.ancestor_words(list(range(-1, 69)), 70)
    assert far[69].tolist() == [2 ** 64 - 1, 2 ** 6 - 1]


def test_plan_by_hand():
    # pages of 4; request 0 holds 6 tokens in 2 pages and wants 3 more (one page), request 1 is new
    p = ora.plan([-1, 0, 0, -1], [0, 3, 4], [6, 0], [2, 0], [[5, 1, -1], [-1, -1, -1]], [7, 3, 9], 0,
                 page_size=4, num_pages=10, max_nodes=3, max_path=3)
    assert p["block_table"].tolist() == [[5, 1, 7], [3, -1, -1]]
    assert p["pages"].tolist() == [3, 1] and p["free_head"] == 2 and p["error"] == 0
    assert p["slots"].tolist() == [[6, 7, 28], [12, -1, -1]]
    assert p["position"].tolist() == [6, 7, 7, 0] and p["depth"].tolist() == [0, 1, 1, 0]


def test_attention_of_one_key_and_of_two():
    q = np.ones((2, 1, 2))
    k = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])
    v = np.array([[[1.0, 2.0]], [[3.0, 6.0]]])
    cache = np.zeros((1, 4, 1, 2))
    out, lse, _, _ = ora.attention(q, k, v, cache, cache, np.array([[0]]), [0], [0, 2], None,
                                   max_nodes=2, scale=1.0)
    assert np.allclose(out[:, 0], [[1, 2], [2, 4]]) and np.allclose(lse[:, 0], [1, 1 + np.log(2)])


@pytest.mark.parametrize("mode", [ora.FIXED, ora.IID, ora.DISTINCT])
def test_the_first_token_follows_the_target(mode):
    # a root with three children on 5 tokens, one distribution for every node: 40000 draws of the
    # children and of the uniforms; each frequency lies within 4.5 standard deviations
    rng = np.random.default_rng(7 + mode)
    V, n, kids = 5, 40000, 3
    p = np.array([0.4, 0.3, 0.15, 0.1, 0.05])
    q = np.array([0.1, 0.2, 0.3, 0.15, 0.25])
    B = n
    if mode == ora.IID:
        children = rng.choice(V, size=(B, kids), p=q)
    elif mode == ora.DISTINCT:
        children = np.argsort(-(np.log(q) + rng.gumbel(size=(B, V))), axis=1)[:, :kids]
    else:
        children = np.tile([2, 0, 2], (B, 1))
    tokens = np.concatenate([np.zeros((B, 1), dtype=np.int64), children], axis=1).reshape(-1)
    parents = np.tile([-1, 0, 0, 0], B)
    start = np.arange(B + 1) * 4
    target = np.broadcast_to(p, (4 * B, V))
    draft = np.broadcast_to(q, (4 * B, V))
    o = ora.verify(target, draft, tokens, parents, start, rng.random(4 * B), rng.random(B), mode=mode,
                   max_nodes=4, max_path=2)
    first = o["emitted"][:, 0]
    share = np.bincount(first, minlength=V) / n
    assert o["error"] == 0
    assert np.all(np.abs(share - p) < 4.5 * np.sqrt(p * (1 - p) / n)), share


def test_commit_by_hand():
    k = np.arange(6.0).reshape(1, 3, 1, 2)
    cache = np.zeros((1, 2, 2, 1, 2))
    kc, vc, length, err = ora.commit(k, -k, cache, cache, [0, 3], np.array([[0, 2, -1]]), [1],
                                     np.array([[3, 0, -1]]), [5], max_nodes=3)
    assert kc[0].reshape(4, 2).tolist() == [[4, 5], [0, 0], [0, 0], [0, 1]]
    assert vc[0].reshape(4, 2).tolist() == [[-4, -5], [0, 0], [0, 0], [0, -1]]
    assert length.tolist() == [7] and err == 0
