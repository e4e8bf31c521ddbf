"""The oracle of the operators around a verification step against closed forms and library routines."""
import numpy as np
import pytest
import torch

from oracle import serving as ora


def test_attention_of_a_chunk_is_causal_softmax():
    g = torch.Generator().manual_seed(0)
    n, old, Hq, Hkv, D = 5, 6, 4, 2, 8
    k, v = torch.randn((2, 1, 16, Hkv, D), generator=g, dtype=torch.float64)
    q = torch.randn((n, Hq, D), generator=g, dtype=torch.float64)
    out, lse, weight, _ = ora.attention(q.numpy(), k.numpy(), v.numpy(), np.zeros((1, 1), int), [old], [0, n],
                                        max_chunk=n, scale=D ** -0.5)
    keys, values = (x[0, :old + n].repeat_interleave(2, 1).transpose(0, 1) for x in (k, v))
    z = q.transpose(0, 1) @ keys.transpose(1, 2) * D ** -0.5
    z.masked_fill_(torch.arange(old + n) > old + torch.arange(n)[:, None], -float("inf"))
    want = (torch.softmax(z, -1) @ values).transpose(0, 1)
    assert np.allclose(out, want.numpy(), atol=1e-13)
    assert np.allclose(lse, torch.logsumexp(z, -1).T.numpy(), atol=1e-13)
    assert np.all(weight >= np.abs(out) - 1e-13)


def test_rotation_keeps_distances_and_depends_on_the_difference_of_positions():
    rng = np.random.default_rng(0)
    freq = (100.0 ** (-np.arange(4) / 4)).astype(np.float32)
    a, b = rng.standard_normal((2, 1, 1, 8))
    for inter in (False, True):
        turn = lambda x, p: ora.rotate(x, None, [p], freq, eps=0.0, interleaved=inter)[0][0, 0]  # noqa: E731
        assert np.isclose(np.linalg.norm(turn(a, 1000)), np.linalg.norm(a))
        assert np.isclose(turn(a, 1005) @ turn(b, 1002), turn(a, 5) @ turn(b, 2))
        assert np.allclose(turn(a, 0), a[0, 0])


def test_norm_is_rms():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    y, _ = ora.rotate(x, np.array([1.0, 2.0, 1.0, 1.0]), [0], np.ones(1, np.float32), eps=0.0, interleaved=False)
    assert np.allclose(y, [[[1.2, 3.2, 0.0, 0.0]]])


def test_penalties_by_hand():
    logits = np.array([[2.0, -2.0, 1.0, 0.5], [2.0, -2.0, 1.0, 0.5]])
    out, _, written, err = ora.penalize(
        logits, np.array([1, 3]), [0, 2], np.array([[0, 2, 2]]), [3], [1], [2.0], [0.25], [0.1],
        paths=[[0], [0, 1]], max_nodes=2, bias_start=[0, 2], bias_token=[2, 2], bias=[1.0, 0.5],
        mask=np.array([[0b0111], [0b1111]], np.int32))
    # 0 in the prompt alone: halved; 1 the root's token: doubled, once; 2 emitted twice, biases 1.5
    assert np.allclose(out[0], [1.0, -4.35, 0.5 - 0.45 + 1.5, -np.inf])
    assert np.allclose(out[1], [1.0, -4.35, 0.5 - 0.45 + 1.5, 0.25 - 0.35])
    assert written.all() and err == 0


def test_pages_come_free_with_their_last_holder_and_in_order_of_ids():
    table = [[5, 3, 1], [5, 3, 0]]
    o = ora.resize([0, 24], [3, 3], table, [-1] * 5 + [2, 4], 5, page_size=8, num_pages=7, chunk_start=[0, 0, 2], rows=2,
                   shares=[0, 0, 0, 1, 0, 1, 0])
    # request 0 gives 5, 3, 1 back, of which 1 comes free and is taken again by request 1
    assert o["block_table"][1].tolist() == [5, 3, 0] or o["error"]
    assert o["shares"].tolist() == [0] * 7
    wide = [r + [-1] for r in table]
    o = ora.resize([0, 24], [3, 3], wide, [-1] * 5 + [2, 4], 5, page_size=8, num_pages=7, chunk_start=[0, 0, 2], rows=2,
                   shares=[0, 0, 0, 1, 0, 1, 0])
    assert o["block_table"][1].tolist() == [5, 3, 0, 1] and o["free_head"] == 5 and o["error"] == 0
    assert o["slots"].tolist() == [8, 9] and o["position"].tolist() == [24, 25] and o["pages"].tolist() == [0, 4]


def test_a_fork_shares_full_pages_and_copies_the_last():
    k = np.arange(4 * 2, dtype=np.float64).reshape(1, 4, 2, 1, 1)
    o = ora.fork([0], [1], [3, 0], [2, 0], [[2, 0], [-1, -1]], [3], 0, [0] * 4, k, -k, num_pages=4)
    assert o["block_table"].tolist() == [[2, 0], [2, 3]] and o["shares"].tolist() == [0, 0, 1, 0]
    assert o["k_cache"][0, 3, :, 0, 0].tolist() == [0.0, 7.0] and o["v_cache"][0, 3, 0, 0, 0] == 0.0
    assert o["prefix_len"].tolist() == [3, 3] and o["pages"].tolist() == [2, 2] and o["free_head"] == 1


@pytest.mark.parametrize("pair", [(0, 0), (0, 5), (-1, 1), (0, 2)])
def test_forks_that_may_not_be(pair):
    k = np.zeros((1, 4, 2, 1, 1))
    o = ora.fork([pair[0]], [pair[1]], [2, 0, 2], [1, 0, 1], [[2], [-1], [0]], [3], 0, [0] * 4, k, k, num_pages=4)
    assert o["error"] == ora.ERR_REQUEST and o["prefix_len"].tolist() == [2, 0, 2]
