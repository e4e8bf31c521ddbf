"""GPU: infinite and NaN values of drafted nodes behind a prefix whose keys are shared out over
several workgroups. The rule is that of short prefixes: a row that does not see the node keeps its
bits, one that sees it gets the value in the columns where it lies, however small its weight."""
from __future__ import annotations

import pytest
import torch

import test_gpu_tree_attention as att

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("most,D", [(6, 64), (40, 128), (100, 64), (6, 256), (40, 256)])
@pytest.mark.parametrize("far", [False, True])
def test_wild_values_behind_a_split_prefix(what, most, D, far):
    c = att.case(most + D, [2500, 700], [most, 3], 4, 2, D, 16, kind="star")
    if far:
        # the prefix's first key scores 8 * 40 = 320 and the others a few: in float32 the share that
        # holds the nodes then weighs nothing beside the first one (e^-300)
        c["q"][:, :, 0] = 8.0
        for b in range(2):
            page = int(c["table"][b, 0])
            c["k_cache"][page, 0, :, 0] = 40.0 * D ** 0.5
    out, lse, _, _, _ = att.check(c)
    wild = most - 2
    others = [i for i in range(most + 3) if i != wild]
    cols = [d for d in range(D) if d != 5]
    c["v_tree"][wild, :, 5] = what
    got, got_lse, _ = att.run(c)
    assert torch.equal(got[others], out[others]) and torch.equal(got_lse, lse)
    assert torch.equal(got[wild][:, cols], out[wild][:, cols])
    x = got[wild][:, 5].float()
    assert torch.all(torch.isnan(x)) if what != what else torch.all(x == what)
    # its keys wild too: no other row changes
    c["k_tree"][wild] = what
    got, got_lse, _ = att.run(c)
    assert torch.equal(got[others], out[others]) and torch.equal(got_lse[others], lse[others])
