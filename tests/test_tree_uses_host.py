"""The binding of the operators on drafted trees refuses tensors in host memory before any device
work (no GPU needed)."""
import os

import pytest
import torch

import device_draft_verification_specverify_amd as sv
from device_draft_verification_specverify_amd import tree

pytestmark = pytest.mark.skipif(not os.path.exists(sv.LIBRARY),
                                reason="libspecverify.so not built (run __graft_entry__.build())")


def ints(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


def test_calls_with_tensors_in_host_memory():
    kv = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    calls = [
        lambda: tree.specverify_tree_plan(ints(3), ints(2), ints(1), ints(1), ints(1, 4), ints(4),
                                          ints(1), page_size=16, num_pages=4, max_nodes=3, max_path=3),
        lambda: tree.specverify_tree_attention(kv, kv, kv, cache, cache, ints(1, 4), ints(1), ints(2),
                                               max_nodes=3),
        lambda: tree.specverify_tree_verify(torch.zeros(3, 50), None, ints(3), ints(3), ints(2),
                                            torch.zeros(3, dtype=torch.float64),
                                            torch.zeros(1, dtype=torch.float64),
                                            mode=tree.DRAFT_FIXED, max_nodes=3, max_path=3),
        lambda: tree.specverify_tree_commit(kv[None], kv[None], cache[None], cache[None], ints(2),
                                            ints(1, 3), ints(1), ints(1, 3, dtype=torch.int64), ints(1)),
    ]
    for call in calls:
        with pytest.raises(sv.SpecVerifyError, match="must be a device tensor"):
            call()
