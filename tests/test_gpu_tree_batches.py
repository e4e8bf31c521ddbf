"""GPU: a request of a batch against the same request alone, and rows behind the last request."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import test_gpu_tree_attention as att
import test_gpu_tree_cache as cache
import test_gpu_tree_verify as ver
from device_draft_verification_specverify_amd import tree
from tree_helpers import DEV, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_alone_and_in_a_batch(D):
    # shared out differently, so not the same bits: each within its tolerance of float64
    c = att.case(19 + D, [500, 64, 1000, 3], [9, 2, 17, 1], 8, 2, D, 16)
    att.check(c)
    for b in range(4):
        lo, hi = int(c["start"][b]), int(c["start"][b + 1])
        att.check(c | {n: c[n][lo:hi] for n in ("q", "k_tree", "v_tree", "anc")} |
                  {"table": c["table"][b:b + 1], "lengths": c["lengths"][b:b + 1],
                   "start": np.array([0, hi - lo], dtype=np.int32)})


@pytest.mark.parametrize("mode", ver.MODES)
def test_verification_alone_and_in_a_batch(mode):
    c = ver.case(3 + mode, 40, 6, "random", 40000, mode)
    all_ = ver.check(c)
    for b in range(0, 40, 13):
        lo, hi = int(c["node_start"][b]), int(c["node_start"][b + 1])
        one = c | {n: c[n][lo:hi] for n in ("target", "tokens", "parents", "u")} | {
            "draft": None if c["draft"] is None else c["draft"][lo:hi], "r": c["r"][b:b + 1],
            "node_start": np.array([0, hi - lo], dtype=np.int32)}
        got = ver.run(one)
        assert np.array_equal(got["emitted"][0], all_["emitted"][b])
        assert np.array_equal(got["path"][0], all_["path"][b])


def test_plan_leaves_rows_behind_the_last_request_as_they_were():
    c = cache.plan_case(10, 3, "chain", 6, 4, 20)
    used = len(c["parents"])
    T, B = used + 5, 3
    i32 = dict(dtype=torch.int32, device=DEV)
    par = dev(np.concatenate([c["parents"], np.full(5, 77, dtype=np.int32)]))
    args = [dev(c[k]) for k in ("node_start", "prefix_len", "pages", "block_table", "free_pages")]
    head = torch.zeros(1, **i32)
    anc = torch.full((T, 1), -9, dtype=torch.int64, device=DEV)
    depth, position = torch.full((T,), -9, **i32), torch.full((T,), -9, **i32)
    slots = torch.empty((B, 6), dtype=torch.int64, device=DEV)
    pages, head_out = torch.empty(B, **i32), torch.empty(1, **i32)
    width = c["block_table"].shape[1]
    status = tree._lib().specverify_tree_plan(
        par.data_ptr(), *(t.data_ptr() for t in args), head.data_ptr(), B, T, 6, 6, 4, width, width,
        c["num_pages"], len(c["free_pages"]), anc.data_ptr(), depth.data_ptr(),
        position.data_ptr(), slots.data_ptr(), pages.data_ptr(), head_out.data_ptr(), None,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0
    for t in (anc, depth, position):
        assert torch.all(t[used:] == -9) and not torch.any(t[:used] == -9)
