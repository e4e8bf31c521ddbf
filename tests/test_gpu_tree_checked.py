"""GPU: the operators on drafted trees in the build with device-side index checks, loaded beside the
product library. No check may fail; verification there also takes the way of a workgroup that has
waited for the others' sums in vain (every second workgroup of a request finds some of them
missing), and has to give the product's results all the same."""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest
import torch

import device_draft_verification_specverify_amd as sv
import test_gpu_tree_attention as att
import test_gpu_tree_cache as cache
import test_gpu_tree_draw as draw
import test_gpu_tree_verify as ver
from device_draft_verification_specverify_amd import build
from oracle import tree as ora

pytestmark = pytest.mark.gpu


@pytest.fixture
def checked(monkeypatch):
    """A function that runs what it is given on the checked library; no check fails in the test."""
    assert os.path.exists(build.CHECKED_LIBRARY), "run __graft_entry__.build() first"
    lib = ctypes.CDLL(build.CHECKED_LIBRARY)
    for name, (res, args) in sv._SIGNATURES.items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    product = sv.load_library()

    def on_checked(fn):
        monkeypatch.setattr(sv, "_lib", lib)
        try:
            sv.check_count(reset=True)
            out = fn()
            torch.cuda.synchronize()
            assert sv.check_count() == 0
            return out
        finally:
            monkeypatch.setattr(sv, "_lib", product)

    return on_checked


# several workgroups a request: rows in registers, rows read again (64 requests, or shares of more
# chunks than a workgroup takes at once), rows that begin anywhere
@pytest.mark.parametrize("mode", ver.MODES)
@pytest.mark.parametrize("B,most,V,stride", [(3, 20, 40000, None), (5, 12, 128256, None),
                                             (64, 4, 40000, None), (40, 6, 60000, None),
                                             (3, 9, 40000, 40003), (2, 7, 300000, None)])
def test_verification_without_the_others_sums(checked, mode, B, most, V, stride):
    c = ver.case(B + V + mode, B, most, "random", V, mode)
    want = ver.check(c, stride=stride)
    got = checked(lambda: ver.run(c, stride=stride))
    for k in ("accept_len", "path", "emitted", "out_token"):
        assert np.array_equal(got[k], want[k]), k
    assert got["error"] == want["error"]


def test_draws_without_the_others_sums(checked):
    c = draw.stars(7, 64, 128256, 20, 2, ora.IID)
    want = ver.check(c)
    assert np.array_equal(checked(lambda: ver.run(c))["out_token"], want["out_token"])


def test_wrong_rows_without_the_others_sums(checked):
    c = ver.case(9, 6, 5, "chain", 60000, ora.IID)
    c["target"][c["node_start"][1], 50000] = float("nan")
    c["draft"][c["node_start"][3], 100] = -1.0
    want = ver.check(c)
    got = checked(lambda: ver.run(c))
    assert got["error"] == want["error"]
    assert np.array_equal(got["accept_len"], want["accept_len"])


@pytest.mark.parametrize("mode", ver.MODES)
@pytest.mark.parametrize("B,most,V", [(3, 20, 1000), (64, 4, 9000), (2, 65, 300)])
def test_verification_checks_no_wrong_index(checked, mode, B, most, V):
    c = ver.case(B + V + mode, B, most, "random", V, mode)
    want = ver.check(c)
    got = checked(lambda: ver.run(c))
    assert np.array_equal(got["emitted"], want["emitted"]) and got["error"] == want["error"]


@pytest.mark.parametrize("D,most,lengths", [(64, 5, [3000, 0, 70]), (128, 33, [2000, 5]),
                                            (80, 100, [40, 900]), (256, 9, [1500, 33]),
                                            (200, 60, [700, 1])])
@pytest.mark.parametrize("page_size", [2, 16])
def test_attention_checks_no_wrong_index(checked, D, most, lengths, page_size):
    c = att.case(D + most, lengths, [most] * len(lengths), 8, 2, D, page_size)
    want, _, _, _, _ = att.check(c)
    got, _, err = checked(lambda: att.run(c))
    assert err == 0 and torch.equal(got, want)


def test_attention_of_bad_data_checks_no_wrong_index(checked):
    c = att.case(3, [70, 40, 20], [4, 2, 3], 4, 2, 64, 16)
    c["table"][0, 2] = -1
    c["table"][1, 0] = c["k_cache"].shape[0]
    c["start"] = np.array([0, 4, 3, 9], dtype=np.int32)
    _, _, want = att.run(c)
    assert checked(lambda: att.run(c))[2] == want == ora.ERR_PAGE | ora.ERR_TREE


def test_plan_and_commit_check_no_wrong_index(checked):
    checked(lambda: cache.check_plan(cache.plan_case(5, 300, "random", 65, 16, 300)))
    checked(lambda: cache.check_plan(cache.plan_case(6, 20, "chain", 9, 4, 30, spare=10)))
    checked(lambda: cache.check_commit(
        cache.commit_case(7, 9, 3, 3, 80, 16, torch.bfloat16, "head")))
    checked(lambda: cache.check_commit(
        cache.commit_case(8, 2, 1, 1, 8, 1, torch.float32, "token")))
