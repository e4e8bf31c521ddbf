"""GPU: operators on drafted trees at the ends of their ranges: memory behind 32 bits of offset,
axes in unusual orders, pages that requests share, more requests than workgroups."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import device_draft_verification_specverify_amd as sv
import test_gpu_tree_attention as att
import test_gpu_tree_cache as cache
import test_gpu_tree_verify as ver
from tree_helpers import DEV

pytestmark = pytest.mark.gpu


def spread(tensors, strides):
    """The tensors with these strides, one behind the other within an innermost gap."""
    size = 1 + sum((n - 1) * s for n, s in zip(tensors[0].shape, strides))
    apart = tensors[0].shape[-1] * 64
    wide = torch.empty(size + apart * len(tensors), dtype=tensors[0].dtype, device=DEV)
    out = []
    for i, t in enumerate(tensors):
        view = wide.as_strided(t.shape, strides, i * apart)
        view.copy_(t)
        out.append(view)
    return out


def test_attention_over_pages_behind_32_bits():
    c = att.case(31, [400, 37, 0], [9, 3, 2], 8, 2, 64, 16)
    pages = c["k_cache"].shape[0]
    stride = (1 << 32) // pages // 64 * 64                 # 8 GiB from the first page to the last
    c["k_cache"], c["v_cache"] = spread([c["k_cache"], c["v_cache"]], (stride, 256, 128, 1))
    att.check(c)


def test_attention_over_tokens_behind_32_bits():
    # the axis of a page's tokens outermost
    c = att.case(32, [300, 70], [5, 12], 4, 2, 128, 64)
    stride = (1 << 32) // 64
    c["k_cache"], c["v_cache"] = spread([c["k_cache"], c["v_cache"]], (1 << 18, stride, 1 << 15, 1))
    att.check(c)


def test_attention_of_rows_behind_32_bits():
    c = att.case(33, [100, 3], [6, 3], 4, 2, 64, 16)
    for names in (["q"], ["k_tree", "v_tree"]):
        far = spread([c[n] for n in names], (1 << 28, 1 << 16, 1))  # 4 GiB from row 0 to row 8
        c |= dict(zip(names, far))
    out = spread([torch.zeros((9, 4, 64), dtype=torch.bfloat16, device=DEV)],
                 (1 << 28, 1 << 16, 1))[0]
    att.check(c, out=out)


def test_attention_with_the_heads_outermost():
    c = att.case(34, [90, 40], [7, 20], 6, 2, 80, 16, torch.float16, layout="head")
    for name in ("q", "k_tree", "v_tree"):
        c[name] = c[name].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.zeros((6, 27, 80), dtype=torch.float16, device=DEV).transpose(0, 1)
    att.check(c, out=out)


def test_requests_that_share_pages():
    c = att.case(35, [128, 128, 64], [3, 3, 3], 4, 2, 64, 16)
    c["table"][1] = c["table"][0]
    c["table"][2, :4] = c["table"][0, 4:8]
    att.check(c)


@pytest.mark.parametrize("mode", ver.MODES)
def test_verify_of_rows_behind_32_bits(mode):
    c = ver.case(36 + mode, 2, 5, "random", 9000, mode)
    ref = ver.reference(c)
    T, V = c["target"].shape
    step = 1 << 29                                          # 2 GiB from row to row
    wide = torch.empty((T - 1) * step + 2 * V + 8, dtype=torch.float32, device=DEV)
    put = [wide.as_strided((T, V), (step, 1), at) for at in (0, V + 8)]
    far = []
    for x, name in zip(put, ("target", "draft")):
        if c[name] is not None:
            x.copy_(torch.from_numpy(c[name]).to(DEV))
        far.append(None if c[name] is None else x)
    o = ver.tree.specverify_tree_verify(
        far[0], far[1], *(ver.dev(c[k]) for k in ("tokens", "parents", "node_start", "u", "r")),
        mode=mode, max_nodes=c["max_nodes"], max_path=c["max_path"])
    torch.cuda.synchronize()
    for k in ("accept_len", "path", "emitted", "out_token"):
        assert np.array_equal(getattr(o, k).cpu().numpy(), ref[k]), k


@pytest.mark.parametrize("mode", ver.MODES)
def test_verify_of_more_requests_than_workgroups(mode):
    ver.check(ver.case(40 + mode, 600, 4, "random", 4100, mode))


def test_commit_behind_32_bits():
    c = cache.commit_case(44, 5, 3, 2, 64, 16, torch.bfloat16, "token", fused=False)
    L, pages = c["k_cache"].shape[:2]
    near = {k: cache.bits(c[k]) for k in ("k_tree", "v_tree", "k_cache", "v_cache")}
    c["k_cache"], c["v_cache"] = spread([c["k_cache"], c["v_cache"]],
                                        (1 << 31, (1 << 31) // pages // 8192 * 8192, 256, 128, 1))
    c["k_tree"], c["v_tree"] = spread([c["k_tree"], c["v_tree"]], (256, 1 << 27, 128, 1))
    for k, x in near.items():
        assert np.array_equal(cache.bits(c[k]), x), k
    assert cache.check_commit(c) == 0


@pytest.mark.parametrize("over", [dict(max_nodes=-100), dict(max_nodes=0), dict(max_path=-1),
                                  dict(max_path=6), dict(page_size=24), dict(num_pages=0)])
def test_plan_refuses_sizes_before_any_work(over):
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.full((1, 4), -1, **i32)
    sizes = dict(page_size=16, num_pages=8, max_nodes=5, max_path=5) | over
    with pytest.raises(sv.SpecVerifyError, match="status -1"):
        ver.tree.specverify_tree_plan(
            torch.tensor([-1, 0], **i32), torch.tensor([0, 2], **i32), torch.zeros(1, **i32),
            torch.zeros(1, **i32), table, torch.arange(8, **i32), torch.zeros(1, **i32), **sizes)
    torch.cuda.synchronize()
    assert torch.all(table == -1)
