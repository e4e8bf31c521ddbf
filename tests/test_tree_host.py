"""The C ABI of the operators on drafted token trees on the host (no GPU needed): exports, workspace
sizes and the refusals that come before any device work."""
import os
import re

import pytest
import torch

import device_draft_verification_specverify_amd as sv
from device_draft_verification_specverify_amd import tree

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "specverify_tree.h")

pytestmark = pytest.mark.skipif(not os.path.exists(sv.LIBRARY),
                                reason="libspecverify.so not built (run __graft_entry__.build())")

EINVAL, EDTYPE, EWORKSPACE, EALIGN = -1, -2, -3, -4


def test_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(specverify_[a-z_]+)\s*\(", text))
    assert names == set(tree._TREE_SIGNATURES)
    for n in names:
        assert hasattr(tree._lib(), n), n


PLAN = dict(parents=16, node_start=16, prefix_len=16, pages_in=16, block_table=16, free_pages=16,
            free_head_in=16, B=2, T=5, max_nodes=4, max_path=3, page_size=16, max_pages=8,
            table_stride=8, num_pages=20, num_free=4, ancestors=16, depth=16, position=16, slots=16,
            pages_out=32, free_head_out=32, device_error=None, stream=None)
ATT = dict(q=16, k_tree=16, v_tree=16, k_cache=16, v_cache=16, dtype=1, B=2, T=5, Hq=4, Hkv=2, D=64,
           max_nodes=4, qt=256, qh=64, nt=128, nh=64, cp=2048, ct=128, ch=64, num_pages=9,
           page_size=16, table=16, max_pages=8, table_stride=8, prefix_len=16, node_start=16,
           ancestors=None, scale=0.125, out=16, ot=256, oh=64, lse=None, err=None, ws=256,
           bytes=1 << 30, stream=None)
VER = dict(target=16, draft=16, dtype=0, mode=1, tokens=16, parents=16, node_start=16, B=2, T=5,
           V=100, max_nodes=4, max_path=3, ts=100, ds=100, u=16, r=16, accept=16, path=16,
           emitted=None, out=16, err=None, ws=256, bytes=1 << 30, stream=None)
COM = dict(k_tree=16, v_tree=16, k_cache=16, v_cache=16, dtype=1, layers=2, B=2, T=5, H=2, D=64,
           max_nodes=4, max_path=3, nl=640, nt=128, nh=64, cl=18432, cp=2048, ct=128, ch=64,
           num_pages=9, page_size=16, node_start=16, path=16, accept=16, slots=16, len_in=16,
           len_out=16, err=None, stream=None)


def call(name, base, **over):
    assert set(over) <= set(base)
    args = base | over
    fn = getattr(tree._lib(), name)
    assert len(args) == len(tree._TREE_SIGNATURES[name][1])
    return fn(*args.values())


@pytest.mark.parametrize("over", [dict(parents=None), dict(node_start=None), dict(prefix_len=None),
                                  dict(pages_in=None), dict(block_table=None), dict(free_pages=None),
                                  dict(free_head_in=None), dict(ancestors=None), dict(depth=None),
                                  dict(position=None), dict(slots=None), dict(pages_out=None),
                                  dict(free_head_out=None), dict(B=0), dict(T=-1), dict(T=1 << 31),
                                  dict(max_nodes=0), dict(max_nodes=129), dict(max_path=0),
                                  dict(max_path=5), dict(page_size=0), dict(page_size=12),
                                  dict(max_pages=0), dict(table_stride=7), dict(num_pages=0),
                                  dict(num_free=-1), dict(B=1 << 30), dict(pages_out=16),
                                  dict(free_head_out=16), dict(max_pages=1 << 28, table_stride=1 << 28)])
def test_plan_refusals(over):
    assert call("specverify_tree_plan", PLAN, **over) == EINVAL


@pytest.mark.parametrize("status,over", [
    *[(EINVAL, {k: None}) for k in ("q", "k_tree", "v_tree", "k_cache", "v_cache", "table",
                                    "prefix_len", "node_start", "out")],
    *[(EINVAL, {k: -8}) for k in ("qt", "qh", "nt", "nh", "cp", "ct", "ch", "ot", "oh")],
    *[(EALIGN, {k: 68}) for k in ("qt", "qh", "nt", "nh", "cp", "ct", "ch", "ot", "oh")],
    *[(EALIGN, {k: 24}) for k in ("q", "k_tree", "v_tree", "k_cache", "v_cache", "out")],
    (EINVAL, dict(B=0)), (EINVAL, dict(T=-1)), (EINVAL, dict(Hq=5)), (EINVAL, dict(Hq=0)),
    (EINVAL, dict(Hkv=0)), (EINVAL, dict(D=0)), (EINVAL, dict(D=60)), (EINVAL, dict(D=264)),
    (EINVAL, dict(max_nodes=0)), (EINVAL, dict(max_nodes=129)), (EINVAL, dict(Hq=1 << 16)),
    (EINVAL, dict(page_size=24)), (EINVAL, dict(page_size=0)), (EINVAL, dict(max_pages=0)),
    (EINVAL, dict(max_pages=1 << 27, table_stride=1 << 27)), (EINVAL, dict(table_stride=7)),
    (EINVAL, dict(num_pages=0)), (EINVAL, dict(scale=0.0)), (EINVAL, dict(scale=-1.0)),
    (EINVAL, dict(scale=float("nan"))), (EINVAL, dict(scale=float("inf"))),
    (EDTYPE, dict(dtype=0)), (EDTYPE, dict(dtype=3)), (EWORKSPACE, dict(ws=None)),
    (EWORKSPACE, dict(bytes=100)), (EALIGN, dict(ws=264)), (0, dict(T=0, q=None, out=None))])
def test_attention_refusals(status, over):
    assert call("specverify_tree_attention", ATT, **over) == status


@pytest.mark.parametrize("status,over", [
    *[(EINVAL, {k: None}) for k in ("target", "draft", "tokens", "parents", "node_start", "u", "r",
                                    "accept", "path", "out")],
    (EINVAL, dict(mode=0)), (EINVAL, dict(mode=3)), (EINVAL, dict(mode=-1)), (EINVAL, dict(B=0)),
    (EINVAL, dict(T=-1)), (EINVAL, dict(V=0)), (EINVAL, dict(V=(1 << 22) + 1)),
    (EINVAL, dict(max_nodes=0)), (EINVAL, dict(max_nodes=129)), (EINVAL, dict(max_path=0)),
    (EINVAL, dict(max_path=5)), (EINVAL, dict(ts=-1)), (EINVAL, dict(ds=-1)), (EDTYPE, dict(dtype=2)),
    (EWORKSPACE, dict(ws=None)), (EWORKSPACE, dict(bytes=8)), (EALIGN, dict(ws=260))])
def test_verify_refusals(status, over):
    assert call("specverify_tree_verify", VER, **over) == status


@pytest.mark.parametrize("status,over", [
    *[(EINVAL, {k: None}) for k in ("k_tree", "v_tree", "k_cache", "v_cache", "node_start", "path",
                                    "accept", "slots", "len_in", "len_out")],
    *[(EINVAL, {k: -8}) for k in ("nl", "nt", "nh", "cl", "cp", "ct", "ch")],
    *[(EALIGN, {k: 68}) for k in ("nl", "nt", "nh", "cl", "cp", "ct", "ch")],
    *[(EALIGN, {k: 24}) for k in ("k_tree", "v_tree", "k_cache", "v_cache")],
    (EINVAL, dict(layers=0)), (EINVAL, dict(B=0)), (EINVAL, dict(T=-1)), (EINVAL, dict(H=0)),
    (EINVAL, dict(H=1 << 16)), (EINVAL, dict(D=4)), (EINVAL, dict(D=264)),
    (EINVAL, dict(max_nodes=129)), (EINVAL, dict(max_path=5)), (EINVAL, dict(num_pages=0)),
    (EINVAL, dict(page_size=3)), (EINVAL, dict(layers=1 << 16, B=1 << 16)), (EDTYPE, dict(dtype=5))])
def test_commit_refusals(status, over):
    assert call("specverify_tree_commit", COM, **over) == status


def test_workspace_sizes():
    lib = tree._lib()
    n = lib.specverify_tree_attention_workspace_size(64, 576, 32, 8, 128, 9)
    assert n > 0 and n % 256 == 0
    for bad in ((0, 5, 4, 2, 64, 4), (2, 5, 5, 2, 64, 4), (2, 5, 4, 2, 65, 4), (2, 5, 4, 2, 64, 0)):
        assert lib.specverify_tree_attention_workspace_size(*bad) == 0
    assert lib.specverify_tree_verify_workspace_size(64, 128256, 9) > 0
    for bad in ((0, 10, 2), (1, 0, 2), (1, 10, 200), (1, 1 << 23, 2)):
        assert lib.specverify_tree_verify_workspace_size(*bad) == 0


@pytest.mark.parametrize("over", [dict(ot=0), dict(oh=0), dict(oh=56), dict(ot=248), dict(ot=64),
                                  dict(ot=64, oh=256), dict(ot=0, oh=0)])
def test_attention_refuses_an_output_whose_rows_overlap(over):
    assert call("specverify_tree_attention", ATT, **over) == EINVAL


@pytest.mark.parametrize("scale", [3e38, 2.4e38])
def test_attention_refuses_a_scale_that_overflows_in_base_two(scale):
    assert call("specverify_tree_attention", ATT, scale=scale) == EINVAL


@pytest.mark.parametrize("over", [dict(cl=0), dict(cp=0), dict(ct=0), dict(ch=0), dict(ch=56),
                                  dict(cp=2040), dict(cl=18424), dict(ch=128)])
def test_commit_refuses_a_cache_whose_tokens_overlap(over):
    assert call("specverify_tree_commit", COM, **over) == EINVAL


def test_binding_refuses_a_table_of_overlapping_rows():
    dev = torch.device("cpu")
    one = torch.zeros((1, 6), dtype=torch.int32)
    assert tree._table(one, 1, dev) == (6, 6)
    assert tree._table(torch.zeros((3, 9), dtype=torch.int32)[:, :6], 3, dev) == (6, 9)
    assert tree._table(torch.zeros(20, dtype=torch.int32).as_strided((1, 6), (2, 1)), 1, dev)[1] == 6
    for bad in (one.expand(3, 6), torch.zeros(20, dtype=torch.int32).as_strided((3, 6), (4, 1))):
        with pytest.raises(sv.SpecVerifyError, match="block_table"):
            tree._table(bad, 3, dev)


def test_binding_refuses_a_workspace_of_fewer_bytes_than_it_shows():
    dev = torch.device("cpu")
    ok = torch.empty(1024, dtype=torch.uint8)
    assert tree._scratch(ok, 512, dev, "size") is ok
    for bad in (torch.empty(1, dtype=torch.uint8).expand(1 << 20), ok[::2], ok.to(torch.float32)):
        with pytest.raises(sv.SpecVerifyError, match="ws"):
            tree._scratch(bad, 512, dev, "size")
    with pytest.raises(sv.SpecVerifyError, match="size"):
        tree._scratch(None, 0, dev, "size")
