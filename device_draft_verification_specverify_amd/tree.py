"""Python binding of the operators on drafted token trees (include/specverify_tree.h).

Argument marshalling only, as in the package: every step runs in the HIP kernels of
``libspecverify.so``; torch supplies device memory and the stream. A serving loop calls
``specverify_tree_plan``, ``specverify_tree_attention`` (once per layer),
``specverify_tree_verify`` and ``specverify_tree_commit`` per decoding step; none of them
waits for the GPU, and all of them can be captured into a graph.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from dataclasses import dataclass

import torch

from . import (SV_BF16, SV_ERR_ROW, SV_ERR_TOKEN, SV_F32, SpecVerifyError, _check, _need, _ptr,
               load_library)

SV_F16 = 2
SV_ERR_TREE = 8
SV_ERR_PAGE = 16
SV_ERR_UNIFORM = 32
SV_ERR_LENGTH = 64
DRAFT_FIXED = 0
DRAFT_IID = 1
DRAFT_DISTINCT = 2
MAX_TREE_NODES = 128
MAX_TREE_VOCAB = 1 << 22
MAX_HEAD_DIM = 256

_P = ctypes.c_void_p
_I = ctypes.c_int64
_INT = ctypes.c_int
_SZ = ctypes.c_size_t

_TREE_SIGNATURES = {
    "specverify_tree_plan": (_INT, [_P] * 7 + [_I] * 9 + [_P] * 8),
    "specverify_tree_attention_workspace_size": (_SZ, [_I] * 6),
    "specverify_tree_attention": (_INT, [_P] * 5 + [_INT] + [_I] * 15 + [_P, _I, _I] + [_P] * 3 +
                                  [ctypes.c_float, _P, _I, _I, _P, _P, _P, _SZ, _P]),
    "specverify_tree_verify_workspace_size": (_SZ, [_I] * 3),
    "specverify_tree_verify": (_INT, [_P, _P, _INT, _INT] + [_P] * 3 + [_I] * 7 + [_P] * 8 +
                               [_SZ, _P]),
    "specverify_tree_commit": (_INT, [_P] * 4 + [_INT] + [_I] * 16 + [_P] * 8),
}

_DTYPES = {torch.float32: SV_F32, torch.bfloat16: SV_BF16, torch.float16: SV_F16}

_bound = None


def _lib() -> ctypes.CDLL:
    global _bound
    lib = load_library()
    if _bound is not lib:
        for name, (res, args) in _TREE_SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _bound = lib
    return lib


def _on(device: torch.device):
    """The device of the tensors as the current one, as the C entry points ask."""
    return nullcontext() if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _same_device(device: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise SpecVerifyError(f"{name} is on {t.device}, the others on {device}")


def _strided(t: torch.Tensor, ndim: int, name: str) -> None:
    if not t.is_cuda or t.dim() != ndim or (t.numel() and t.shape[-1] > 1 and t.stride(-1) != 1):
        raise SpecVerifyError(f"{name}: want a {ndim}-d device tensor with a contiguous last axis")


def _same_layout(a: torch.Tensor, b: torch.Tensor, names: str) -> None:
    if a.shape != b.shape or a.stride() != b.stride() or a.dtype != b.dtype:
        raise SpecVerifyError(f"{names} differ in shape, strides or type")


def _dtype(t: torch.Tensor, allowed: tuple, name: str) -> int:
    if t.dtype not in allowed:
        raise SpecVerifyError(f"{name} must be one of {allowed}, got {t.dtype}")
    return _DTYPES[t.dtype]


def _error_word(t: torch.Tensor | None) -> None:
    if t is not None:
        _need(t, torch.int32, (1,), "device_error")


@dataclass
class TreePlanOutputs:
    ancestors: torch.Tensor  # [T, ceil(max_nodes / 64)] int64 (the masks' 64 bits)
    depth: torch.Tensor      # [T] int32
    position: torch.Tensor   # [T] int32
    slots: torch.Tensor      # [B, max_path] int64
    pages: torch.Tensor      # [B] int32: pages owned now
    free_head: torch.Tensor  # [1] int32


def specverify_tree_plan(parents: torch.Tensor, node_start: torch.Tensor, prefix_len: torch.Tensor,
                         pages: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                         free_head: torch.Tensor, *, page_size: int, num_pages: int,
                         max_nodes: int, max_path: int,
                         device_error: torch.Tensor | None = None) -> TreePlanOutputs:
    """Ancestor masks, depths, positions, and room in the cache: block_table [B, max_pages] int32
    is filled in place with pages from free_pages[free_head:], the rest comes back new."""
    lib = _lib()
    dev = parents.device
    T, B = parents.numel(), prefix_len.numel()
    _need(parents, torch.int32, (T,), "parents")
    _need(node_start, torch.int32, (B + 1,), "node_start")
    _need(prefix_len, torch.int32, (B,), "prefix_len")
    _need(pages, torch.int32, (B,), "pages")
    _need(free_pages, torch.int32, (free_pages.numel(),), "free_pages")
    _need(free_head, torch.int32, (1,), "free_head")
    _strided(block_table, 2, "block_table")
    if block_table.dtype != torch.int32 or block_table.shape[0] != B:
        raise SpecVerifyError(f"block_table: want int32 [{B}, max_pages]")
    _error_word(device_error)
    _same_device(dev, node_start=node_start, prefix_len=prefix_len, pages=pages,
                 block_table=block_table, free_pages=free_pages, free_head=free_head,
                 device_error=device_error)
    words = (max_nodes + 63) // 64
    out = TreePlanOutputs(
        ancestors=torch.empty((T, words), dtype=torch.int64, device=dev),
        depth=torch.empty(T, dtype=torch.int32, device=dev),
        position=torch.empty(T, dtype=torch.int32, device=dev),
        slots=torch.empty((B, max(max_path, 0)), dtype=torch.int64, device=dev),
        pages=torch.empty(B, dtype=torch.int32, device=dev),
        free_head=torch.empty(1, dtype=torch.int32, device=dev))
    width = block_table.shape[1]
    with _on(dev):
        st = lib.specverify_tree_plan(
            parents.data_ptr(), node_start.data_ptr(), prefix_len.data_ptr(), pages.data_ptr(),
            block_table.data_ptr(), free_pages.data_ptr(), free_head.data_ptr(), B, T, max_nodes,
            max_path, page_size, width, max(width, block_table.stride(0)), num_pages,
            free_pages.numel(), out.ancestors.data_ptr(), out.depth.data_ptr(),
            out.position.data_ptr(), out.slots.data_ptr(), out.pages.data_ptr(),
            out.free_head.data_ptr(), _ptr(device_error), _stream(dev))
    _check(st, "specverify_tree_plan")
    return out


def tree_attention_workspace(B: int, T: int, Hq: int, Hkv: int, D: int, max_nodes: int,
                             device) -> torch.Tensor:
    n = int(_lib().specverify_tree_attention_workspace_size(B, T, Hq, Hkv, D, max_nodes))
    if n == 0:
        raise SpecVerifyError("sizes rejected by specverify_tree_attention_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)  # any contents will do


def specverify_tree_attention(q: torch.Tensor, k_tree: torch.Tensor, v_tree: torch.Tensor,
                              k_cache: torch.Tensor, v_cache: torch.Tensor,
                              block_table: torch.Tensor, prefix_len: torch.Tensor,
                              node_start: torch.Tensor, ancestors: torch.Tensor | None = None, *,
                              max_nodes: int, scale: float | None = None,
                              out: torch.Tensor | None = None, want_lse: bool = False,
                              device_error: torch.Tensor | None = None,
                              ws: torch.Tensor | None = None):
    """(out [T, Hq, D], lse [T, Hq] float32 or None): the drafted nodes' attention.

    q [T, Hq, D], k_tree and v_tree [T, Hkv, D], k_cache and v_cache [num_pages, page_size, Hkv, D]
    (bfloat16 or float16, last axis contiguous, other strides multiples of 8 elements; the keys'
    and values' strides agree), ancestors [T, ceil(max_nodes / 64)] int64 or None for chains,
    scale 1 / sqrt(D) if not given."""
    lib = _lib()
    for t, ndim, name in ((q, 3, "q"), (k_tree, 3, "k_tree"), (v_tree, 3, "v_tree"),
                          (k_cache, 4, "k_cache"), (v_cache, 4, "v_cache")):
        _strided(t, ndim, name)
    _same_layout(k_tree, v_tree, "k_tree and v_tree")
    _same_layout(k_cache, v_cache, "k_cache and v_cache")
    dev = q.device
    T, Hq, D = q.shape
    num_pages, page_size, Hkv = k_cache.shape[:3]
    B = prefix_len.numel()
    if k_tree.shape != (T, Hkv, D) or k_cache.shape[3] != D:
        raise SpecVerifyError("q [T, Hq, D], k_tree [T, Hkv, D] and k_cache [.., .., Hkv, D] disagree")
    dt = _dtype(q, (torch.bfloat16, torch.float16), "q")
    if k_tree.dtype != q.dtype or k_cache.dtype != q.dtype:
        raise SpecVerifyError("q, the nodes' and the cache's types differ")
    _need(prefix_len, torch.int32, (B,), "prefix_len")
    _need(node_start, torch.int32, (B + 1,), "node_start")
    _strided(block_table, 2, "block_table")
    if block_table.dtype != torch.int32 or block_table.shape[0] != B:
        raise SpecVerifyError(f"block_table: want int32 [{B}, max_pages]")
    if ancestors is not None:
        _need(ancestors, torch.int64, (T, (max_nodes + 63) // 64), "ancestors")
    if out is None:
        out = torch.empty((T, Hq, D), dtype=q.dtype, device=dev)
    else:
        _strided(out, 3, "out")
        if out.shape != (T, Hq, D) or out.dtype != q.dtype:
            raise SpecVerifyError(f"out: want {q.dtype} [{T}, {Hq}, {D}]")
    _error_word(device_error)
    _same_device(dev, k_tree=k_tree, v_tree=v_tree, k_cache=k_cache, v_cache=v_cache,
                 block_table=block_table, prefix_len=prefix_len, node_start=node_start,
                 ancestors=ancestors, out=out, device_error=device_error, ws=ws)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if want_lse else None
    if ws is None:
        ws = tree_attention_workspace(B, T, Hq, Hkv, D, max_nodes, dev)
    width = block_table.shape[1]
    qs, ns, cs, os_ = q.stride(), k_tree.stride(), k_cache.stride(), out.stride()
    with _on(dev):
        st = lib.specverify_tree_attention(
            q.data_ptr(), k_tree.data_ptr(), v_tree.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), dt, B, T, Hq, Hkv, D, max_nodes, qs[0], qs[1], ns[0], ns[1], cs[0],
            cs[1], cs[2], num_pages, page_size, block_table.data_ptr(), width,
            max(width, block_table.stride(0)), prefix_len.data_ptr(), node_start.data_ptr(),
            _ptr(ancestors), D ** -0.5 if scale is None else scale, out.data_ptr(), os_[0], os_[1],
            _ptr(lse), _ptr(device_error), ws.data_ptr(), ws.numel(), _stream(dev))
    _check(st, "specverify_tree_attention")
    return out, lse


@dataclass
class TreeVerifyOutputs:
    accept_len: torch.Tensor  # [B] int32
    path: torch.Tensor        # [B, max_path] int32
    emitted: torch.Tensor     # [B, max_path] int32
    out_token: torch.Tensor   # [B] int32


def tree_verify_workspace(B: int, V: int, max_nodes: int, device) -> torch.Tensor:
    n = int(_lib().specverify_tree_verify_workspace_size(B, V, max_nodes))
    if n == 0:
        raise SpecVerifyError("sizes rejected by specverify_tree_verify_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)  # any contents will do


def specverify_tree_verify(target_probs: torch.Tensor, draft_probs: torch.Tensor | None,
                           tokens: torch.Tensor, parents: torch.Tensor, node_start: torch.Tensor,
                           u: torch.Tensor, r: torch.Tensor, *, mode: int, max_nodes: int,
                           max_path: int, device_error: torch.Tensor | None = None,
                           ws: torch.Tensor | None = None) -> TreeVerifyOutputs:
    """The accepted path and the emitted token of every request.

    target_probs and draft_probs [T, V] (float32 or bfloat16, last axis contiguous; draft_probs
    None for DRAFT_FIXED), tokens and parents [T] int32, u [T] and r [B] float64 in [0, 1)."""
    lib = _lib()
    _strided(target_probs, 2, "target_probs")
    T, V = target_probs.shape
    B = r.numel()
    dev = target_probs.device
    dt = _dtype(target_probs, (torch.float32, torch.bfloat16), "target_probs")
    if draft_probs is not None:
        _strided(draft_probs, 2, "draft_probs")
        if draft_probs.shape != (T, V) or draft_probs.dtype != target_probs.dtype:
            raise SpecVerifyError(f"draft_probs: want {target_probs.dtype} [{T}, {V}]")
    _need(tokens, torch.int32, (T,), "tokens")
    _need(parents, torch.int32, (T,), "parents")
    _need(node_start, torch.int32, (B + 1,), "node_start")
    _need(u, torch.float64, (T,), "u")
    _need(r, torch.float64, (B,), "r")
    _error_word(device_error)
    _same_device(dev, draft_probs=draft_probs, tokens=tokens, parents=parents,
                 node_start=node_start, u=u, r=r, device_error=device_error, ws=ws)
    width = max(max_path, 0)
    out = TreeVerifyOutputs(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                            path=torch.empty((B, width), dtype=torch.int32, device=dev),
                            emitted=torch.empty((B, width), dtype=torch.int32, device=dev),
                            out_token=torch.empty(B, dtype=torch.int32, device=dev))
    if ws is None:
        ws = tree_verify_workspace(B, V, max_nodes, dev)
    with _on(dev):
        st = lib.specverify_tree_verify(
            target_probs.data_ptr(), _ptr(draft_probs), dt, mode, tokens.data_ptr(),
            parents.data_ptr(), node_start.data_ptr(), B, T, V, max_nodes, max_path,
            target_probs.stride(0), 0 if draft_probs is None else draft_probs.stride(0),
            u.data_ptr(), r.data_ptr(), out.accept_len.data_ptr(), out.path.data_ptr(),
            out.emitted.data_ptr(), out.out_token.data_ptr(), _ptr(device_error), ws.data_ptr(),
            ws.numel(), _stream(dev))
    _check(st, "specverify_tree_verify")
    return out


def specverify_tree_commit(k_tree: torch.Tensor, v_tree: torch.Tensor, k_cache: torch.Tensor,
                           v_cache: torch.Tensor, node_start: torch.Tensor, path: torch.Tensor,
                           accept_len: torch.Tensor, slots: torch.Tensor, prefix_len: torch.Tensor,
                           *, max_nodes: int = MAX_TREE_NODES, out: torch.Tensor | None = None,
                           device_error: torch.Tensor | None = None) -> torch.Tensor:
    """Writes the accepted nodes' keys and values of every layer into the caches and returns the
    new prefix lengths [B] int32 (into `out`, which may be prefix_len itself).

    k_tree and v_tree [layers, T, H, D], k_cache and v_cache [layers, num_pages, page_size, H, D]
    (float32, bfloat16 or float16, last axis contiguous, other strides multiples of 16 bytes)."""
    lib = _lib()
    for t, ndim, name in ((k_tree, 4, "k_tree"), (v_tree, 4, "v_tree"), (k_cache, 5, "k_cache"),
                          (v_cache, 5, "v_cache")):
        _strided(t, ndim, name)
    _same_layout(k_tree, v_tree, "k_tree and v_tree")
    _same_layout(k_cache, v_cache, "k_cache and v_cache")
    L, T, H, D = k_tree.shape
    num_pages, page_size = k_cache.shape[1:3]
    if k_cache.shape[0] != L or k_cache.shape[3:] != (H, D) or k_cache.dtype != k_tree.dtype:
        raise SpecVerifyError("k_tree [layers, T, H, D] and k_cache [layers, .., .., H, D] disagree")
    dt = _dtype(k_tree, tuple(_DTYPES), "k_tree")
    B, dev = prefix_len.numel(), k_cache.device
    if path.dim() != 2:
        raise SpecVerifyError("path: want [B, max_path]")
    max_path = path.shape[1]
    _need(node_start, torch.int32, (B + 1,), "node_start")
    _need(path, torch.int32, (B, max_path), "path")
    _need(accept_len, torch.int32, (B,), "accept_len")
    _need(slots, torch.int64, (B, max_path), "slots")
    _need(prefix_len, torch.int32, (B,), "prefix_len")
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=dev)
    else:
        _need(out, torch.int32, (B,), "out")
    _error_word(device_error)
    _same_device(dev, k_tree=k_tree, v_tree=v_tree, v_cache=v_cache, node_start=node_start,
                 path=path, accept_len=accept_len, slots=slots, prefix_len=prefix_len, out=out,
                 device_error=device_error)
    ns, cs = k_tree.stride(), k_cache.stride()
    with _on(dev):
        st = lib.specverify_tree_commit(
            k_tree.data_ptr(), v_tree.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), dt, L, B,
            T, H, D, max_nodes, max_path, ns[0], ns[1], ns[2], cs[0], cs[1], cs[2], cs[3],
            num_pages, page_size, node_start.data_ptr(), path.data_ptr(), accept_len.data_ptr(),
            slots.data_ptr(), prefix_len.data_ptr(), out.data_ptr(), _ptr(device_error),
            _stream(dev))
    _check(st, "specverify_tree_commit")
    return out
