"""Python binding of the operators on drafted token trees (include/specverify_tree.h).

Argument marshalling only, as in the package: every step runs in the HIP kernels of
``libspecverify.so``; torch supplies device memory and the stream. A serving loop calls
``specverify_tree_plan``, ``specverify_tree_attention`` (once per layer),
``specverify_tree_verify`` and ``specverify_tree_commit`` per decoding step; none of them
waits for the GPU, and all of them can be captured into a graph.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import (SV_BF16, SV_ERR_ROW, SV_ERR_TOKEN, SV_F32, SpecVerifyError, _check,  # noqa: F401
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


_current_device = torch._C._cuda_getDevice            # torch.cuda.current_device and
_raw_stream = torch._C._cuda_getCurrentRawStream       # current_stream without their wrappers


def _call(name: str, device: torch.device, *args) -> None:
    """Enqueues on the tensors' device's current stream, with that device current as the C entry
    points ask."""
    index = device.index
    fn = getattr(_bound, name)
    if _current_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(index))
    if st:
        _check(st, name)


def _want(t: torch.Tensor, dtype: torch.dtype, shape: tuple, dev: torch.device, name: str) -> None:
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != dev:
        raise SpecVerifyError(f"{name}: want contiguous {dtype} {tuple(shape)} on {dev}, got "
                              f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()} on "
                              f"{t.device}")


def _strided(t: torch.Tensor, dev: torch.device, ndim: int, name: str) -> tuple:
    """The strides of a tensor whose last axis is contiguous."""
    strides = t.stride()
    if (len(strides) != ndim or (strides[-1] != 1 and t.shape[-1] > 1 and t.numel()) or
            t.device != dev):
        raise SpecVerifyError(f"{name}: want a {ndim}-d tensor on {dev} with a contiguous last "
                              f"axis")
    return strides


def _device(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise SpecVerifyError(f"{name} must be a device tensor")
    return t.device


def _pair(a: torch.Tensor, b: torch.Tensor, dev: torch.device, ndim: int, names: str) -> tuple:
    """The strides that two tensors of one shape and type share."""
    strides = _strided(a, dev, ndim, names)
    if a.shape != b.shape or strides != b.stride() or a.dtype is not b.dtype or b.device != dev:
        raise SpecVerifyError(f"{names} differ in shape, strides, type or device")
    return strides


def _dtype(t: torch.Tensor, allowed: tuple, name: str) -> int:
    if t.dtype not in allowed:
        raise SpecVerifyError(f"{name} must be one of {allowed}, got {t.dtype}")
    return _DTYPES[t.dtype]


def _table(t: torch.Tensor, B: int, dev: torch.device) -> tuple:
    """(max_pages, row stride) of a block table."""
    stride = _strided(t, dev, 2, "block_table")[0]
    rows, width = t.shape
    if t.dtype is not torch.int32 or rows != B:
        raise SpecVerifyError(f"block_table: want int32 [{B}, max_pages]")
    if rows > 1 and stride < width:  # rows that overlap, as of an expanded tensor
        raise SpecVerifyError(f"block_table: rows of {width} entries are {stride} apart")
    return width, max(width, stride)


def _optional(t: torch.Tensor | None, dtype: torch.dtype, shape: tuple, dev: torch.device,
              name: str) -> int | None:
    if t is None:
        return None
    _want(t, dtype, shape, dev, name)
    return t.data_ptr()


def _scratch(ws: torch.Tensor | None, nbytes: int, dev: torch.device, name: str) -> torch.Tensor:
    if nbytes == 0:
        raise SpecVerifyError(f"sizes rejected by {name}")
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)  # any contents will do
    if ws.device != dev:
        raise SpecVerifyError(f"ws is on {ws.device}, the tensors on {dev}")
    if ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise SpecVerifyError("ws: want a contiguous uint8 tensor")
    return ws


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
    _lib()
    dev = _device(parents, "parents")
    T, B, free = parents.numel(), prefix_len.numel(), free_pages.numel()
    i32 = torch.int32
    _want(parents, i32, (T,), dev, "parents")
    _want(node_start, i32, (B + 1,), dev, "node_start")
    _want(prefix_len, i32, (B,), dev, "prefix_len")
    _want(pages, i32, (B,), dev, "pages")
    _want(free_pages, i32, (free,), dev, "free_pages")
    _want(free_head, i32, (1,), dev, "free_head")
    width, stride = _table(block_table, B, dev)
    err = _optional(device_error, i32, (1,), dev, "device_error")
    empty = torch.empty
    ancestors = empty((T, max((max_nodes + 63) // 64, 0)), dtype=torch.int64, device=dev)
    depth = empty(T, dtype=i32, device=dev)
    position = empty(T, dtype=i32, device=dev)
    slots = empty((B, max(max_path, 0)), dtype=torch.int64, device=dev)
    now = empty(B, dtype=i32, device=dev)
    head = empty(1, dtype=i32, device=dev)
    _call("specverify_tree_plan", dev, parents.data_ptr(), node_start.data_ptr(),
          prefix_len.data_ptr(), pages.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(),
          free_head.data_ptr(), B, T, max_nodes, max_path, page_size, width, stride, num_pages,
          free, ancestors.data_ptr(), depth.data_ptr(), position.data_ptr(), slots.data_ptr(),
          now.data_ptr(), head.data_ptr(), err)
    return TreePlanOutputs(ancestors, depth, position, slots, now, head)


def tree_attention_workspace(B: int, T: int, Hq: int, Hkv: int, D: int, max_nodes: int,
                             device) -> torch.Tensor:
    n = int(_lib().specverify_tree_attention_workspace_size(B, T, Hq, Hkv, D, max_nodes))
    return _scratch(None, n, device, "specverify_tree_attention_workspace_size")


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
    dev = _device(q, "q")
    qs = _strided(q, dev, 3, "q")
    ns = _pair(k_tree, v_tree, dev, 3, "k_tree and v_tree")
    cs = _pair(k_cache, v_cache, dev, 4, "k_cache and v_cache")
    T, Hq, D = q.shape
    num_pages, page_size, Hkv, width = k_cache.shape
    B = prefix_len.numel()
    if k_tree.shape != (T, Hkv, D) or width != D:
        raise SpecVerifyError("q [T, Hq, D], k_tree [T, Hkv, D] and k_cache [pages, page_size, "
                              "Hkv, D] disagree")
    dt = _dtype(q, (torch.bfloat16, torch.float16), "q")
    if k_tree.dtype is not q.dtype or k_cache.dtype is not q.dtype:
        raise SpecVerifyError("q, the nodes' and the cache's types differ")
    _want(prefix_len, torch.int32, (B,), dev, "prefix_len")
    _want(node_start, torch.int32, (B + 1,), dev, "node_start")
    max_pages, table_stride = _table(block_table, B, dev)
    anc = _optional(ancestors, torch.int64, (T, (max_nodes + 63) // 64), dev, "ancestors")
    if out is None:
        out = torch.empty((T, Hq, D), dtype=q.dtype, device=dev)
    elif out.shape != (T, Hq, D) or out.dtype is not q.dtype:
        raise SpecVerifyError(f"out: want {q.dtype} [{T}, {Hq}, {D}]")
    os_ = _strided(out, dev, 3, "out")
    err = _optional(device_error, torch.int32, (1,), dev, "device_error")
    lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if want_lse else None
    ws = _scratch(ws, lib.specverify_tree_attention_workspace_size(B, T, Hq, Hkv, D, max_nodes),
                  dev, "specverify_tree_attention_workspace_size")
    _call("specverify_tree_attention", dev, q.data_ptr(), k_tree.data_ptr(), v_tree.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), dt, B, T, Hq, Hkv, D, max_nodes, qs[0], qs[1],
          ns[0], ns[1], cs[0], cs[1], cs[2], num_pages, page_size, block_table.data_ptr(),
          max_pages, table_stride, prefix_len.data_ptr(), node_start.data_ptr(), anc,
          D ** -0.5 if scale is None else scale, out.data_ptr(), os_[0], os_[1],
          lse.data_ptr() if want_lse else None, err, ws.data_ptr(), ws.numel())
    return out, lse


@dataclass
class TreeVerifyOutputs:
    accept_len: torch.Tensor  # [B] int32
    path: torch.Tensor        # [B, max_path] int32
    emitted: torch.Tensor     # [B, max_path] int32
    out_token: torch.Tensor   # [B] int32


def tree_verify_workspace(B: int, V: int, max_nodes: int, device) -> torch.Tensor:
    n = int(_lib().specverify_tree_verify_workspace_size(B, V, max_nodes))
    return _scratch(None, n, device, "specverify_tree_verify_workspace_size")


def specverify_tree_verify(target_probs: torch.Tensor, draft_probs: torch.Tensor | None,
                           tokens: torch.Tensor, parents: torch.Tensor, node_start: torch.Tensor,
                           u: torch.Tensor, r: torch.Tensor, *, mode: int, max_nodes: int,
                           max_path: int, device_error: torch.Tensor | None = None,
                           ws: torch.Tensor | None = None) -> TreeVerifyOutputs:
    """The accepted path and the emitted token of every request.

    target_probs and draft_probs [T, V] (float32 or bfloat16, last axis contiguous; draft_probs
    None for DRAFT_FIXED), tokens and parents [T] int32, u [T] and r [B] float64 in [0, 1)."""
    lib = _lib()
    dev = _device(target_probs, "target_probs")
    t_stride = _strided(target_probs, dev, 2, "target_probs")[0]
    T, V = target_probs.shape
    B = r.numel()
    dt = _dtype(target_probs, (torch.float32, torch.bfloat16), "target_probs")
    q, d_stride = None, 0
    if draft_probs is not None:
        d_stride = _strided(draft_probs, dev, 2, "draft_probs")[0]
        if draft_probs.shape != (T, V) or draft_probs.dtype is not target_probs.dtype:
            raise SpecVerifyError(f"draft_probs: want {target_probs.dtype} [{T}, {V}]")
        q = draft_probs.data_ptr()
    i32 = torch.int32
    _want(tokens, i32, (T,), dev, "tokens")
    _want(parents, i32, (T,), dev, "parents")
    _want(node_start, i32, (B + 1,), dev, "node_start")
    _want(u, torch.float64, (T,), dev, "u")
    _want(r, torch.float64, (B,), dev, "r")
    err = _optional(device_error, i32, (1,), dev, "device_error")
    width = max(max_path, 0)
    accept_len = torch.empty(B, dtype=i32, device=dev)
    path = torch.empty((B, width), dtype=i32, device=dev)
    emitted = torch.empty((B, width), dtype=i32, device=dev)
    out_token = torch.empty(B, dtype=i32, device=dev)
    ws = _scratch(ws, lib.specverify_tree_verify_workspace_size(B, V, max_nodes), dev,
                  "specverify_tree_verify_workspace_size")
    _call("specverify_tree_verify", dev, target_probs.data_ptr(), q, dt, mode, tokens.data_ptr(),
          parents.data_ptr(), node_start.data_ptr(), B, T, V, max_nodes, max_path, t_stride,
          d_stride, u.data_ptr(), r.data_ptr(), accept_len.data_ptr(), path.data_ptr(),
          emitted.data_ptr(), out_token.data_ptr(), err, ws.data_ptr(), ws.numel())
    return TreeVerifyOutputs(accept_len, path, emitted, out_token)


def specverify_tree_commit(k_tree: torch.Tensor, v_tree: torch.Tensor, k_cache: torch.Tensor,
                           v_cache: torch.Tensor, node_start: torch.Tensor, path: torch.Tensor,
                           accept_len: torch.Tensor, slots: torch.Tensor, prefix_len: torch.Tensor,
                           *, max_nodes: int = MAX_TREE_NODES, out: torch.Tensor | None = None,
                           device_error: torch.Tensor | None = None) -> torch.Tensor:
    """Writes the accepted nodes' keys and values of every layer into the caches and returns the
    new prefix lengths [B] int32 (into `out`, which may be prefix_len itself).

    k_tree and v_tree [layers, T, H, D], k_cache and v_cache [layers, num_pages, page_size, H, D]
    (float32, bfloat16 or float16, last axis contiguous, other strides multiples of 16 bytes)."""
    _lib()
    dev = _device(k_cache, "k_cache")
    ns = _pair(k_tree, v_tree, dev, 4, "k_tree and v_tree")
    cs = _pair(k_cache, v_cache, dev, 5, "k_cache and v_cache")
    L, T, H, D = k_tree.shape
    layers, num_pages, page_size, heads, width = k_cache.shape
    if layers != L or heads != H or width != D or k_cache.dtype is not k_tree.dtype:
        raise SpecVerifyError("k_tree [layers, T, H, D] and k_cache [layers, pages, page_size, H, "
                              "D] disagree")
    dt = _dtype(k_tree, tuple(_DTYPES), "k_tree")
    B = prefix_len.numel()
    max_path = path.shape[-1] if path.dim() else 0
    i32 = torch.int32
    _want(node_start, i32, (B + 1,), dev, "node_start")
    _want(path, i32, (B, max_path), dev, "path")
    _want(accept_len, i32, (B,), dev, "accept_len")
    _want(slots, torch.int64, (B, max_path), dev, "slots")
    _want(prefix_len, i32, (B,), dev, "prefix_len")
    if out is None:
        out = torch.empty(B, dtype=i32, device=dev)
    else:
        _want(out, i32, (B,), dev, "out")
    err = _optional(device_error, i32, (1,), dev, "device_error")
    _call("specverify_tree_commit", dev, k_tree.data_ptr(), v_tree.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), dt, L, B, T, H, D, max_nodes, max_path, ns[0], ns[1], ns[2], cs[0],
          cs[1], cs[2], cs[3], num_pages, page_size, node_start.data_ptr(), path.data_ptr(),
          accept_len.data_ptr(), slots.data_ptr(), prefix_len.data_ptr(), out.data_ptr(), err)
    return out
