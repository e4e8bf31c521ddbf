"""Python binding of the operators around a verification step (include/specverify_serving.h).

Argument marshalling only, as in the package: every step runs in the HIP kernels of
``libspecverify.so``; torch supplies device memory and the stream. A serving loop calls
``specverify_pages_resize``, then ``specverify_rotate`` and ``specverify_chunk_attention`` once per
layer, for the tokens of prompts; ``specverify_pages_fork`` for further replies to one prompt;
``specverify_rotate`` and ``specverify_penalize`` also around a step of drafted trees (``tree``).
None of them waits for the GPU, and all of them can be captured into a graph. They serve: nothing
here records gradients.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

import torch

from . import SV_F32, SpecVerifyError, load_library
from . import tree as _tree
from .tree import (_DTYPES, _device, _dtype, _optional, _pair, _scratch, _strided, _table, _want)

SV_ERR_REQUEST = 128
SV_ERR_PENALTY = 256
MAX_PAGE_BATCH = 1 << 16
MAX_CACHE_PAGES = 1 << 26

_P = ctypes.c_void_p
_I = ctypes.c_int64
_INT = ctypes.c_int
_SZ = ctypes.c_size_t

_SERVING_SIGNATURES = {
    "specverify_pages_resize_workspace_size": (_SZ, [_I] * 2),
    "specverify_pages_resize": (_INT, [_P] * 7 + [_I] * 7 + [_P] * 7 + [_SZ, _P]),
    "specverify_pages_fork_workspace_size": (_SZ, [_I] * 2),
    "specverify_pages_fork": (_INT, [_P] * 10 + [_INT] + [_I] * 14 + [_P] * 6 + [_SZ, _P]),
    "specverify_rotate": (_INT, [_P] * 3 + [_INT] + [_I] * 5 + [_INT] + [_I] * 4 +
                          [_P, _P, _INT, ctypes.c_float, _P, _P] + [_P, _I, _I] * 2 + [_P] * 3 +
                          [_I] * 5 + [_P] * 2),
    "specverify_chunk_attention_workspace_size": (_SZ, [_I] * 6),
    "specverify_chunk_attention": (_INT, [_P] * 3 + [_INT] + [_I] * 13 + [_P, _I, _I, _P, _P,
                                                                         ctypes.c_float, _P, _I, _I,
                                                                         _P, _P, _P, _SZ, _P]),
    "specverify_penalize": (_INT, [_P, _INT] + [_P] * 13 + [_I] * 10 + [_P, _INT, _P, _P]),
}

_bound = None


def _lib() -> ctypes.CDLL:
    global _bound
    lib = _tree._lib()
    if _bound is not lib:
        for name, (res, args) in _SERVING_SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _bound = lib
    return lib


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name: str, *sizes: int) -> int:
    return int(getattr(_lib(), name)(*sizes))


_call = _tree._call  # on the tensors' device, on its current stream


@dataclass
class PagesOutputs:
    pages: torch.Tensor              # [B] int32: pages owned now
    free_head: torch.Tensor          # [1] int32
    shares: torch.Tensor | None      # [num_pages] int32
    position: torch.Tensor | None    # [rows] int32
    slots: torch.Tensor | None       # [rows] int64
    prefix_len: torch.Tensor | None  # [B] int32 (a fork's)


def pages_resize_workspace(B: int, num_pages: int, device) -> torch.Tensor:
    n = int(_lib().specverify_pages_resize_workspace_size(B, num_pages))
    return _scratch(None, n, device, "specverify_pages_resize_workspace_size")


def specverify_pages_resize(prefix_len: torch.Tensor, pages: torch.Tensor,
                            block_table: torch.Tensor, free_pages: torch.Tensor,
                            free_head: torch.Tensor, *, page_size: int, num_pages: int,
                            chunk_start: torch.Tensor | None = None, rows: int = 0,
                            shares: torch.Tensor | None = None,
                            device_error: torch.Tensor | None = None,
                            ws: torch.Tensor | None = None) -> PagesOutputs:
    """Pages for every request's cached tokens (prefix_len [B]) and the new ones of its chunk
    (chunk_start [B + 1], `rows` in all; None: none), taken from free_pages[free_head:] or given
    back to it; positions and slots of the new tokens.

    block_table [B, max_pages] and free_pages [at least num_pages] are updated in place, pages,
    free_head and shares come back new. A request ends by prefix_len 0 and no new tokens."""
    _lib()
    dev = _device(prefix_len, "prefix_len")
    i32 = torch.int32
    B, free = prefix_len.numel(), free_pages.numel()
    _want(prefix_len, i32, (B,), dev, "prefix_len")
    _want(pages, i32, (B,), dev, "pages")
    _want(free_pages, i32, (free,), dev, "free_pages")
    _want(free_head, i32, (1,), dev, "free_head")
    start = _optional(chunk_start, i32, (B + 1,), dev, "chunk_start")
    held = _optional(shares, i32, (num_pages,), dev, "shares")
    err = _optional(device_error, i32, (1,), dev, "device_error")
    width, stride = _table(block_table, B, dev)
    if rows < 0 or (start is None and rows):
        raise SpecVerifyError("rows: new tokens want a chunk_start")
    empty = torch.empty
    now = empty(B, dtype=i32, device=dev)
    head = empty(1, dtype=i32, device=dev)
    left = None if shares is None else empty(num_pages, dtype=i32, device=dev)
    position = slots = None
    if start is not None:
        position = empty(rows, dtype=i32, device=dev)
        slots = empty(rows, dtype=torch.int64, device=dev)
    ws = _scratch(ws, _workspace_bytes("specverify_pages_resize_workspace_size", B, num_pages), dev,
                  "specverify_pages_resize_workspace_size")
    _call("specverify_pages_resize", dev, prefix_len.data_ptr(), start, pages.data_ptr(),
          block_table.data_ptr(), free_pages.data_ptr(), free_head.data_ptr(), held, B, rows,
          page_size, width, stride, num_pages, free, now.data_ptr(), head.data_ptr(),
          None if left is None else left.data_ptr(),
          None if position is None else position.data_ptr(),
          None if slots is None else slots.data_ptr(), err, ws.data_ptr(), ws.numel())
    return PagesOutputs(now, head, left, position, slots, None)


def pages_fork_workspace(B: int, forks: int, device) -> torch.Tensor:
    n = int(_lib().specverify_pages_fork_workspace_size(B, forks))
    return _scratch(None, n, device, "specverify_pages_fork_workspace_size")


def specverify_pages_fork(source: torch.Tensor, target: torch.Tensor, prefix_len: torch.Tensor,
                          pages: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                          free_head: torch.Tensor, shares: torch.Tensor, k_cache: torch.Tensor,
                          v_cache: torch.Tensor, *, device_error: torch.Tensor | None = None,
                          ws: torch.Tensor | None = None) -> PagesOutputs:
    """Request source[i]'s cache for request target[i], which owns nothing yet: its full pages are
    shared, the tokens of its last page copied in every layer into a page from the free list.

    source and target [forks] int32, k_cache and v_cache [layers, num_pages, page_size, H, D]
    (float32, bfloat16 or float16, last axis contiguous, other strides multiples of 16 bytes).
    block_table and the caches are updated in place, the rest comes back new."""
    _lib()
    dev = _device(k_cache, "k_cache")
    cs = _pair(k_cache, v_cache, dev, 5, "k_cache and v_cache")
    layers, num_pages, page_size, H, D = k_cache.shape
    dt = _dtype(k_cache, tuple(_DTYPES), "k_cache")
    i32 = torch.int32
    F, B, free = source.numel(), prefix_len.numel(), free_pages.numel()
    _want(source, i32, (F,), dev, "source")
    _want(target, i32, (F,), dev, "target")
    _want(prefix_len, i32, (B,), dev, "prefix_len")
    _want(pages, i32, (B,), dev, "pages")
    _want(free_pages, i32, (free,), dev, "free_pages")
    _want(free_head, i32, (1,), dev, "free_head")
    _want(shares, i32, (num_pages,), dev, "shares")
    width, stride = _table(block_table, B, dev)
    err = _optional(device_error, i32, (1,), dev, "device_error")
    empty = torch.empty
    length = empty(B, dtype=i32, device=dev)
    now = empty(B, dtype=i32, device=dev)
    head = empty(1, dtype=i32, device=dev)
    held = empty(num_pages, dtype=i32, device=dev)
    ws = _scratch(ws, _workspace_bytes("specverify_pages_fork_workspace_size", B, F), dev,
                  "specverify_pages_fork_workspace_size")
    _call("specverify_pages_fork", dev, source.data_ptr(), target.data_ptr(), prefix_len.data_ptr(),
          pages.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(), free_head.data_ptr(),
          shares.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), dt, F, B, layers, H, D, cs[0],
          cs[1], cs[2], cs[3], page_size, width, stride, num_pages, free, length.data_ptr(),
          now.data_ptr(), head.data_ptr(), held.data_ptr(), err, ws.data_ptr(), ws.numel())
    return PagesOutputs(now, head, held, None, None, length)


def specverify_rotate(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor | None,
                      position: torch.Tensor, inv_freq: torch.Tensor, *,
                      q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                      eps: float = 1e-6, interleaved: bool = False,
                      out_q: torch.Tensor | None = None, out_k: torch.Tensor | None = None,
                      slots: torch.Tensor | None = None, k_cache: torch.Tensor | None = None,
                      v_cache: torch.Tensor | None = None,
                      device_error: torch.Tensor | None = None):
    """(q [T, Hq, D], k [T, Hkv, D] or None): normed by head (weights [D], None for none) and
    rotated by position [T] int32 with inv_freq [R / 2] float32.

    With slots [T] int64 and k_cache, v_cache [num_pages, page_size, Hkv, D] the keys and v go into
    the cache, and k comes back only into a given out_k. q, k, v, outputs and cache are float32,
    bfloat16 or float16 with a contiguous last axis and other strides multiples of 16 bytes;
    out_q and out_k may be q and k."""
    _lib()
    dev = _device(q, "q")
    qs = _strided(q, dev, 3, "q")
    T, Hq, D = q.shape
    dt = _dtype(q, tuple(_DTYPES), "q")
    cached = k_cache is not None
    if cached != (v_cache is not None) or cached != (slots is not None) or (cached and v is None):
        raise SpecVerifyError("v, slots, k_cache and v_cache belong together")
    ks = _strided(k, dev, 3, "k") if v is None else _pair(k, v, dev, 3, "k and v")
    Hkv = k.shape[1]
    if k.shape != (T, Hkv, D) or k.dtype is not q.dtype:
        raise SpecVerifyError("q [T, Hq, D] and k [T, Hkv, D] disagree")
    _want(position, torch.int32, (T,), dev, "position")
    _want(inv_freq, torch.float32, (inv_freq.numel(),), dev, "inv_freq")
    wt = SV_F32
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            if w.dtype is not torch.float32:
                _want(w, q.dtype, (D,), dev, name)
            _want(w, w.dtype, (D,), dev, name)
            wt = _DTYPES[w.dtype]
    if q_weight is not None and k_weight is not None and q_weight.dtype is not k_weight.dtype:
        raise SpecVerifyError("q_weight and k_weight differ in type")
    if out_q is None:
        out_q = torch.empty((T, Hq, D), dtype=q.dtype, device=dev)
    elif out_q.shape != q.shape or out_q.dtype is not q.dtype:
        raise SpecVerifyError(f"out_q: want {q.dtype} [{T}, {Hq}, {D}]")
    if out_k is None and not cached:
        out_k = torch.empty((T, Hkv, D), dtype=q.dtype, device=dev)
    elif out_k is not None and (out_k.shape != k.shape or out_k.dtype is not q.dtype):
        raise SpecVerifyError(f"out_k: want {q.dtype} [{T}, {Hkv}, {D}]")
    qo = _strided(out_q, dev, 3, "out_q")
    ko = _strided(out_k, dev, 3, "out_k") if out_k is not None else (0, 0)
    cs, num_pages, page_size = (0, 0, 0), 0, 0
    if cached:
        cs = _pair(k_cache, v_cache, dev, 4, "k_cache and v_cache")
        num_pages, page_size = k_cache.shape[:2]
        if k_cache.shape[2:] != (Hkv, D) or k_cache.dtype is not q.dtype:
            raise SpecVerifyError("k [T, Hkv, D] and k_cache [pages, page_size, Hkv, D] disagree")
        _want(slots, torch.int64, (T,), dev, "slots")
    err = _optional(device_error, torch.int32, (1,), dev, "device_error")
    _call("specverify_rotate", dev, q.data_ptr(), k.data_ptr(), None if v is None else v.data_ptr(),
          dt, T, Hq, Hkv, D, 2 * inv_freq.numel(), int(interleaved), qs[0], qs[1], ks[0], ks[1],
          None if q_weight is None else q_weight.data_ptr(),
          None if k_weight is None else k_weight.data_ptr(), wt, eps, position.data_ptr(),
          inv_freq.data_ptr(), out_q.data_ptr(), qo[0], qo[1],
          None if out_k is None else out_k.data_ptr(), ko[0], ko[1],
          slots.data_ptr() if cached else None, k_cache.data_ptr() if cached else None,
          v_cache.data_ptr() if cached else None, cs[0], cs[1], cs[2], num_pages, page_size, err)
    return out_q, out_k


def chunk_attention_workspace(B: int, T: int, Hq: int, Hkv: int, D: int, max_chunk: int,
                              device) -> torch.Tensor:
    n = int(_lib().specverify_chunk_attention_workspace_size(B, T, Hq, Hkv, D, max_chunk))
    return _scratch(None, n, device, "specverify_chunk_attention_workspace_size")


def specverify_chunk_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               block_table: torch.Tensor, prefix_len: torch.Tensor,
                               chunk_start: torch.Tensor, *, max_chunk: int,
                               scale: float | None = None, out: torch.Tensor | None = None,
                               want_lse: bool = False, device_error: torch.Tensor | None = None,
                               ws: torch.Tensor | None = None):
    """(out [T, Hq, D], lse [T, Hq] float32 or None): the attention of chunks of new tokens, whose
    keys and values are in the cache already, over all that is cached up to each of them.

    q [T, Hq, D], k_cache and v_cache [num_pages, page_size, Hkv, D] (bfloat16 or float16, last axis
    contiguous, other strides multiples of 8 elements; the caches' strides agree), prefix_len [B]
    (the tokens in front) and chunk_start [B + 1] int32, max_chunk the longest chunk at most,
    scale 1 / sqrt(D) if not given."""
    _lib()
    dev = _device(q, "q")
    qs = _strided(q, dev, 3, "q")
    cs = _pair(k_cache, v_cache, dev, 4, "k_cache and v_cache")
    T, Hq, D = q.shape
    num_pages, page_size, Hkv, width = k_cache.shape
    B = prefix_len.numel()
    if width != D:
        raise SpecVerifyError("q [T, Hq, D] and k_cache [pages, page_size, Hkv, D] disagree")
    dt = _dtype(q, (torch.bfloat16, torch.float16), "q")
    if k_cache.dtype is not q.dtype:
        raise SpecVerifyError("q's and the cache's types differ")
    _want(prefix_len, torch.int32, (B,), dev, "prefix_len")
    _want(chunk_start, torch.int32, (B + 1,), dev, "chunk_start")
    max_pages, table_stride = _table(block_table, B, dev)
    if out is None:
        out = torch.empty((T, Hq, D), dtype=q.dtype, device=dev)
    elif out.shape != (T, Hq, D) or out.dtype is not q.dtype:
        raise SpecVerifyError(f"out: want {q.dtype} [{T}, {Hq}, {D}]")
    os_ = _strided(out, dev, 3, "out")
    err = _optional(device_error, torch.int32, (1,), dev, "device_error")
    lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if want_lse else None
    ws = _scratch(ws, _workspace_bytes("specverify_chunk_attention_workspace_size", B, T, Hq, Hkv, D,
                                       max_chunk), dev, "specverify_chunk_attention_workspace_size")
    _call("specverify_chunk_attention", dev, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          dt, B, T, Hq, Hkv, D, max_chunk, qs[0], qs[1], cs[0], cs[1], cs[2], num_pages, page_size,
          block_table.data_ptr(), max_pages, table_stride, prefix_len.data_ptr(),
          chunk_start.data_ptr(), D ** -0.5 if scale is None else scale, out.data_ptr(), os_[0],
          os_[1], lse.data_ptr() if want_lse else None, err, ws.data_ptr(), ws.numel())
    return out, lse


def specverify_penalize(logits: torch.Tensor, tokens: torch.Tensor, node_start: torch.Tensor,
                        history: torch.Tensor, prefix_len: torch.Tensor, prompt_len: torch.Tensor,
                        repetition: torch.Tensor, presence: torch.Tensor, frequency: torch.Tensor,
                        *, ancestors: torch.Tensor | None = None, max_nodes: int = 1,
                        bias_start: torch.Tensor | None = None,
                        bias_token: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                        mask: torch.Tensor | None = None, out: torch.Tensor | None = None,
                        device_error: torch.Tensor | None = None) -> torch.Tensor:
    """The logits [T, V] (float32 or bfloat16) of drafted nodes with their requests' penalties,
    biases and masks, into `out` (either type; may be `logits`).

    tokens [T] and node_start [B + 1] int32, ancestors [T, ceil(max_nodes / 64)] int64 or None for
    chains, history [B, max_history] int32 with prefix_len and prompt_len [B] int32, repetition,
    presence and frequency [B] float32, bias_start [B + 1] int32 with bias_token int32 and bias
    float32, mask [T, ceil(V / 32)] int32 (a bit 1 for an allowed id)."""
    _lib()
    dev = _device(logits, "logits")
    stride = _strided(logits, dev, 2, "logits")[0]
    T, V = logits.shape
    B = prefix_len.numel()
    types = (torch.float32, torch.bfloat16)
    dt = _dtype(logits, types, "logits")
    i32, f32 = torch.int32, torch.float32
    _want(tokens, i32, (T,), dev, "tokens")
    _want(node_start, i32, (B + 1,), dev, "node_start")
    _want(prefix_len, i32, (B,), dev, "prefix_len")
    _want(prompt_len, i32, (B,), dev, "prompt_len")
    for name, x in (("repetition", repetition), ("presence", presence), ("frequency", frequency)):
        _want(x, f32, (B,), dev, name)
    anc = _optional(ancestors, torch.int64, (T, (max_nodes + 63) // 64), dev, "ancestors")
    h_stride = _strided(history, dev, 2, "history")[0]
    if history.dtype is not i32 or history.shape[0] != B:
        raise SpecVerifyError(f"history: want int32 [{B}, max_history]")
    most = history.shape[1]
    if B > 1 and h_stride < most:
        raise SpecVerifyError(f"history: rows of {most} entries are {h_stride} apart")
    if (bias_start is None) != (bias is None) or (bias_start is None) != (bias_token is None):
        raise SpecVerifyError("bias_start, bias_token and bias belong together")
    N = 0 if bias is None else bias.numel()
    if N == 0:  # none at all
        bias_start = bias_token = bias = None
    bs = _optional(bias_start, i32, (B + 1,), dev, "bias_start")
    bt = _optional(bias_token, i32, (N,), dev, "bias_token")
    bv = _optional(bias, f32, (N,), dev, "bias")
    m_stride = 0
    if mask is not None:
        m_stride = _strided(mask, dev, 2, "mask")[0]
        if mask.dtype is not i32 or mask.shape != (T, (V + 31) // 32):
            raise SpecVerifyError(f"mask: want int32 [{T}, {(V + 31) // 32}]")
    if out is None:
        out = torch.empty((T, V), dtype=logits.dtype, device=dev)
    elif out.shape != (T, V):
        raise SpecVerifyError(f"out: want [{T}, {V}]")
    o_stride = _strided(out, dev, 2, "out")[0]
    if T <= 1:  # the stride of a single row says nothing
        stride, o_stride = (max(x, V) for x in (stride, o_stride))
        m_stride = max(m_stride, (V + 31) // 32)
        if out.data_ptr() == logits.data_ptr():
            o_stride = stride
    err = _optional(device_error, i32, (1,), dev, "device_error")
    _call("specverify_penalize", dev, logits.data_ptr(), dt, tokens.data_ptr(),
          node_start.data_ptr(), anc, history.data_ptr(), prefix_len.data_ptr(),
          prompt_len.data_ptr(), repetition.data_ptr(), presence.data_ptr(), frequency.data_ptr(),
          bs, bt, bv, None if mask is None else mask.data_ptr(), B, T, V, max_nodes, most, N, stride,
          o_stride, max(most, h_stride), m_stride, out.data_ptr(), _dtype(out, types, "out"), err)
    return out
