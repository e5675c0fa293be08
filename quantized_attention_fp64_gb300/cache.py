"""The 8-bit paged key/value cache over the C ABI (argument marshalling only).

A cache keeps the keys and values of growing sequences as int8 codes with one
fp32 scale for each block of 32 tokens and head, in pages that a page table
hands out to the sequences: ``cache_append`` writes new tokens,
``cache_attention`` lets queries attend to them (decoding, chunks of a prompt,
cross attention to an encoder's states), ``cache_read`` reads tokens back and
``cache_copy_pages`` moves pages. Which page belongs to whom is the caller's
bookkeeping. Every step runs in the library's CUDA kernels.

Page tables, lengths, starts, counts and page lists are int32 CUDA tensors, so
a captured CUDA graph can be replayed while a program changes them. What they
hold is checked on the device: a length that reaches past the table is cut, a
page number outside the cache counts as a page without tokens, and
``device_error()`` then returns SAGE_ERR_DEVICE_PAGE (-16).
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass, field

import torch

from . import _lib
from .api import (_LAYOUTS, SAGE_ERR_LAYOUT, SAGE_ERR_SHAPE, SageError, _check, _stream_handle, _workspace)

SAGE_ERR_DTYPE = -3
SAGE_ERR_DEVICE_PAGE = -16

BLOCK = 32  # tokens that share a scale


@dataclass(frozen=True, eq=False)
class QuantizedCache:
    """The cache's four arrays (see sage_cache): one object for all sequences of a layer."""

    k_codes: torch.Tensor   # int8 [num_pages, H, page_size/32, D/64, 32, 64]
    v_codes: torch.Tensor   # int8 [num_pages, H, page_size/32, D, 32]
    k_scale: torch.Tensor   # float32 [num_pages, H, page_size/32]
    v_scale: torch.Tensor   # float32 [num_pages, H, page_size/32]
    num_pages: int = field(init=False)
    page_size: int = field(init=False)
    H: int = field(init=False)
    D: int = field(init=False)
    c: _lib.Cache = field(init=False, repr=False)

    def __post_init__(self):
        ts = (self.k_codes, self.v_codes, self.k_scale, self.v_scale)
        for t, dtype in zip(ts, (torch.int8, torch.int8, torch.float32, torch.float32)):
            if not isinstance(t, torch.Tensor):
                raise TypeError("expected torch tensors")
            if not t.is_cuda or t.device != self.k_codes.device:
                raise ValueError("the cache's tensors must live on one CUDA device")
            if t.dtype != dtype:
                raise SageError(SAGE_ERR_DTYPE, "codes must be int8 and scales float32")
            if not t.is_contiguous():
                raise SageError(SAGE_ERR_LAYOUT, "the cache's tensors must be contiguous")
        if self.v_codes.dim() != 5:
            raise SageError(SAGE_ERR_SHAPE, "v_codes must be [num_pages, H, page_size/32, D, 32]")
        P, H, n, D, _ = self.v_codes.shape
        if (tuple(self.v_codes.shape) != (P, H, n, D, BLOCK)
                or tuple(self.k_codes.shape) != (P, H, n, D // 64, BLOCK, 64)
                or tuple(self.k_scale.shape) != (P, H, n) or tuple(self.v_scale.shape) != (P, H, n)):
            raise SageError(SAGE_ERR_SHAPE, "codes and scales do not belong to one cache")
        # sizes the library refuses (head dimension, pages) are refused here, once
        _check(_lib.load().sage_cache_size(P, n * BLOCK, H, D, ctypes.byref(ctypes.c_size_t(0)), None, None))
        for name, value in (("num_pages", P), ("page_size", n * BLOCK), ("H", H), ("D", D)):
            object.__setattr__(self, name, value)
        object.__setattr__(self, "c", _lib.Cache(*(t.data_ptr() for t in ts), P, n * BLOCK, H, D))

    @property
    def device(self) -> torch.device:
        return self.k_codes.device


def alloc_cache(num_pages: int, H: int, device, D: int = 128, page_size: int = 64) -> QuantizedCache:
    """An empty cache of num_pages pages of page_size tokens (a multiple of 32)."""
    n = ctypes.c_size_t(0)
    _check(_lib.load().sage_cache_size(num_pages, page_size, H, D, ctypes.byref(n), None, None))
    nb = page_size // BLOCK
    return QuantizedCache(
        k_codes=torch.zeros((num_pages, H, nb, D // 64, BLOCK, 64), dtype=torch.int8, device=device),
        v_codes=torch.zeros((num_pages, H, nb, D, BLOCK), dtype=torch.int8, device=device),
        k_scale=torch.zeros((num_pages, H, nb), dtype=torch.float32, device=device),
        v_scale=torch.zeros((num_pages, H, nb), dtype=torch.float32, device=device))


class _on:
    """The cache's device as the current one for the call, without cost where it is already."""

    __slots__ = ("index", "ctx")

    def __init__(self, index: int):
        self.index, self.ctx = index, None

    def __enter__(self):
        if self.index != torch.cuda.current_device():
            self.ctx = torch.cuda.device(self.index)
            self.ctx.__enter__()
        return _stream_handle(self.index)

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _ints(t, n: int | None, cache: QuantizedCache, what: str):
    """Address of an int32 vector of n entries on the cache's device (None: NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch tensor")
    if t.device != cache.k_codes.device:
        raise ValueError(f"{what} must live on the cache's device")
    if t.dtype != torch.int32:
        raise SageError(SAGE_ERR_DTYPE, f"{what} must be int32")
    if t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise SageError(SAGE_ERR_SHAPE, f"{what} must have one entry for each sequence")
    if not t.is_contiguous():
        raise SageError(SAGE_ERR_LAYOUT, f"{what} must be contiguous")
    return t.data_ptr()


def _table(t, B: int, cache: QuantizedCache) -> _lib.PageTable:
    if not isinstance(t, torch.Tensor):
        raise TypeError("page_table must be a torch tensor")
    if t.device != cache.k_codes.device:
        raise ValueError("page_table must live on the cache's device")
    if t.dtype != torch.int32:
        raise SageError(SAGE_ERR_DTYPE, "page_table must be int32")
    if t.dim() != 2 or t.shape[0] != B:
        raise SageError(SAGE_ERR_SHAPE, "page_table must be [B, max_pages]")
    n = t.shape[1]
    if n > 1 and t.stride(1) != 1:
        raise SageError(SAGE_ERR_LAYOUT, "the page table's rows must be contiguous")
    # an empty table has no address: any aligned one does, it is not read
    return _lib.PageTable(t.data_ptr() or cache.k_codes.data_ptr(), t.stride(0) if n else 0, n)


def _tokens(t, cache: QuantizedCache, layout: str, what: str):
    """(B, T, heads) and (pointer, strides) of a BF16 [B, T, heads, D] tensor (or [B, heads, T, D])."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected torch tensors")
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if t.device != cache.k_codes.device:
        raise ValueError(f"{what} must live on the cache's device")
    if t.dtype != torch.bfloat16:
        raise SageError(SAGE_ERR_DTYPE, "inputs and output must be bfloat16")
    if t.dim() != 4 or t.shape[3] != cache.D:
        raise SageError(SAGE_ERR_SHAPE, f"{what} must be 4-d with the cache's head dimension")
    st = t.stride()
    if st[3] != 1:
        raise SageError(SAGE_ERR_LAYOUT, "the channel stride must be 1")
    sh = t.shape
    # an empty tensor has no address: it is not read
    ptr = t.data_ptr() or cache.k_codes.data_ptr()
    if layout == "NHD":
        return (sh[0], sh[1], sh[2]), (ptr, st[0], st[1], st[2])
    return (sh[0], sh[2], sh[1]), (ptr, st[0], st[2], st[1])


def _check_layout(layout: str):
    if layout not in _LAYOUTS:
        raise SageError(SAGE_ERR_LAYOUT, "tensor_layout must be NHD or HND")


def _check_cache(cache):
    if not isinstance(cache, QuantizedCache):
        raise TypeError("expected a QuantizedCache")


def cache_append(cache: QuantizedCache, k, v, page_table, starts, counts=None, tensor_layout: str = "NHD") -> None:
    """Writes new tokens into the cache (sage_cache_append): tokens 0 .. counts[b] - 1
    of k and v ([B, T, H, D] BF16) become tokens starts[b] .. of sequence b, whose pages
    page_table[b] names. counts None: T tokens for each sequence. A block's scale grows
    with its tokens; older codes of the block are then rounded again. Tokens behind the
    last new one in its block are lost, so a sequence may be cut back and written on.
    The pages written must belong to one sequence only."""
    _check_cache(cache)
    _check_layout(tensor_layout)
    (B, T, H), ki = _tokens(k, cache, tensor_layout, "k")
    shape, vi = _tokens(v, cache, tensor_layout, "v")
    if shape != (B, T, H) or H != cache.H:
        raise SageError(SAGE_ERR_SHAPE, "k and v must be [B, T, H, D] with the cache's heads")
    table = _table(page_table, B, cache)
    if starts is None:
        raise TypeError("starts must be a torch tensor")
    st, ct = _ints(starts, B, cache, "starts"), _ints(counts, B, cache, "counts")
    if B == 0:
        return
    with _on(cache.k_codes.get_device()) as stream:
        _check(_lib.load().sage_cache_append(cache.c, table, st, ct, _lib.Bf16Tensor(*ki), _lib.Bf16Tensor(*vi), B, T,
                                             stream))


def cache_read(cache: QuantizedCache, page_table, starts, T: int, counts=None, tensor_layout: str = "NHD", out=None):
    """Reads tokens starts[b] .. starts[b] + counts[b] - 1 of each sequence back as BF16
    (sage_cache_read); counts None: T tokens each. Returns (k, v), each [B, T, H, D];
    rows counts[b] and up are 0, or left as they were in the tensors given as out."""
    _check_cache(cache)
    _check_layout(tensor_layout)
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise SageError(SAGE_ERR_SHAPE, "page_table must be [B, max_pages]")
    B, T = page_table.shape[0], int(T)
    if T < 0:
        raise SageError(SAGE_ERR_SHAPE, "T must not be negative")
    table = _table(page_table, B, cache)
    if starts is None:
        raise TypeError("starts must be a torch tensor")
    st, ct = _ints(starts, B, cache, "starts"), _ints(counts, B, cache, "counts")
    device = cache.k_codes.device
    if out is None:
        shape = (B, T, cache.H, cache.D) if tensor_layout == "NHD" else (B, cache.H, T, cache.D)
        if counts is None:
            out = tuple(torch.empty(shape, dtype=torch.bfloat16, device=device) for _ in (0, 1))
        else:
            out = tuple(torch.zeros((2,) + shape, dtype=torch.bfloat16, device=device))
    k, v = out
    ks, ko = _tokens(k, cache, tensor_layout, "out")
    vs, vo = _tokens(v, cache, tensor_layout, "out")
    if ks != (B, T, cache.H) or vs != ks:
        raise SageError(SAGE_ERR_SHAPE, "out must be two tensors [B, T, H, D]")
    if B:
        with _on(cache.k_codes.get_device()) as stream:
            _check(_lib.load().sage_cache_read(cache.c, table, st, ct, B, T, *ko, *vo, stream))
    return k, v


def cache_copy_pages(cache: QuantizedCache, src, dst) -> None:
    """Copies page src[i] to page dst[i] for every i (sage_cache_copy_pages): codes and
    scales of all heads. src, dst: int32 CUDA vectors of one length. An entry with
    dst < 0 or dst == src stands for nothing. No page may be named twice in dst, nor be
    in dst and the src of another entry; lists that break this copy nothing and set the
    device error word."""
    _check_cache(cache)
    if src is None or dst is None:
        raise TypeError("src and dst must be torch tensors")
    s = _ints(src, None, cache, "src")
    n = src.shape[0]
    d = _ints(dst, n, cache, "dst")
    if n == 0:
        return
    with _on(cache.k_codes.get_device()) as stream:
        _check(_lib.load().sage_cache_copy_pages(cache.c, s, d, n, stream))


def cache_attention_workspace_size(B: int, T: int, H: int, H_kv: int, D: int = 128) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.load().sage_cache_attention_workspace_size(B, T, H, H_kv, D, ctypes.byref(n)))
    return n.value


def cache_attention(q, cache: QuantizedCache, page_table, lengths, q_lengths=None, is_causal: bool = False,
                    sm_scale=None, return_lse: bool = False, tensor_layout: str = "NHD", out=None, workspace=None):
    """Attention of q ([B, T, H, D] BF16) to the cache (sage_cache_attention): sequence b
    has lengths[b] tokens there; query head h reads key/value head h // (H // cache.H).
    With is_causal the queries are the sequence's last tokens (already appended): row t
    sees the tokens up to lengths[b] - q_lengths[b] + t; otherwise every row sees all.
    q_lengths None: T queries for each sequence. A row that sees no token gets 0 and a
    log-sum-exp of -inf; rows q_lengths[b] and up are the same, or left as they were in a
    given out. Returns out, or (out, lse) with lse fp32 [B, H, T], the natural-log
    log-sum-exp of each row's scaled logits.

    workspace: a uint8 tensor of cache_attention_workspace_size bytes that no other call
    uses at the same time; None: the library's own, one for each thread and stream (a
    captured graph gets its own from its memory pool)."""
    _check_cache(cache)
    _check_layout(tensor_layout)
    (B, T, H), qi = _tokens(q, cache, tensor_layout, "q")
    Hkv = cache.H
    if H % Hkv if Hkv else H:
        raise SageError(SAGE_ERR_SHAPE, "the query heads must be a multiple of the cache's heads")
    table = _table(page_table, B, cache)
    if lengths is None:
        raise TypeError("lengths must be a torch tensor")
    lens, q_lens = _ints(lengths, B, cache, "lengths"), _ints(q_lengths, B, cache, "q_lengths")
    device = cache.k_codes.device
    if out is None:
        make = torch.empty if q_lengths is None else torch.zeros
        out = make(q.shape, dtype=torch.bfloat16, device=device)
    shape, oi = _tokens(out, cache, tensor_layout, "out")
    if shape != (B, T, H):
        raise SageError(SAGE_ERR_SHAPE, "out must have q's shape")
    lse = None
    if return_lse:
        if q_lengths is None:
            lse = torch.empty((B, H, T), dtype=torch.float32, device=device)
        else:
            lse = torch.full((B, H, T), float("-inf"), dtype=torch.float32, device=device)
    if out.numel() == 0:
        return (out, lse) if return_lse else out
    lib = _lib.load()
    with _on(cache.k_codes.get_device()) as stream:
        n = cache_attention_workspace_size(B, T, H, Hkv, cache.D)
        if workspace is None and n:
            if torch.cuda.is_current_stream_capturing():
                workspace = torch.empty(n, dtype=torch.uint8, device=device)
            else:
                workspace = _workspace(device, stream, n)
        elif workspace is not None and workspace.device != device:
            raise ValueError("workspace must live on the cache's device")
        _check(lib.sage_cache_attention(
            cache.c, table, lens, q_lens, _lib.Bf16Tensor(*qi), B, T, H,
            float("nan") if sm_scale is None else float(sm_scale), bool(is_causal), *oi,
            lse.data_ptr() if return_lse else None, workspace.data_ptr() if workspace is not None else None,
            workspace.numel() * workspace.element_size() if workspace is not None else 0, stream))
    return (out, lse) if return_lse else out
