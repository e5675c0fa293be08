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
import threading
from dataclasses import dataclass, field

import torch

from . import _lib
from .api import (_LAYOUTS, SAGE_ERR_LAYOUT, SAGE_ERR_SHAPE, SageError, _check, _get_device, _stream_handle, _workspace)

SAGE_ERR_DTYPE = -3
SAGE_ERR_DEVICE_PAGE = -16

BLOCK = 32  # tokens that share a scale


def _signature(*sizes) -> tuple:
    """What stands for a cache in the keys of kept calls, which are not checked again: all its
    sizes and its device. The sizes themselves: a number given out for them would have to be
    the same for all threads, whoever asks first."""
    return sizes


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
    address: int = field(init=False, repr=False)   # of c, which lives as long as the object
    signature: tuple = field(init=False, repr=False)  # the same for caches of the same sizes on one device

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
        c = _lib.Cache(*(t.data_ptr() or 16 for t in ts), P, n * BLOCK, H, D)  # an empty array has no address
        for name, value in (("c", c), ("address", ctypes.addressof(c)), ("signature", _signature(P, n, H, D, self.k_codes.get_device()))):
            object.__setattr__(self, name, value)

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
        if self.index != _get_device():
            self.ctx = torch.cuda.device(self.index)
            self.ctx.__enter__()
        return _stream_handle(self.index)

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


# A call whose shapes, strides, types, devices and flags this thread has seen
# before skips the checks: the thread keeps one filled argument struct for each
# such signature and changes only the pointers (answering token by token, a
# call's host work counts; the signatures are written out flat for the same
# reason). Per thread, so that no other thread rewrites a struct while the
# library reads it. Calls that give out or workspace, and page copies, go the
# full way (attention with out: 12 us of host time, 9.4 without).


def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


class _Kept(threading.local):
    def __init__(self):  # once in each thread
        self.calls = {}


_kept = _Kept()


def _keep(key, value):
    calls = _kept.calls
    if len(calls) > 256:
        calls.clear()
    calls[key] = value


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


def _table(t, B: int, cache: QuantizedCache):
    """(address, row stride, entries of a row) of an int32 [B, max_pages] page table."""
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
    return t.data_ptr() or cache.address, t.stride(0) if n else 0, n


def _tokens(t, cache: QuantizedCache, layout: str, what: str):
    """(B, T, heads) and the C tensor of a BF16 [B, T, heads, D] tensor (or [B, heads, T, D])."""
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
    if layout == "NHD":
        return (sh[0], sh[1], sh[2]), _lib.Bf16Tensor(t.data_ptr(), st[0], st[1], st[2])
    return (sh[0], sh[2], sh[1]), _lib.Bf16Tensor(t.data_ptr(), st[0], st[2], st[1])


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
    try:
        key = ("append", cache.signature, tensor_layout, k.shape, k.stride(), k.dtype, k.get_device(), v.shape, v.stride(),
               v.dtype, v.get_device(), page_table.shape, page_table.stride(), page_table.dtype, page_table.get_device(),
               starts.shape, starts.stride(), starts.dtype, starts.get_device(), _meta(counts))
        kept = _kept.calls.get(key)
    except (AttributeError, TypeError):
        key = kept = None
    if kept is not None and kept[0] == _get_device():
        index, fn, ref, args, ki, vi = kept
        args.cache = cache.address
        args.table_dev = page_table.data_ptr()
        args.starts_dev = starts.data_ptr()
        if counts is not None:
            args.counts_dev = counts.data_ptr()
        ki.ptr_dev = k.data_ptr()
        vi.ptr_dev = v.data_ptr()
        args.cuda_stream = _stream_handle(index)
        rc = fn(ref)
        if rc:
            _check(rc)
        return
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
    if k.numel() == 0:
        return
    index = cache.k_codes.get_device()
    args = _lib.CacheAppendArgs(cache.address, *table, st, ct, ki, vi, B, T)
    with _on(index) as stream:
        args.cuda_stream = stream
        _check(_lib.load().sage_cache_append(ctypes.byref(args)))
    if key is not None and table[2]:
        _keep(key, (index, _lib.load().sage_cache_append, ctypes.byref(args), args, args.k, args.v))


def cache_read(cache: QuantizedCache, page_table, starts, T: int, counts=None, tensor_layout: str = "NHD", out=None):
    """Reads tokens starts[b] .. starts[b] + counts[b] - 1 of each sequence back as BF16
    (sage_cache_read); counts None: T tokens each. Returns (k, v), each [B, T, H, D];
    rows counts[b] and up are 0, or left as they were in the tensors given as out."""
    kept = key = None
    if out is None:
        try:
            key = ("read", cache.signature, tensor_layout, T, page_table.shape, page_table.stride(), page_table.dtype,
                   page_table.get_device(), starts.shape, starts.stride(), starts.dtype, starts.get_device(), _meta(counts))
            kept = _kept.calls.get(key)
        except (AttributeError, TypeError):
            key = None
    if kept is not None and kept[0] == _get_device():
        index, fn, ref, args, ko, vo, shape = kept
        k = torch.empty(shape, dtype=torch.bfloat16, device=page_table.device)
        v = torch.empty_like(k)
        args.cache = cache.address
        args.table_dev = page_table.data_ptr()
        args.starts_dev = starts.data_ptr()
        if counts is not None:
            args.counts_dev = counts.data_ptr()
        ko.ptr_dev = k.data_ptr()
        vo.ptr_dev = v.data_ptr()
        args.cuda_stream = _stream_handle(index)
        rc = fn(ref)
        if rc:
            _check(rc)
        return k, v
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
    shape = (B, T, cache.H, cache.D) if tensor_layout == "NHD" else (B, cache.H, T, cache.D)
    zero_rest = out is None
    if out is None:
        out = [torch.empty(shape, dtype=torch.bfloat16, device=cache.k_codes.device) for _ in (0, 1)]
    k, v = out
    ks, ko = _tokens(k, cache, tensor_layout, "out")
    vs, vo = _tokens(v, cache, tensor_layout, "out")
    if ks != (B, T, cache.H) or vs != ks:
        raise SageError(SAGE_ERR_SHAPE, "out must be two tensors [B, T, H, D]")
    if k.numel() == 0:
        return k, v
    index = cache.k_codes.get_device()
    args = _lib.CacheReadArgs(cache.address, *table, st, ct, ko, vo, B, T, zero_rest)
    with _on(index) as stream:
        args.cuda_stream = stream
        _check(_lib.load().sage_cache_read(ctypes.byref(args)))
    if key is not None and table[2]:
        _keep(key, (index, _lib.load().sage_cache_read, ctypes.byref(args), args, args.k_out, args.v_out, shape))
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
        _check(_lib.load().sage_cache_copy_pages(cache.address, s, d, n, stream))


_NAN = float("nan")


def _call_workspace(device, stream: int, need: int) -> torch.Tensor:
    """The thread's workspace for its calls on this stream, or one from the captured graph's
    memory pool: a replay may run beside other calls."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(need, dtype=torch.uint8, device=device)
    return _workspace(device, stream, need)


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

    The call is planned for page_table's width, since the lengths are on the device: for a
    small call, a view of its first columns that the longest sequence needs is quicker than
    a table of many times that width.

    workspace: a uint8 tensor of cache_attention_workspace_size bytes (4 to 43 MB) that no
    other call uses at the same time; None: the library's own, one for each thread and
    stream (a captured graph gets its own from its memory pool)."""
    kept = key = None
    if out is None and workspace is None:
        try:
            key = ("attention", cache.signature, tensor_layout, bool(is_causal), bool(return_lse), q.shape, q.stride(),
                   q.dtype, q.get_device(), page_table.shape, page_table.stride(), page_table.dtype,
                   page_table.get_device(), lengths.shape, lengths.stride(), lengths.dtype, lengths.get_device(),
                   _meta(q_lengths))
            kept = _kept.calls.get(key)
        except (AttributeError, TypeError):
            key = None
    if kept is not None and kept[0] == _get_device():
        index, fn, ref, args, qi, oi, shape, lse_shape, need = kept
        device = q.device
        out = torch.empty_like(q) if shape is None else torch.empty(shape, dtype=torch.bfloat16, device=device)
        stream = _stream_handle(index)
        args.cache = cache.address
        args.table_dev = page_table.data_ptr()
        args.lengths_dev = lengths.data_ptr()
        if q_lengths is not None:
            args.q_lengths_dev = q_lengths.data_ptr()
        qi.ptr_dev = q.data_ptr()
        oi.ptr_dev = out.data_ptr()
        args.sm_scale = _NAN if sm_scale is None else float(sm_scale)
        if need:
            workspace = _call_workspace(device, stream, need)
            args.workspace_dev = workspace.data_ptr()
        args.cuda_stream = stream
        lse = None
        if return_lse:
            lse = torch.empty(lse_shape, dtype=torch.float32, device=device)
            args.lse_dev = lse.data_ptr()
        rc = fn(ref)
        if rc:
            _check(rc)
        return (out, lse) if return_lse else out
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
    zero_rest = out is None
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=device)
    shape, oi = _tokens(out, cache, tensor_layout, "out")
    if shape != (B, T, H):
        raise SageError(SAGE_ERR_SHAPE, "out must have q's shape")
    # with a given out, padding rows of the log-sum-exp are -inf all the same
    lse = None
    if return_lse:
        if zero_rest or q_lengths is None:
            lse = torch.empty((B, H, T), dtype=torch.float32, device=device)
        else:
            lse = torch.full((B, H, T), float("-inf"), dtype=torch.float32, device=device)
    if out.numel() == 0:
        return (out, lse) if return_lse else out
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor):
            raise TypeError("workspace must be a torch tensor")
        if workspace.device != device:
            raise ValueError("workspace must live on the cache's device")
        if not workspace.is_contiguous():
            raise SageError(SAGE_ERR_LAYOUT, "workspace must be contiguous")
    index = cache.k_codes.get_device()
    need = cache_attention_workspace_size(B, T, H, Hkv, cache.D)
    args = _lib.CacheAttentionArgs(cache.address, *table, lens, q_lens, qi, oi, B, T, H,
                                   _NAN if sm_scale is None else float(sm_scale), bool(is_causal), zero_rest,
                                   lse.data_ptr() if return_lse else None)
    with _on(index) as stream:
        if workspace is None and need:
            workspace = _call_workspace(device, stream, need)
        if workspace is not None:
            args.workspace_dev = workspace.data_ptr()
            args.workspace_bytes = workspace.numel() * workspace.element_size()
        args.cuda_stream = stream
        _check(_lib.load().sage_cache_attention(ctypes.byref(args)))
    if key is not None and table[2]:
        if need:
            args.workspace_bytes = need
        _keep(key, (index, _lib.load().sage_cache_attention, ctypes.byref(args), args, args.q, args.out,
                    None if q.is_contiguous() else q.shape, (B, H, T), need))
    return (out, lse) if return_lse else out
