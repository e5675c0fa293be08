"""Attention over packed prompts over the C ABI (argument marshalling only)."""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from .api import _LAYOUTS, SAGE_ERR_LAYOUT, SAGE_ERR_SHAPE, SageError, _check, _get_device, _stream_handle
from .cache import SAGE_ERR_DTYPE, _call_workspace, _keep, _kept, _meta, _NAN, _on

SAGE_ERR_DEVICE_OFFSETS = -17


def _packed(t, what: str, layout: str, device):
    """(rows, heads, D) and the C tensor of a BF16 [rows, heads, D] tensor (or [heads, rows, D])."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected torch tensors")
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if t.device != device:
        raise ValueError(f"{what} must live on q's device")
    if t.dtype != torch.bfloat16:
        raise SageError(SAGE_ERR_DTYPE, "inputs and output must be bfloat16")
    if t.dim() != 3:
        raise SageError(SAGE_ERR_SHAPE, f"{what} must be 3-d: packed rows, heads and channels")
    sh, st = t.shape, t.stride()
    if st[2] != 1 and sh[2] != 1:
        raise SageError(SAGE_ERR_LAYOUT, "the channel stride must be 1")
    s, h = (0, 1) if layout == "NHD" else (1, 0)
    return (sh[s], sh[h], sh[2]), _lib.Bf16Tensor(t.data_ptr() or 16, 0, st[s], st[h])


def _offsets(t, n: int | None, device, what: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{what} must live on q's device")
    if t.dtype != torch.int32:
        raise SageError(SAGE_ERR_DTYPE, f"{what} must be int32")
    if t.dim() != 1 or t.shape[0] == 0 or (n is not None and t.shape[0] != n):
        raise SageError(SAGE_ERR_SHAPE, f"{what} must have one entry more than there are sequences")
    if not t.is_contiguous():
        raise SageError(SAGE_ERR_LAYOUT, f"{what} must be contiguous")
    return t.data_ptr()


def prompt_attention_workspace_size(N: int, M: int, H: int, H_kv: int, D: int = 128, B: int = 1) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.load().sage_prompt_attention_workspace_size(N, M, H, H_kv, D, B, ctypes.byref(n)))
    return n.value


def prompt_attention(q, k, v, offsets, kv_offsets=None, is_causal: bool = True, sm_scale=None, return_lse: bool = False,
                     tensor_layout: str = "NHD", out=None, workspace=None):
    """Attention over whole prompts of different lengths, packed one behind the other (sage_prompt_attention).

    q: BF16 [N, H, D], k and v: [M, H_kv, D] ("HND": [H, N, D], [H_kv, M, D]); query head h reads key/value head
    h // (H // H_kv). offsets: int32 [B + 1] on the device: sequence b's queries are rows offsets[b] ..
    offsets[b + 1] - 1, and its keys those of kv_offsets (None: the same). With is_causal the queries are the last of
    the sequence's tokens: of n queries and m keys row t sees keys 0 .. m - n + t. Returns out, or (out, lse) with lse
    fp32 [H, N], the natural-log log-sum-exp of each row's scaled logits. A row that sees no key gets 0 and -inf; rows
    behind the last sequence are the same, or left as they were in a given out (their lse is -inf all the same).

    out: a tensor to write to, which must not overlap q, k or v.

    With offsets that decrease or leave the tensors no row belongs to a sequence, and ``device_error()`` then returns
    SAGE_ERR_DEVICE_OFFSETS (-17). workspace: a uint8 tensor of prompt_attention_workspace_size bytes that no other
    call uses at the same time; None: the library's own, one for each thread and stream (a captured graph gets its own
    from its memory pool)."""
    kept = key = None
    if out is None and workspace is None:
        try:
            key = ("prompt", tensor_layout, bool(is_causal), bool(return_lse), q.shape, q.stride(), q.dtype, q.get_device(),
                   k.shape, k.stride(), k.dtype, k.get_device(), v.shape, v.stride(), v.dtype, v.get_device(),
                   offsets.shape, offsets.stride(), offsets.dtype, offsets.get_device(), _meta(kv_offsets))
            kept = _kept.calls.get(key)
        except (AttributeError, TypeError):
            key = None
    if kept is not None and kept[0] == _get_device():
        index, fn, ref, args, qi, ki, vi, oi, like, lse_shape, need = kept
        device = q.device
        out = torch.empty_like(q) if like else torch.empty(q.shape, dtype=torch.bfloat16, device=device)
        stream = _stream_handle(index)
        qi.ptr_dev, ki.ptr_dev, vi.ptr_dev, oi.ptr_dev = q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr()
        args.offsets_dev = offsets.data_ptr()
        if kv_offsets is not None:
            args.kv_offsets_dev = kv_offsets.data_ptr()
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
    if tensor_layout not in _LAYOUTS:
        raise SageError(SAGE_ERR_LAYOUT, "tensor_layout must be NHD or HND")
    if not isinstance(q, torch.Tensor):
        raise TypeError("expected torch tensors")
    device = q.device
    (N, H, D), qi = _packed(q, "q", tensor_layout, device)
    (M, Hkv, d), ki = _packed(k, "k", tensor_layout, device)
    shape, vi = _packed(v, "v", tensor_layout, device)
    if shape != (M, Hkv, d) or d != D:
        raise SageError(SAGE_ERR_SHAPE, "k and v must have one shape and q's head dimension")
    if H % Hkv if Hkv else H:
        raise SageError(SAGE_ERR_SHAPE, "the query heads must be a multiple of the key/value heads")
    off = _offsets(offsets, None, device, "offsets")
    B = offsets.shape[0] - 1
    kv_off = None if kv_offsets is None else _offsets(kv_offsets, B + 1, device, "kv_offsets")
    given = out is not None
    if not given:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=device)
    shape, oi = _packed(out, "out", tensor_layout, device)
    if shape != (N, H, D):
        raise SageError(SAGE_ERR_SHAPE, "out must have q's shape")
    lse = None
    if return_lse:
        lse = (torch.full if given else torch.empty)((H, N), *((float("-inf"),) if given else ()), dtype=torch.float32,
                                                     device=device)
    need = prompt_attention_workspace_size(N, M, H, Hkv, D, B)  # refuses sizes, too
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor):
            raise TypeError("workspace must be a torch tensor")
        if workspace.device != device:
            raise ValueError("workspace must live on q's device")
        if not workspace.is_contiguous():
            raise SageError(SAGE_ERR_LAYOUT, "workspace must be contiguous")
    if out.numel() == 0:
        return (out, lse) if return_lse else out
    index = q.get_device()
    args = _lib.PromptAttentionArgs(qi, ki, vi, oi, N, M, H, Hkv, D, B, off, kv_off,
                                    _NAN if sm_scale is None else float(sm_scale), bool(is_causal), not given,
                                    lse.data_ptr() if return_lse else None)
    with _on(index) as stream:
        if workspace is None and need:
            workspace = _call_workspace(device, stream, need)
        if workspace is not None:
            args.workspace_dev = workspace.data_ptr()
            args.workspace_bytes = workspace.numel() * workspace.element_size()
        args.cuda_stream = stream
        _check(_lib.load().sage_prompt_attention(ctypes.byref(args)))
    if key is not None and k.numel():
        if need:
            args.workspace_bytes = need
        _keep(key, (index, _lib.load().sage_prompt_attention, ctypes.byref(args), args, args.q, args.k, args.v, args.out,
                    q.is_contiguous(), (H, N), need))
    return (out, lse) if return_lse else out
