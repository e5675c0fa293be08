"""Rotary positions over the C ABI (argument marshalling only).

``rotary_table`` makes the frequencies of a model once; ``rotary`` turns a
step's queries and keys by their positions, before ``prompt_attention``,
``cache_append`` or ``cache_attention`` take them.
"""

from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass, field

import torch

from . import _lib
from .api import _LAYOUTS, SAGE_ERR_LAYOUT, SAGE_ERR_SHAPE, SageError, _check, _get_device, _stream_handle
from .cache import SAGE_ERR_DTYPE, _keep, _kept, _on

SAGE_ERR_ARG = -13


@dataclass(frozen=True, eq=False)
class RotaryTable:
    """Frequencies of ``rotary_dim`` channels as the kernel takes them (see sage_rotary_turns)."""

    turns: torch.Tensor      # int64 [rotary_dim / 2]: the part of a turn that a position adds, in 2^-64
    inv_freq: torch.Tensor   # float64 [rotary_dim / 2], on the host: the same in radians
    magnitude: float = 1.0   # factor of every turned channel
    rotary_dim: int = field(init=False)

    def __post_init__(self):
        t = self.turns
        if not isinstance(t, torch.Tensor):
            raise TypeError("expected torch tensors")
        if not t.is_cuda:
            raise ValueError("turns must live on a CUDA device")
        if t.dtype != torch.int64:
            raise SageError(SAGE_ERR_DTYPE, "turns must be int64")
        if t.dim() != 1 or t.shape[0] == 0 or t.shape[0] % 8:
            raise SageError(SAGE_ERR_SHAPE, "turns must be a vector of a multiple of 8 entries")
        if not t.is_contiguous():
            raise SageError(SAGE_ERR_LAYOUT, "turns must be contiguous")
        object.__setattr__(self, "rotary_dim", 2 * t.shape[0])

    @property
    def device(self) -> torch.device:
        return self.turns.device


def rotary_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                    original_length: int | None = None, fast_turns: float = 32.0, slow_turns: float = 1.0) -> torch.Tensor:
    """float64 [rotary_dim / 2]: base^(-2i / rotary_dim), scaled for contexts ``factor`` times as long.

    scaling None: as they are. "linear": all divided by factor (positions interpolated). "ntk": the base times
    factor^(rotary_dim / (rotary_dim - 2)), so that the slowest pair is divided by factor and the fastest is left.
    "yarn": by parts: pairs that make fast_turns turns or more within original_length are left, those that make
    slow_turns or fewer are divided by factor, and those between are blended linearly in their number."""
    if rotary_dim <= 0 or rotary_dim % 2:
        raise SageError(SAGE_ERR_ARG, "rotary_dim must be positive and even")
    if not (math.isfinite(base) and base > 0.0) or not (math.isfinite(factor) and factor > 0.0):
        raise SageError(SAGE_ERR_ARG, "base and factor must be finite and positive")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise SageError(SAGE_ERR_ARG, 'scaling must be None, "linear", "ntk" or "yarn"')
    if scaling is None and factor != 1.0:
        raise SageError(SAGE_ERR_ARG, "a factor needs a scaling")
    if scaling == "ntk":
        if rotary_dim <= 2:
            raise SageError(SAGE_ERR_ARG, "ntk scaling needs a rotary_dim above 2")
        base = base * factor ** (rotary_dim / (rotary_dim - 2.0))
    half = rotary_dim // 2
    w = torch.tensor([base ** (-2.0 * i / rotary_dim) for i in range(half)], dtype=torch.float64)
    if scaling == "linear":
        return w / factor
    if scaling != "yarn":
        return w
    if original_length is None or original_length <= 0:
        raise SageError(SAGE_ERR_ARG, "yarn scaling needs the original_length")
    if base == 1.0 or not 0.0 < slow_turns <= fast_turns:
        raise SageError(SAGE_ERR_ARG, "yarn scaling needs a base other than 1 and 0 < slow_turns <= fast_turns")

    def pair(turns: float) -> float:
        # base^(-2i / rotary_dim) * original_length = 2 pi turns, solved for i
        return rotary_dim * math.log(original_length / (2.0 * math.pi * turns)) / (2.0 * math.log(base))

    low = max(math.floor(pair(fast_turns)), 0)
    high = min(math.ceil(pair(slow_turns)), rotary_dim - 1)
    part = ((torch.arange(half, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp_(0.0, 1.0)
    return w * (1.0 - part) + w / factor * part


def rotary_table(rotary_dim: int | None = None, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                 original_length: int | None = None, fast_turns: float = 32.0, slow_turns: float = 1.0,
                 inv_freq=None, magnitude: float | None = None, device=None) -> RotaryTable:
    """The frequencies of rotary_inv_freq, or those given as inv_freq (radians for each position), for use with
    ``rotary`` on ``device``. rotary_dim: a multiple of 16. magnitude None: 1, with "yarn" 0.1 ln(factor) + 1."""
    if inv_freq is not None:
        w = torch.as_tensor(inv_freq).detach().to("cpu", torch.float64).contiguous()
        if w.dim() != 1 or (rotary_dim is not None and rotary_dim != 2 * w.shape[0]):
            raise SageError(SAGE_ERR_SHAPE, "inv_freq must have rotary_dim / 2 entries")
        if scaling is not None or factor != 1.0:
            raise SageError(SAGE_ERR_ARG, "inv_freq takes no scaling")
    elif rotary_dim is None:
        raise SageError(SAGE_ERR_ARG, "rotary_dim or inv_freq must be given")
    else:
        w = rotary_inv_freq(rotary_dim, base, scaling, factor, original_length, fast_turns, slow_turns)
    n = w.shape[0]
    if n == 0 or n % 8:
        raise SageError(SAGE_ERR_ARG, "rotary_dim must be a positive multiple of 16")
    if magnitude is None:
        magnitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1.0 else 1.0
    if not math.isfinite(magnitude):
        raise SageError(SAGE_ERR_ARG, "magnitude must be finite")
    turns = torch.empty(n, dtype=torch.int64)
    _check(_lib.load().sage_rotary_turns(ctypes.cast(w.data_ptr(), ctypes.POINTER(ctypes.c_double)), n,
                                         ctypes.cast(turns.data_ptr(), ctypes.POINTER(ctypes.c_uint64))))
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return RotaryTable(turns=turns.to(device), inv_freq=w, magnitude=float(magnitude))


def _heads(t, what: str, layout: str, device):
    """(B, T, heads, D) and the C tensor of a [B, T, heads, D] or [N, heads, D] tensor (or HND)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected torch tensors")
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if t.device != device:
        raise ValueError(f"{what} must live on the table's device")
    if t.dtype != torch.bfloat16:
        raise SageError(SAGE_ERR_DTYPE, "inputs and output must be bfloat16")
    if t.dim() not in (3, 4):
        raise SageError(SAGE_ERR_SHAPE, f"{what} must be 3-d or 4-d")
    sh, st = t.shape, t.stride()
    if st[-1] != 1 and sh[-1] != 1:
        raise SageError(SAGE_ERR_LAYOUT, "the channel stride must be 1")
    B, sb = (sh[0], st[0]) if t.dim() == 4 else (1, 0)
    s, h = (-3, -2) if layout == "NHD" else (-2, -3)
    return (B, sh[s], sh[h], sh[-1]), _lib.Bf16Tensor(t.data_ptr() or 16, sb, st[s], st[h])


def _same_place(out, x):
    if out.data_ptr() == x.data_ptr() and out.numel() and (out.stride() != x.stride() or out.shape != x.shape):
        raise SageError(SAGE_ERR_LAYOUT, "an output in its input's place must have its shape and strides")


def rotary(q, k, positions, table: RotaryTable, interleaved: bool = False, inverse: bool = False,
           tensor_layout: str = "NHD", out=None):
    """Turns queries and keys by their positions (sage_rotary): returns (q, k) turned, or q alone with k None.

    q: BF16 [B, T, H, D] or packed [N, H, D] ("HND": [B, H, T, D], [H, N, D]), k the same with its own heads.
    positions: int32 [B, T] or [T] ([N] for packed tensors), any strides. The pairs are channels
    (i, i + rotary_dim / 2), or with interleaved (2i, 2i + 1); channels from table.rotary_dim on stay as they are.
    inverse turns back (the gradient, and what moves keys between positions: turn back, then to the new one).
    out: (q, k) to write to (q alone with k None); each may be its input itself, else must not overlap it."""
    kept = key = None
    if out is None and k is not None:
        try:
            key = ("rotary", tensor_layout, bool(interleaved), bool(inverse), q.shape, q.stride(), q.dtype,
                   q.get_device(), k.shape, k.stride(), k.dtype, k.get_device(), positions.shape, positions.stride(),
                   positions.dtype, positions.get_device(), table.turns.shape, table.turns.get_device())
            kept = _kept.calls.get(key)
        except (AttributeError, TypeError):
            key = None
    if kept is not None and kept[0] == _get_device():
        index, fn, ref, args, qi, ki, qo, ko, like = kept
        if like:  # (the quicker call: 1.4 us instead of 1.8)
            q_out, k_out = torch.empty_like(q), torch.empty_like(k)
        else:
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
            k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=q.device)
        qi.ptr_dev, ki.ptr_dev = q.data_ptr(), k.data_ptr()
        qo.ptr_dev, ko.ptr_dev = q_out.data_ptr(), k_out.data_ptr()
        args.turns_dev = table.turns.data_ptr()
        args.positions_dev = positions.data_ptr()
        args.magnitude = table.magnitude
        args.cuda_stream = _stream_handle(index)
        rc = fn(ref)
        if rc:
            _check(rc)
        return q_out, k_out
    if tensor_layout not in _LAYOUTS:
        raise SageError(SAGE_ERR_LAYOUT, "tensor_layout must be NHD or HND")
    if not isinstance(table, RotaryTable):
        raise TypeError("expected a RotaryTable")
    device = table.device
    (B, T, H, D), qi = _heads(q, "q", tensor_layout, device)
    Hkv, ki = 0, _lib.Bf16Tensor()
    if k is not None:
        shape, ki = _heads(k, "k", tensor_layout, device)
        if k.dim() != q.dim() or shape[:2] != (B, T) or shape[3] != D:
            raise SageError(SAGE_ERR_SHAPE, "q and k must have the same tokens and head dimension")
        Hkv = shape[2]
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a torch tensor")
    if positions.device != device:
        raise ValueError("positions must live on the table's device")
    if positions.dtype != torch.int32:
        raise SageError(SAGE_ERR_DTYPE, "positions must be int32")
    if tuple(positions.shape) not in ((T,), (B, T)) or (q.dim() == 3 and positions.dim() != 1):
        raise SageError(SAGE_ERR_SHAPE, "positions must be [B, T] or [T] ([N] for packed tensors)")
    ps = positions.stride()
    given = out is not None
    if not given:
        outs = [torch.empty(t.shape, dtype=torch.bfloat16, device=device) for t in (q, k) if t is not None]
    else:
        outs = [out] if k is None and isinstance(out, torch.Tensor) else list(out)
        if len(outs) != (1 if k is None else 2):
            raise SageError(SAGE_ERR_SHAPE, "out must be (q, k), or q alone without k")
    made = []
    for o, x, shape in zip(outs, (q, k), ((B, T, H, D), (B, T, Hkv, D))):
        got, c = _heads(o, "out", tensor_layout, device)
        if o.dim() != x.dim() or got != shape:
            raise SageError(SAGE_ERR_SHAPE, "out must have its input's shape")
        _same_place(o, x)
        made.append(c)
    args = _lib.RotaryArgs(qi, ki, made[0], made[1] if Hkv else _lib.Bf16Tensor(), B, T, H, Hkv, D, table.rotary_dim,
                           table.turns.data_ptr(), positions.data_ptr() or 16, ps[0] if len(ps) == 2 else 0, ps[-1],
                           table.magnitude, bool(interleaved), bool(inverse))
    index = table.turns.get_device()
    with _on(index) as stream:
        args.cuda_stream = stream
        _check(_lib.load().sage_rotary(ctypes.byref(args)))
    if key is not None and q.numel() and k.numel():
        _keep(key, (index, _lib.load().sage_rotary, ctypes.byref(args), args, args.q, args.k, args.q_out, args.k_out,
                    q.is_contiguous() and k.is_contiguous()))
    if k is None:
        return outs[0]
    return outs[0], outs[1]
