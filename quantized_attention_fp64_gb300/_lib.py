"""ctypes binding of libsage.so: loads the library and declares every entry
point of include/sage.h with its C signature. Argument marshalling only."""

from __future__ import annotations

import ctypes
import os
import re

from ._build import LIB_PATH, ROOT

c_i64 = ctypes.c_int64
c_int = ctypes.c_int
c_vp = ctypes.c_void_p
c_size_p = ctypes.POINTER(ctypes.c_size_t)
I64x4 = c_i64 * 4


class Bf16Tensor(ctypes.Structure):
    """sage_bf16_tensor"""
    _fields_ = [("ptr_dev", c_vp), ("stride_b", c_i64), ("stride_s", c_i64), ("stride_h", c_i64)]


class Quantized(ctypes.Structure):
    """sage_quantized"""
    _fields_ = [("q_codes_dev", c_vp), ("k_codes_dev", c_vp), ("vt_codes_dev", c_vp), ("q_scale_dev", c_vp),
                ("k_scale_dev", c_vp), ("v_scale_dev", c_vp), ("k_mean_dev", c_vp), ("q16_dev", c_vp),
                ("k16_dev", c_vp)]


class SageattnArgs(ctypes.Structure):
    """sage_sageattn_args"""
    _fields_ = [("q_dev", c_vp), ("k_dev", c_vp), ("v_dev", c_vp), ("q_shape", I64x4), ("k_shape", I64x4),
                ("v_shape", I64x4), ("q_strides", I64x4), ("k_strides", I64x4), ("v_strides", I64x4),
                ("out_strides", I64x4), ("q_dtype", ctypes.c_int32), ("k_dtype", ctypes.c_int32),
                ("v_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("is_causal", ctypes.c_int32),
                ("smooth_k", ctypes.c_int32), ("sm_scale", ctypes.c_float), ("tensor_layout", ctypes.c_char * 4),
                ("out_dev", c_vp), ("lse_dev", c_vp), ("workspace_dev", c_vp), ("workspace_bytes", ctypes.c_size_t),
                ("cuda_stream", c_vp)]


class Cache(ctypes.Structure):
    """sage_cache"""
    _fields_ = [("k_codes_dev", c_vp), ("v_codes_dev", c_vp), ("k_scale_dev", c_vp), ("v_scale_dev", c_vp),
                ("num_pages", c_i64), ("page_size", c_i64), ("H", c_i64), ("D", c_i64)]


_TABLE_FIELDS = [("cache", c_vp), ("table_dev", c_vp), ("table_stride", c_i64), ("max_pages", c_i64)]


class CacheAppendArgs(ctypes.Structure):
    """sage_cache_append_args"""
    _fields_ = _TABLE_FIELDS + [("starts_dev", c_vp), ("counts_dev", c_vp), ("k", Bf16Tensor), ("v", Bf16Tensor),
                                ("B", c_i64), ("T", c_i64), ("cuda_stream", c_vp)]


class CacheReadArgs(ctypes.Structure):
    """sage_cache_read_args"""
    _fields_ = _TABLE_FIELDS + [("starts_dev", c_vp), ("counts_dev", c_vp), ("k_out", Bf16Tensor),
                                ("v_out", Bf16Tensor), ("B", c_i64), ("T", c_i64), ("zero_rest", ctypes.c_int32),
                                ("cuda_stream", c_vp)]


class CacheAttentionArgs(ctypes.Structure):
    """sage_cache_attention_args"""
    _fields_ = _TABLE_FIELDS + [("lengths_dev", c_vp), ("q_lengths_dev", c_vp), ("q", Bf16Tensor), ("out", Bf16Tensor),
                                ("B", c_i64), ("T", c_i64), ("H", c_i64), ("sm_scale", ctypes.c_float),
                                ("is_causal", ctypes.c_int32), ("zero_rest", ctypes.c_int32), ("lse_dev", c_vp),
                                ("workspace_dev", c_vp), ("workspace_bytes", ctypes.c_size_t), ("cuda_stream", c_vp)]


_SCORES_FIELDS = [("scores_stride_b", c_i64), ("scores_stride_h", c_i64), ("scores_size", c_i64)]


class CacheAddWeightsArgs(ctypes.Structure):
    """sage_cache_add_weights_args"""
    _fields_ = _TABLE_FIELDS + [("lengths_dev", c_vp), ("q_lengths_dev", c_vp), ("q", Bf16Tensor), ("B", c_i64),
                                ("T", c_i64), ("H", c_i64), ("sm_scale", ctypes.c_float), ("is_causal", ctypes.c_int32),
                                ("lse_dev", c_vp), ("scores_dev", c_vp)] + _SCORES_FIELDS + [("cuda_stream", c_vp)]


class CacheEvictArgs(ctypes.Structure):
    """sage_cache_evict_args"""
    _fields_ = _TABLE_FIELDS + [("out_table_dev", c_vp), ("out_table_stride", c_i64), ("out_max_pages", c_i64),
                                ("lengths_dev", c_vp), ("scores_dev", c_vp)] + _SCORES_FIELDS + [
        ("B", c_i64), ("keep", c_i64), ("recent", c_i64), ("lengths_out_dev", c_vp), ("kept_dev", c_vp),
        ("kept_size", c_i64), ("scores_out_dev", c_vp), ("workspace_dev", c_vp), ("workspace_bytes", ctypes.c_size_t),
        ("cuda_stream", c_vp)]


class RotaryArgs(ctypes.Structure):
    """sage_rotary_args"""
    _fields_ = [("q", Bf16Tensor), ("k", Bf16Tensor), ("q_out", Bf16Tensor), ("k_out", Bf16Tensor), ("B", c_i64),
                ("T", c_i64), ("H", c_i64), ("Hkv", c_i64), ("D", c_i64), ("rotary_dim", c_i64), ("turns_dev", c_vp),
                ("positions_dev", c_vp), ("positions_stride_b", c_i64), ("positions_stride_t", c_i64),
                ("magnitude", ctypes.c_float), ("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32),
                ("cuda_stream", c_vp)]


class PromptAttentionArgs(ctypes.Structure):
    """sage_prompt_attention_args"""
    _fields_ = [("q", Bf16Tensor), ("k", Bf16Tensor), ("v", Bf16Tensor), ("out", Bf16Tensor), ("N", c_i64), ("M", c_i64),
                ("H", c_i64), ("Hkv", c_i64), ("D", c_i64), ("B", c_i64), ("offsets_dev", c_vp),
                ("kv_offsets_dev", c_vp), ("sm_scale", ctypes.c_float), ("is_causal", ctypes.c_int32),
                ("zero_rest", ctypes.c_int32), ("lse_dev", c_vp), ("workspace_dev", c_vp),
                ("workspace_bytes", ctypes.c_size_t), ("cuda_stream", c_vp)]


_SIGNATURES = {
    "sage_bundle_size": (c_int, [c_i64, c_i64, c_i64, c_i64, c_size_p, c_vp, ctypes.POINTER(Quantized)]),
    "sage_quantize_scratch_size": (c_int, [c_i64, c_i64, c_i64, c_i64, c_size_p]),
    "sage_workspace_size": (c_int, [c_i64, c_i64, c_i64, c_i64, c_size_p]),
    "sage_quantize": (c_int, [ctypes.POINTER(Bf16Tensor)] * 3 + [c_i64, c_i64, c_i64, c_i64, c_int,
                                                                ctypes.POINTER(Quantized), c_vp, ctypes.c_size_t,
                                                                c_vp]),
    "sage_quantize_noalloc": (c_int, [ctypes.POINTER(Bf16Tensor)] * 3 + [c_i64, c_i64, c_i64, c_i64, c_int,
                                                                        ctypes.POINTER(Quantized), c_vp]),
    "sage_attention": (c_int, [ctypes.POINTER(Quantized), c_i64, c_i64, c_i64, c_i64, ctypes.c_float, c_vp,
                               c_i64, c_i64, c_i64, c_vp]),
    "sage_attention_ex": (c_int, [ctypes.POINTER(Quantized), c_i64, c_i64, c_i64, c_i64, ctypes.c_float, c_int,
                                  c_vp, c_i64, c_i64, c_i64, c_vp, c_vp]),
    "sage_attention_simt": (c_int, [ctypes.POINTER(Quantized), c_i64, c_i64, c_i64, c_i64, ctypes.c_float, c_int,
                                    c_vp, c_i64, c_i64, c_i64, c_vp, c_vp]),
    "sage_lse_smooth_k_term": (c_int, [ctypes.POINTER(Bf16Tensor), c_vp, c_i64, c_i64, c_i64, c_i64, ctypes.c_float,
                                       c_vp, c_vp]),
    "sage_sageattn": (c_int, [c_vp, c_vp, c_vp, I64x4, I64x4, I64x4, I64x4, I64x4, I64x4, c_int, c_int, c_int,
                              ctypes.c_char_p, c_int, ctypes.c_float, c_int, c_int, c_vp, I64x4, c_int, c_vp,
                              ctypes.c_size_t, c_vp]),
    "sage_sageattn_ex": (c_int, [c_vp, c_vp, c_vp, I64x4, I64x4, I64x4, I64x4, I64x4, I64x4, c_int, c_int, c_int,
                                 ctypes.c_char_p, c_int, ctypes.c_float, c_int, c_vp, I64x4, c_int, c_vp, c_vp,
                                 ctypes.c_size_t, c_vp]),
    "sage_sageattn_args_call": (c_int, [ctypes.POINTER(SageattnArgs)]),
    "sage_host_workspace_size": (c_int, [c_i64, c_i64, c_i64, c_i64, c_int, c_size_p]),
    "sage_sageattn_host": (c_int, [c_vp, c_vp, c_vp, I64x4, c_int, ctypes.c_char_p, c_int, ctypes.c_float, c_int, c_vp,
                                   c_int, c_vp, ctypes.c_size_t, c_vp]),
    "sage_cache_size": (c_int, [c_i64, c_i64, c_i64, c_i64, c_size_p, c_vp, ctypes.POINTER(Cache)]),
    "sage_cache_append": (c_int, [ctypes.POINTER(CacheAppendArgs)]),
    "sage_cache_read": (c_int, [ctypes.POINTER(CacheReadArgs)]),
    "sage_cache_copy_pages": (c_int, [c_vp, c_vp, c_vp, c_i64, c_vp]),
    "sage_cache_attention_workspace_size": (c_int, [c_i64, c_i64, c_i64, c_i64, c_i64, c_size_p]),
    "sage_cache_attention": (c_int, [ctypes.POINTER(CacheAttentionArgs)]),
    "sage_cache_add_weights": (c_int, [ctypes.POINTER(CacheAddWeightsArgs)]),
    "sage_cache_evict": (c_int, [ctypes.POINTER(CacheEvictArgs)]),
    "sage_cache_evict_workspace_size": (c_int, [c_i64, c_i64, c_i64, c_i64, c_i64, c_size_p]),
    "sage_rotary": (c_int, [ctypes.POINTER(RotaryArgs)]),
    "sage_rotary_turns": (c_int, [ctypes.POINTER(ctypes.c_double), c_i64, ctypes.POINTER(ctypes.c_uint64)]),
    "sage_prompt_attention": (c_int, [ctypes.POINTER(PromptAttentionArgs)]),
    "sage_prompt_attention_workspace_size": (c_int, [c_i64] * 6 + [c_size_p]),
    "sage_device_error": (c_int, [c_vp, ctypes.POINTER(c_int)]),
    "sage_selftest_wait_timeout": (c_int, [c_vp]),
    "sage_strerror": (ctypes.c_char_p, [c_int]),
}

_lib = None


def header_functions() -> list[str]:
    """Names of the functions include/sage.h declares."""
    with open(os.path.join(ROOT, "include", "sage.h")) as f:
        text = f.read()
    return re.findall(r"SAGE_API\s+(?:const\s+)?\w+\s*\*?\s*(sage_\w+)\s*\(", text)


def ensure_built() -> str:
    from ._build import build

    return build()


def load():
    """Load libsage.so (it must have been built) and declare its signatures."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with quantized_attention_fp64_gb300._build.build()")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib
