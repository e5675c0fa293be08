"""GB300 (sm_103a) SageAttention-style quantized attention.

The computation lives in the CUDA library ``libsage.so`` (C ABI declared in
``include/sage.h``); this package loads it with ctypes and marshals torch
tensors into it. Build the library with ``quantized_attention_fp64_gb300._build.build()``.
"""

from .api import (  # noqa: F401
    QuantizedQKV,
    SageError,
    alloc_bundle,
    attention,
    attention_simt,
    device_error,
    host_workspace_size,
    lse_smooth_k_term,
    quantize,
    quantize_scratch_size,
    release_workspace_cache,
    sageattn,
    sageattn_ex,
    sageattn_host,
    workspace_size,
)
from .cache import (  # noqa: F401
    QuantizedCache,
    alloc_cache,
    cache_add_weights,
    cache_append,
    cache_attention,
    cache_attention_workspace_size,
    cache_copy_pages,
    cache_evict,
    cache_evict_workspace_size,
    cache_read,
)
from .prompt import prompt_attention, prompt_attention_workspace_size  # noqa: F401
from .rotary import RotaryTable, rotary, rotary_inv_freq, rotary_table  # noqa: F401
