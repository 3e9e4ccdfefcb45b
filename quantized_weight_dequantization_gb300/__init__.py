"""Fused nested 4-bit weight dequantization for NVIDIA GB300 (sm_103a).

The computation lives in the CUDA library ``libdq4.so`` (C ABI in
``include/dq4.h``; for the attention around the 4-bit projections
``include/dq4_attn.h``, for layers with 8-bit weights ``include/dq4_int8.h``); this package is its thin Python binding.  The first use
of the library raises ImportError if it has not been built (see ``build``):
there is no CPU fallback.
"""

from ._attention import (  # noqa: F401
    KV8Cache,
    kv8_append,
    kv8_attention,
    qk_norm_rope,
    qk_norm_rope_backward,
)
from ._binding import (  # noqa: F401
    OUT_BF16,
    OUT_F16,
    OUT_F32,
    Dq4Error,
    dq4,
    dq4_nested,
    dq4_nested_host,
    dq4_nested_transposed,
    dq4_nested_unfused,
    dq4_nested_unfused_static,
    get_lib,
    int8_correction_prep,
    linear,
    out_prod,
    sizes,
)
from ._int8 import (  # noqa: F401
    Int8Rows,
    int8_linear,
    int8_linear_backward,
    int8_moe,
    int8_quantize,
)


def __getattr__(name):
    if name == "lib":
        return get_lib()
    raise AttributeError(name)


__all__ = ["dq4_nested", "dq4_nested_host", "dq4_nested_transposed", "dq4",
           "dq4_nested_unfused", "dq4_nested_unfused_static", "Dq4Error", "get_lib", "sizes",
           "int8_correction_prep", "out_prod", "linear", "OUT_F16", "OUT_BF16", "OUT_F32",
           "KV8Cache", "kv8_append", "kv8_attention", "qk_norm_rope", "qk_norm_rope_backward",
           "Int8Rows", "int8_quantize", "int8_linear", "int8_linear_backward", "int8_moe"]
