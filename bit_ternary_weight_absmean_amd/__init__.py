"""MI355X-native BitNet b1.58 W1.58A8 ternary linear layer.

The compute lives in ``libbt.so`` (hand-written HIP kernels for gfx950 behind the C ABI
of ``include/bt.h``). This module only marshals torch tensors (device memory) and the
current HIP stream into those calls; every step of the path runs in the library's
kernels. Names follow the C ABI: ``pack_weights``, ``quant_act``, ``ternary_gemv``,
``ternary_gemm`` (+ ``unpack_weights``, ``linear``, and ``pack_weights_rows`` for
row-group weight scales, which the product calls then take in place of one scale), and the
attention block around the products: ``lora_apply`` (also through ``linear``),
``qk_norm_rope`` and ``attention``. Around a cache in pages held in 4 bits there are ``Cache4`` with
``cache4_write``, ``cache4_read`` and ``attention4``, and ``Pages`` with ``pages_grow``, ``pages_fork``,
``pages_compact`` and ``pages_copy``; for projections that are not ternary ``pack_int8`` and
``int8_gemm`` (``int8_linear``).
"""
from __future__ import annotations

from ._lib import BTError, lib
from .api import (
    BITS_CODES,
    BITS_PLAIN,
    CALL_GEMM,
    CALL_GEMM_WS,
    CALL_GEMV,
    CALL_LINEAR,
    CALL_QUANT,
    GEMV_AUTO,
    GEMV_DOT4,
    GEMV_LUT,
    GEMV_MAX_M,
    GEMV_MFMA,
    GEMV_STAGED,
    LORA_MAX_RANK,
    STATIC_SCRATCH_BYTES,
    LoraAdapters,
    PackedWeight,
    act_row_bytes,
    attention,
    attention_workspace,
    attention_workspace_bytes,
    binarize_act,
    binary_gemv,
    gemm_split_plan,
    gemm_workspace,
    gemm_workspace_bytes,
    kernel_plan,
    linear,
    linear_static,
    linear_workspace_bytes,
    lora_apply,
    lora_workspace,
    lora_workspace_bytes,
    pack_weights,
    pack_weights_binary,
    pack_weights_rows,
    pack_workspace_bytes,
    packed_weight_bytes,
    qk_norm_rope,
    quant_act,
    rope_frequencies,
    ternary_gemm,
    ternary_gemv,
    ternary_gemv_a1,
    unpack_weights,
)
from .cache import (
    Cache4,
    Pages,
    attention4,
    attention4_plan,
    attention4_workspace,
    attention4_workspace_bytes,
    cache4_page_bytes,
    cache4_read,
    cache4_write,
    pages_compact,
    pages_copy,
    pages_fork,
    pages_grow,
)
from .int8 import (
    Int8Weight,
    int8_gemm,
    int8_linear,
    int8_weight_bytes,
    int8_workspace,
    int8_workspace_bytes,
    pack_int8,
    pack_weights_int8,
)

__all__ = [
    "BITS_CODES", "BITS_PLAIN", "binarize_act", "binary_gemv", "pack_weights_binary", "ternary_gemv_a1",
    "BTError", "lib", "GEMV_AUTO", "GEMV_DOT4", "GEMV_LUT", "GEMV_MFMA", "GEMV_STAGED", "GEMV_MAX_M", "PackedWeight", "act_row_bytes",
    "gemm_split_plan", "gemm_workspace", "gemm_workspace_bytes", "linear", "linear_workspace_bytes", "pack_weights", "pack_weights_rows", "pack_workspace_bytes", "packed_weight_bytes", "quant_act", "ternary_gemm",
    "ternary_gemv", "unpack_weights", "kernel_plan", "CALL_LINEAR", "CALL_GEMV", "CALL_GEMM", "CALL_GEMM_WS", "CALL_QUANT", "linear_static", "STATIC_SCRATCH_BYTES",
    "LORA_MAX_RANK", "LoraAdapters", "lora_apply", "lora_workspace", "lora_workspace_bytes", "qk_norm_rope",
    "rope_frequencies", "attention", "attention_workspace", "attention_workspace_bytes",
    "Cache4", "cache4_page_bytes", "cache4_read", "cache4_write", "attention4", "attention4_plan", "attention4_workspace",
    "attention4_workspace_bytes", "Pages", "pages_compact", "pages_copy", "pages_fork", "pages_grow",
    "Int8Weight", "int8_gemm", "int8_linear", "int8_weight_bytes", "int8_workspace", "int8_workspace_bytes",
    "pack_int8", "pack_weights_int8",
]
