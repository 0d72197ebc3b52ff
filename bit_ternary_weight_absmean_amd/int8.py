"""Products of int8 tokens and int8 weights with a scale for each token and channel (bt_int8_*): argument checks and
marshalling only, as in api.py. For the projections that are not ternary; the tokens are quant_act's."""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import api
from .api import _TYPES, _call, _is, _need, _need_bytes, _ptr, _type_of, _workspace_bytes, act_row_bytes, quant_act


def int8_weight_bytes(N: int, K: int) -> int:
    """bt_int8_weight_bytes: bytes of N x K packed int8 weights."""
    return _workspace_bytes("bt_int8_weight_bytes", N, K)


def int8_workspace_bytes(M: int, N: int, K: int) -> int:
    """bt_int8_workspace_bytes: the scratch of an int8_gemm call (0: none)."""
    return _workspace_bytes("bt_int8_workspace_bytes", M, N, K)


@dataclass(frozen=True, eq=False)
class Int8Weight:
    """Packed int8 weights [N, K] and their scales, from pack_int8 or pack_weights_int8."""

    data: torch.Tensor   # uint8 [int8_weight_bytes(N, K)]
    scale: torch.Tensor  # float32 [N]
    N: int
    K: int

    def __post_init__(self):
        _need_bytes(self.data, "packed weights", int8_weight_bytes(self.N, self.K))
        _need(self.scale, "weight scale", torch.float32, (self.N,), self.data.device)


def pack_int8(codes: torch.Tensor, scale: torch.Tensor) -> Int8Weight:
    """bt_int8_pack: weights ``codes`` [N, K] int8 with a ``scale`` [N] fp32 for each row."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise ValueError("codes must be a tensor [N, K]")
    N, K = codes.shape
    _need(codes, "codes", torch.int8)
    _need(scale, "scale", torch.float32, (N,), codes.device)
    data = torch.empty(max(int8_weight_bytes(N, K), 16), dtype=torch.uint8, device=codes.device)
    _call(codes.device, api.lib().bt_int8_pack, codes.data_ptr(), K, N, K, data.data_ptr())
    return Int8Weight(data, scale, N, K)


def pack_weights_int8(W: torch.Tensor) -> Int8Weight:
    """Weights W [N, K] fp32 quantized by row as bt_quant_act does tokens (127 / max|W[n]|), and packed."""
    _need(W, "W", torch.float32)
    if W.dim() != 2:
        raise ValueError(f"W must be [N, K], got shape {tuple(W.shape)}")
    with torch.cuda.device(W.device):
        codes, scale, _ = quant_act(W)
    N, K = W.shape
    data = torch.empty(max(int8_weight_bytes(N, K), 16), dtype=torch.uint8, device=W.device)
    _call(W.device, api.lib().bt_int8_pack, codes.data_ptr(), act_row_bytes(K), N, K, data.data_ptr())
    return Int8Weight(data, scale, N, K)


def int8_workspace(M: int, weight: Int8Weight) -> torch.Tensor | None:
    """A workspace for int8_gemm with M tokens (its contents do not matter), or None where none is needed."""
    n = int8_workspace_bytes(M, weight.N, weight.K)
    return torch.empty(n, dtype=torch.uint8, device=weight.data.device) if n else None


def int8_gemm(weight: Int8Weight, q, bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
              out_dtype: torch.dtype | None = None, out_acc: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    """bt_int8_gemm: Y = acc * (s_x[m] * scale[n]) + bias[n] of tokens ``q`` = (Xq, s_x, ...) as quant_act makes
    them (what follows the first two is not read). ``out`` [M, N] fp32, bf16 or fp16 (``out_dtype``, fp32 where neither
    is given); ``out_acc`` [M, N] int32 also receives the exact products. Returns out."""
    if not isinstance(weight, Int8Weight):
        raise TypeError(f"weight must be an Int8Weight, got {type(weight).__name__}")
    Xq, sx = q[0], q[1]
    dev, (N, K), at = weight.data.device, (weight.N, weight.K), weight.data.get_device()
    if not isinstance(sx, torch.Tensor) or sx.dim() != 1:
        raise ValueError("s_x must be a 1-D tensor of M scales")
    M, f32 = sx.shape[0], torch.float32
    ld = (K + 255) // 256 * 256
    if not (_is(Xq, torch.int8, (M, ld), at) and _is(sx, f32, (M,), at)):
        _need(Xq, "Xq", torch.int8, (M, ld), dev)
        _need(sx, "s_x", f32, (M,), dev)
    if bias is not None and not _is(bias, f32, (N,), at):
        _need(bias, "bias", f32, (N,), dev)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or f32, device=dev)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    kind = _type_of(out, "out", _TYPES)
    if not _is(out, out.dtype, (M, N), at):
        _need(out, "out", out.dtype, (M, N), dev)
    if out_acc is not None:
        _need(out_acc, "out_acc", torch.int32, (M, N), dev)
    need = _workspace_bytes("bt_int8_workspace_bytes", M, N, K)
    if workspace is not None:
        _need_bytes(workspace, "workspace", need, dev)
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _call(dev, api.lib().bt_int8_gemm, weight.data.data_ptr(), weight.scale.data_ptr(), Xq.data_ptr(), sx.data_ptr(), M, N,
          K, _ptr(bias), out.data_ptr(), kind, _ptr(out_acc), _ptr(workspace))
    return out


def int8_linear(X: torch.Tensor, weight: Int8Weight, bias: torch.Tensor | None = None,
                out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """quant_act and int8_gemm: fp32 X [M, K] in, Y [M, N] out."""
    if not isinstance(X, torch.Tensor) or X.dim() != 2 or X.shape[1] != weight.K:
        raise ValueError(f"X must be a tensor [M, {weight.K}]")
    _need(X, "X", torch.float32, None, weight.data.device)
    with torch.cuda.device(X.device):
        q = quant_act(X)
    return int8_gemm(weight, q, bias=bias, out=out, out_dtype=out_dtype)
