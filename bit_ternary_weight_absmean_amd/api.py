"""Torch-facing wrappers over the C ABI (argument marshalling only).

Every function takes and returns torch tensors on a HIP device, passes raw device
pointers and ``torch.cuda.current_stream().cuda_stream`` to libbt.so, and checks the
returned status. Nothing here computes any part of the method.
"""
from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass
from functools import lru_cache

import torch

from ._lib import check, lib

GEMV_AUTO, GEMV_DOT4, GEMV_MFMA, GEMV_LUT, GEMV_STAGED = 0, 1, 2, 3, 4
GEMV_MAX_M = 16


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _on_device(t: torch.Tensor) -> bool:
    return t.is_cuda


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None, device=None):
    """Reject a tensor the library would read or write out of bounds: wrong dtype, shape
    (None: any), layout or device. Checked before any call, so a bad buffer is a Python
    error and never a device fault."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not _on_device(t):
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the weights on {device}")


def _need_bytes(t: torch.Tensor, name: str, nbytes: int, device=None):
    """A contiguous device buffer of at least ``nbytes`` bytes (any dtype)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name} holds {have} bytes, the call needs {nbytes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not _on_device(t):
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the weights on {device}")


def _outputs(M, N, dev, want_y, want_acc, out_y, out_acc):
    """The (Y, acc) buffers of a product: the caller's (checked) or new ones."""
    if out_y is not None:
        _need(out_y, "out_y", torch.float32, (M, N), dev)
        Y = out_y
    else:
        Y = torch.empty((M, N), dtype=torch.float32, device=dev) if want_y else None
    if out_acc is not None:
        _need(out_acc, "out_acc", torch.int32, (M, N), dev)
        acc = out_acc
    else:
        acc = torch.empty((M, N), dtype=torch.int32, device=dev) if want_acc else None
    if Y is None and acc is None:
        raise ValueError("a product needs Y or acc (want_y / want_acc / out_y / out_acc)")
    return Y, acc


def _check_q(q, K: int, dev):
    """(Xq, s_x, x_sum) as bt_quant_act writes them for K input features."""
    Xq, sx, xsum = q
    if not isinstance(sx, torch.Tensor) or sx.dim() != 1:
        raise ValueError("s_x must be a 1-D tensor of M scales")
    M = sx.shape[0]
    _need(Xq, "Xq", torch.int8, (M, act_row_bytes(K)), dev)
    _need(sx, "s_x", torch.float32, (M,), dev)
    _need(xsum, "x_sum", torch.int32, (M,), dev)
    return M


def packed_weight_bytes(N: int, K: int) -> int:
    return int(lib().bt_packed_weight_bytes(N, K))


def act_row_bytes(K: int) -> int:
    return int(lib().bt_act_row_bytes(K))


def pack_workspace_bytes(N: int, K: int) -> int:
    return int(lib().bt_pack_workspace_bytes(N, K))


@dataclass
class PackedWeight:
    """A 2-bit packed ternary weight matrix and its absmean scale(s) (both on device)."""

    data: torch.Tensor   # uint8 [packed_weight_bytes(N, K)]
    scale: torch.Tensor  # float32 [1] gamma, or [N] row scales when row_scales
    N: int
    K: int
    row_scales: bool = False

    def check(self, packed_bytes: int | None = None):
        """The buffers hold what the library reads for an N x K matrix."""
        _need_bytes(self.data, "packed weights", packed_weight_bytes(self.N, self.K) if packed_bytes is None
                    else packed_bytes)
        _need(self.scale, "weight scale", torch.float32, (max(self.N, 1),) if self.row_scales else (1,),
              self.data.device)


def pack_weights(W: torch.Tensor, workspace: torch.Tensor | None = None) -> PackedWeight:
    """bt_pack_weights: absmean ternarization + 2-bit packing of W [N,K] fp32."""
    _need(W, "W", torch.float32)
    N, K = W.shape
    dev = W.device
    data = torch.empty(max(packed_weight_bytes(N, K), 16), dtype=torch.uint8, device=dev)
    scale = torch.empty(1, dtype=torch.float32, device=dev)
    ws_bytes = pack_workspace_bytes(N, K)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 8), dtype=torch.uint8, device=dev)
    else:
        _need_bytes(workspace, "workspace", ws_bytes, dev)
    check(lib().bt_pack_weights(_ptr(W), N, K, _ptr(data), _ptr(scale), _ptr(workspace), _stream(dev)))
    return PackedWeight(data, scale, N, K)


def pack_weights_rows(W: torch.Tensor, group_rows=None, workspace: torch.Tensor | None = None) -> PackedWeight:
    """bt_pack_weights_rows: packing with row-group scales (``group_rows``: the rows of each
    group in order, summing to N; None: one group per row). The result carries N row scales."""
    _need(W, "W", torch.float32)
    N, K = W.shape
    dev = W.device
    data = torch.empty(max(packed_weight_bytes(N, K), 16), dtype=torch.uint8, device=dev)
    scale = torch.empty(max(N, 1), dtype=torch.float32, device=dev)
    ws_bytes = pack_workspace_bytes(N, K)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 8), dtype=torch.uint8, device=dev)
    else:
        _need_bytes(workspace, "workspace", ws_bytes, dev)
    if group_rows is None:
        groups, ngroups = 0, 0
    else:
        arr = (ctypes.c_int64 * len(group_rows))(*[int(r) for r in group_rows])
        groups, ngroups = ctypes.cast(arr, ctypes.c_void_p).value, len(group_rows)
    check(lib().bt_pack_weights_rows(_ptr(W), N, K, groups, ngroups, _ptr(data), _ptr(scale), _ptr(workspace),
                                     _stream(dev)))
    return PackedWeight(data, scale, N, K, row_scales=True)


def unpack_weights(pw: PackedWeight) -> torch.Tensor:
    """bt_unpack_weights: the ternary codes t in {-1,0,1} as int8 [N,K]."""
    pw.check()
    T = torch.empty((pw.N, pw.K), dtype=torch.int8, device=pw.data.device)
    check(lib().bt_unpack_weights(_ptr(pw.data), pw.N, pw.K, _ptr(T), _stream(pw.data.device)))
    return T


def quant_act(X: torch.Tensor, out=None):
    """bt_quant_act: per-token absmax int8. Returns (Xq [M, act_row_bytes(K)] int8, s_x [M], x_sum [M])."""
    _need(X, "X", torch.float32)
    M, K = X.shape
    dev = X.device
    if out is None:
        Xq = torch.empty((M, act_row_bytes(K)), dtype=torch.int8, device=dev)
        sx = torch.empty(M, dtype=torch.float32, device=dev)
        xsum = torch.empty(M, dtype=torch.int32, device=dev)
    else:
        Xq, sx, xsum = out
        _need(Xq, "Xq", torch.int8, (M, act_row_bytes(K)), dev)
        _need(sx, "s_x", torch.float32, (M,), dev)
        _need(xsum, "x_sum", torch.int32, (M,), dev)
    check(lib().bt_quant_act(_ptr(X), M, K, _ptr(Xq), _ptr(sx), _ptr(xsum), _stream(dev)))
    return Xq, sx, xsum


def _product(fn_name, pw: PackedWeight, q, want_y, want_acc, out_y, out_acc, algo=None, extra=()):
    pw.check()
    dev = pw.data.device
    M = _check_q(q, pw.K, dev)
    Xq, sx, xsum = q
    Y, acc = _outputs(M, pw.N, dev, want_y, want_acc, out_y, out_acc)
    args = [_ptr(pw.data), _ptr(pw.scale), _ptr(Xq), _ptr(sx), _ptr(xsum), M, pw.N, pw.K, _ptr(Y), _ptr(acc)]
    if algo is not None:
        args.append(algo)
    args.extend(extra)
    check(getattr(lib(), fn_name)(*args, _stream(dev)))
    return Y, acc


def ternary_gemv(pw: PackedWeight, q, want_y=True, want_acc=False, out_y=None, out_acc=None, algo=GEMV_AUTO):
    """bt_ternary_gemv_algo (bt_ternary_gemv_rs for row scales): decode product for M <= 16
    tokens. Returns (Y, acc)."""
    fn = "bt_ternary_gemv_rs" if pw.row_scales else "bt_ternary_gemv_algo"
    return _product(fn, pw, q, want_y, want_acc, out_y, out_acc, algo)


def gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    """bt_gemm_workspace_bytes: workspace the split-K route of bt_ternary_gemm_ws uses (0: none)."""
    return int(lib().bt_gemm_workspace_bytes(M, N, K))


def gemm_split_plan(M: int, N: int, K: int) -> tuple[int, int]:
    """bt_gemm_split_plan: (full_tiles, splits) -- the first full_tiles 64 x 256 output tiles
    are computed whole, each later one over `splits` workgroups (splits == 1: no split)."""
    full = ctypes.c_int64(0)
    splits = ctypes.c_int32(0)
    check(lib().bt_gemm_split_plan(M, N, K, ctypes.byref(full), ctypes.byref(splits)))
    return int(full.value), int(splits.value)


def gemm_workspace(M: int, N: int, K: int, device) -> torch.Tensor | None:
    """A zero-filled workspace for bt_ternary_gemm_ws(M, N, K), or None when the shape does not split."""
    n = gemm_workspace_bytes(M, N, K)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def ternary_gemm(pw: PackedWeight, q, want_y=True, want_acc=False, out_y=None, out_acc=None,
                 workspace: torch.Tensor | None = None):
    """bt_ternary_gemm: prefill product on int8 MFMA for any M. Returns (Y, acc).

    With a workspace (see gemm_workspace) the call is bt_ternary_gemm_ws, which splits K
    over several workgroups per tile where that pays; results are identical.
    """
    if workspace is None and not pw.row_scales:
        return _product("bt_ternary_gemm", pw, q, want_y, want_acc, out_y, out_acc)
    if workspace is not None:
        # any size is valid: one below gemm_workspace_bytes selects the unsplit route
        _need_bytes(workspace, "workspace", 0, pw.data.device)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return _product("bt_ternary_gemm_rs" if pw.row_scales else "bt_ternary_gemm_ws", pw, q, want_y, want_acc,
                    out_y, out_acc, extra=(_ptr(workspace), nbytes))


def linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().bt_linear_workspace_bytes(M, N, K))


def linear(X: torch.Tensor, pw: PackedWeight, want_y=True, want_acc=False, out_y=None, out_acc=None,
           workspace: torch.Tensor | None = None, adapters: LoraAdapters | None = None,
           adapter_index: torch.Tensor | None = None):
    """bt_ternary_linear: fp32 X [M,K] in, (Y [M,N] fp32, acc [M,N] int32) out.

    One fused launch for decode-sized M; quantize + GEMV/GEMM otherwise. With ``adapters`` and
    ``adapter_index`` [M] int32, Y also receives each token's low-rank product (lora_apply, of
    the unquantized X); acc stays the shared product's.
    """
    pw.check()
    dev = pw.data.device
    if (adapters is None) != (adapter_index is None):
        raise ValueError("adapters and adapter_index come together")
    if adapters is not None:
        if (adapters.N, adapters.K) != (pw.N, pw.K):
            raise ValueError(f"the adapters are for {adapters.N} x {adapters.K}, the weights are {pw.N} x {pw.K}")
        if out_y is None and not want_y:
            raise ValueError("adapters are added to Y: want_y or out_y is needed")
    if X.dim() != 2:
        raise ValueError(f"X must be [M, K], got shape {tuple(X.shape)}")
    _need(X, "X", torch.float32, device=dev)
    M, K = X.shape
    if K != pw.K:
        raise ValueError(f"X has K = {K}, weights have K = {pw.K}")
    Y, acc = _outputs(M, pw.N, dev, want_y, want_acc, out_y, out_acc)
    ws_bytes = linear_workspace_bytes(M, pw.N, K)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    elif ws_bytes:
        _need_bytes(workspace, "workspace", ws_bytes, dev)
    if adapters is not None:
        _need(adapters.B, "adapters", adapters.B.dtype, None, dev)
        _need(adapter_index, "adapter_index", torch.int32, (M,), dev)
    fn = lib().bt_ternary_linear_rs if pw.row_scales else lib().bt_ternary_linear
    check(fn(_ptr(pw.data), _ptr(pw.scale), _ptr(X), M, pw.N, K, _ptr(Y), _ptr(acc),
             _ptr(workspace) if ws_bytes else 0, _stream(dev)))
    if adapters is not None:
        lora_apply(X, adapters, adapter_index, base=Y, out=Y)
    return Y, acc


STATIC_SCRATCH_BYTES = 64 << 20  # BT_STATIC_SCRATCH_BYTES


def linear_static(X: torch.Tensor, pw: PackedWeight, out_y=None, out_acc=None, want_y=True, want_acc=False):
    """bt_ternary_linear_static: bt_ternary_linear without a workspace (the library's static
    scratch serves the routes that need one). One scale per matrix only. Pass out_y / out_acc
    to keep the call free of allocation."""
    if pw.row_scales:
        raise ValueError("bt_ternary_linear_static takes weights with one scale per matrix")
    pw.check()
    dev = pw.data.device
    if X.dim() != 2:
        raise ValueError(f"X must be [M, K], got shape {tuple(X.shape)}")
    _need(X, "X", torch.float32, device=dev)
    M, K = X.shape
    if K != pw.K:
        raise ValueError(f"X has K = {K}, weights have K = {pw.K}")
    Y, acc = _outputs(M, pw.N, dev, want_y, want_acc, out_y, out_acc)
    check(lib().bt_ternary_linear_static(_ptr(pw.data), _ptr(pw.scale), _ptr(X), M, pw.N, K, _ptr(Y), _ptr(acc),
                                         _stream(dev)))
    return Y, acc


CALL_LINEAR, CALL_GEMV, CALL_GEMM, CALL_GEMM_WS, CALL_QUANT = 0, 1, 2, 3, 4


def kernel_plan(call: int, M: int, N: int, K: int, algo: int = GEMV_AUTO, row_scales: bool = False) -> str:
    """bt_kernel_plan: the kernel instances the call would launch (host-only query)."""
    buf = ctypes.create_string_buffer(512)
    check(lib().bt_kernel_plan(call, M, N, K, algo, int(row_scales), buf, len(buf)))
    return buf.value.decode()


# ------------------------------------------------------------- 1-bit activations
BITS_PLAIN, BITS_CODES = 1, 2


def pack_weights_binary(W: torch.Tensor, workspace: torch.Tensor | None = None) -> PackedWeight:
    """bt_pack_weights_binary: sign bits of W [N,K] fp32 and its absmax (W1A1 weights)."""
    _need(W, "W", torch.float32)
    N, K = W.shape
    dev = W.device
    data = torch.empty(max(int(lib().bt_binary_weight_bytes(N, K)), 16), dtype=torch.uint8, device=dev)
    scale = torch.empty(1, dtype=torch.float32, device=dev)
    ws_bytes = pack_workspace_bytes(N, K)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 8), dtype=torch.uint8, device=dev)
    else:
        _need_bytes(workspace, "workspace", ws_bytes, dev)
    check(lib().bt_pack_weights_binary(_ptr(W), N, K, _ptr(data), _ptr(scale), _ptr(workspace), _stream(dev)))
    return PackedWeight(data, scale, N, K)


def binarize_act(X: torch.Tensor, layout: int, out=None):
    """bt_binarize_act: (bits [M, row_bytes / 4] int32, x_scale [M] = absmax per token)."""
    _need(X, "X", torch.float32)
    M, K = X.shape
    dev = X.device
    words = int(lib().bt_act_bits_row_bytes(K, layout)) // 4
    if out is None:
        Xb = torch.empty((M, words), dtype=torch.int32, device=dev)
        sx = torch.empty(M, dtype=torch.float32, device=dev)
    else:
        Xb, sx = out
        _need(Xb, "Xb", torch.int32, (M, words), dev)
        _need(sx, "x_scale", torch.float32, (M,), dev)
    check(lib().bt_binarize_act(_ptr(X), M, K, layout, _ptr(Xb), _ptr(sx), _stream(dev)))
    return Xb, sx


def _bits_product(fn_name, pw: PackedWeight, b, layout, want_y, want_acc, out_y, out_acc):
    dev = pw.data.device
    pw.check(int(lib().bt_binary_weight_bytes(pw.N, pw.K)) if layout == BITS_PLAIN else None)
    Xb, sx = b
    if not isinstance(sx, torch.Tensor) or sx.dim() != 1:
        raise ValueError("x_scale must be a 1-D tensor of M scales")
    M = sx.shape[0]
    _need(Xb, "Xb", torch.int32, (M, int(lib().bt_act_bits_row_bytes(pw.K, layout)) // 4), dev)
    _need(sx, "x_scale", torch.float32, (M,), dev)
    Y, acc = _outputs(M, pw.N, dev, want_y, want_acc, out_y, out_acc)
    check(getattr(lib(), fn_name)(_ptr(pw.data), _ptr(pw.scale), _ptr(Xb), _ptr(sx), M, pw.N, pw.K, _ptr(Y),
                                  _ptr(acc), _stream(dev)))
    return Y, acc


def binary_gemv(pw: PackedWeight, b, want_y=True, want_acc=False, out_y=None, out_acc=None):
    """bt_binary_gemv (W1A1): ``pw`` from pack_weights_binary, ``b`` from binarize_act(X, BITS_PLAIN)."""
    return _bits_product("bt_binary_gemv", pw, b, BITS_PLAIN, want_y, want_acc, out_y, out_acc)


def ternary_gemv_a1(pw: PackedWeight, b, want_y=True, want_acc=False, out_y=None, out_acc=None):
    """bt_ternary_gemv_a1 (W1.58A1): ``pw`` from pack_weights, ``b`` from binarize_act(X, BITS_CODES)."""
    return _bits_product("bt_ternary_gemv_a1", pw, b, BITS_CODES, want_y, want_acc, out_y, out_acc)


# ------------------------------------------------- the attention block around the products
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}  # BT_F32, BT_BF16, BT_F16


def _type_of(t, name: str, allowed) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in allowed:
        raise TypeError(f"{name} must be one of {[str(a) for a in allowed]}, got {t.dtype}")
    return _TYPES[t.dtype]


def _need_strided(t, name: str, dtype, shape, device, output: bool = False):
    """A device tensor of the given shape whose last dimension is contiguous; as an output, one whose
    elements do not share memory."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not _on_device(t):
        raise ValueError(f"{name} must be a device tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.is_contiguous():
        return
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if output and t.numel():
        span = 1
        for step, n in sorted((t.stride(d), t.shape[d]) for d in range(t.dim()) if t.shape[d] > 1):
            if step < span:
                raise ValueError(f"{name} is an output and must not overlap itself")
            span = step * (n - 1) + span


def _call(dev, fn, *args):
    """A library call on ``dev``'s current stream; ``dev`` need not be the current device."""
    if dev.index == _current_device():
        status = fn(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev.index))
    if status:
        check(status)


# torch.cuda.current_stream(i).cuda_stream and torch.cuda.current_device() without the objects around
# them, where this torch has such (one built without a GPU has not, and serves the host-only queries): a
# decode step's calls are shorter than those take.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _is(t, dtype, shape, device) -> bool:
    """Whether t is a contiguous tensor of that type and shape on device number ``device``: the usual
    case, in as few steps as possible (a decode step's calls take a few microseconds). Where not, the
    checks proper say what is wrong, or find that a strided tensor will do."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous())


@lru_cache(maxsize=4096)
def _workspace_bytes(name: str, *sizes: int) -> int:
    """A workspace size query of the library (a function of the sizes alone)."""
    return int(getattr(lib(), name)(*sizes))


LORA_MAX_RANK = 256  # BT_LORA_MAX_RANK


@dataclass(frozen=True, eq=False)
class LoraAdapters:
    """Low-rank adapters of one projection: ``A`` [L, groups * R, K] and ``B`` [L, N, R] (bf16, fp16 or
    fp32), ``scale`` [L] fp32, optionally the ``ranks`` [L] int32 in use and, for a fused projection, the
    ``group_rows`` (rows of each group, summing to N; every group has its own R rows of A)."""

    A: torch.Tensor
    B: torch.Tensor
    scale: torch.Tensor
    ranks: torch.Tensor | None = None
    group_rows: tuple | None = None

    def __post_init__(self):
        for t, name in ((self.A, "A"), (self.B, "B")):
            _type_of(t, name, _TYPES)
            if t.dim() != 3:
                raise ValueError(f"{name} must have three dimensions, got shape {tuple(t.shape)}")
        L, N, R = self.B.shape
        groups = 1
        if self.group_rows is not None:
            object.__setattr__(self, "group_rows", tuple(int(r) for r in self.group_rows))
            groups = len(self.group_rows)
            if not 1 <= groups <= 8 or min(self.group_rows) < 1 or sum(self.group_rows) != N:
                raise ValueError(f"group_rows {self.group_rows} must be 1 to 8 positive counts that sum to N = {N}")
        if not 1 <= R <= LORA_MAX_RANK:
            raise ValueError(f"the rank must be 1 to {LORA_MAX_RANK}, got {R}")
        dev = self.B.device
        _need(self.B, "B", self.B.dtype)
        _need(self.A, "A", self.B.dtype, (L, groups * R, self.A.shape[2]), dev)
        _need(self.scale, "scale", torch.float32, (L,), dev)
        if self.ranks is not None:
            _need(self.ranks, "ranks", torch.int32, (L,), dev)
        arr = None if self.group_rows is None else struct.pack(f"{groups}q", *self.group_rows)
        for name, value in (("_groups", (arr, groups)), ("_dev", dev), ("_shape", (L, N, R)),
                            ("_K", self.A.shape[2]), ("_type", _TYPES[self.B.dtype])):
            object.__setattr__(self, name, value)

    def __setstate__(self, kept):  # perhaps loaded onto another device than it was saved from
        self.__dict__.update(kept, _dev=kept["B"].device)

    @property
    def K(self) -> int:
        return self.A.shape[2]

    @property
    def N(self) -> int:
        return self.B.shape[1]

    @property
    def rank(self) -> int:
        return self.B.shape[2]


def lora_workspace_bytes(M: int, adapters: LoraAdapters) -> int:
    """bt_lora_workspace_bytes for M tokens."""
    return _workspace_bytes("bt_lora_workspace_bytes", M, adapters.K, adapters.rank, adapters._groups[1])


def lora_workspace(M: int, adapters: LoraAdapters) -> torch.Tensor:
    """A workspace for lora_apply with M tokens (its contents do not matter)."""
    return torch.empty(max(lora_workspace_bytes(M, adapters), 256), dtype=torch.uint8, device=adapters.B.device)


def lora_apply(X: torch.Tensor, adapters: LoraAdapters, index: torch.Tensor, base: torch.Tensor | None = None,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """bt_lora_apply: ``base`` (None: zeros) plus each token's low-rank product. ``index`` [M] int32 names
    the token's adapter (outside [0, L): none). ``out`` may be ``base``. Returns out [M, N] fp32."""
    B, dev = adapters.B, adapters._dev
    (L, N, R), K = adapters._shape, adapters._K
    arr, groups = adapters._groups
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise ValueError("X must be a tensor [M, K]")
    M = X.shape[0]
    f32 = torch.float32
    at = X.get_device()
    if not (X.device == dev and _is(X, f32, (M, K), at) and _is(index, torch.int32, (M,), at)
            and (base is None or _is(base, f32, (M, N), at)) and (out is None or _is(out, f32, (M, N), at))):
        _need(X, "X", f32, (M, K), dev)
        _need(index, "index", torch.int32, (M,), dev)
        if base is not None:
            _need(base, "base", f32, (M, N), dev)
        if out is not None:
            _need(out, "out", f32, (M, N), dev)
    if out is None:
        out = torch.empty((M, N), dtype=f32, device=dev)
    need = _workspace_bytes("bt_lora_workspace_bytes", M, K, R, groups)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    else:
        _need_bytes(workspace, "workspace", need, dev)
    _call(dev, lib().bt_lora_apply, adapters.A.data_ptr(), B.data_ptr(), adapters._type, adapters.scale.data_ptr(),
          _ptr(adapters.ranks), L, R, arr, groups, index.data_ptr(), X.data_ptr(), _ptr(base), M, N, K,
          out.data_ptr(), workspace.data_ptr())
    return out


def rope_frequencies(rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """The usual fp64 angles per position of qk_norm_rope: base ** (-2 p / rot_dim), p < rot_dim / 2."""
    p = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    return float(base) ** (-2.0 * p / rot_dim)


def qk_norm_rope(qkv: torch.Tensor, positions: torch.Tensor | None, inv_freq: torch.Tensor | None, heads: int,
                 kv_heads: int, q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                 eps: float = 1e-6, interleaved: bool = False, rows: torch.Tensor | None = None, out=None,
                 dtype: torch.dtype = torch.bfloat16):
    """bt_qk_norm_rope: per-head norms and position rotation of the Q and K heads of fused QKV rows
    ``qkv`` [M, (heads + 2 kv_heads) * D], and the conversion of Q, K and V to the attention's type.

    ``inv_freq`` [rot_dim / 2] fp64 (None: no rotation) gives the rotated part of the heads. ``out`` =
    (q [M, heads, D], k, v) of one type, rows and heads at strides of whole fours; k and v are [M, kv_heads, D], or
    caches [any, kv_heads, D] with ``rows`` [M] int32 naming each token's row (outside: not written).
    Without ``out``, new tensors of ``dtype``. Returns (q, k, v)."""
    in_type = _type_of(qkv, "qkv", _TYPES)
    if qkv.dim() != 2:
        raise ValueError(f"qkv must be [M, values], got shape {tuple(qkv.shape)}")
    if heads < 1 or kv_heads < 1 or heads % kv_heads:
        raise ValueError(f"heads = {heads} must be a positive multiple of kv_heads = {kv_heads}")
    (M, values), total, dev, at = qkv.shape, heads + 2 * kv_heads, qkv.device, qkv.get_device()
    f32, i32 = torch.float32, torch.int32
    if values == 0 or values % total:
        raise ValueError(f"qkv rows of {values} values are not {total} heads")
    D = values // total
    if not (_on_device(qkv) and qkv.is_contiguous()):
        _need_strided(qkv, "qkv", qkv.dtype, qkv.shape, dev)
    if q_weight is not None and not _is(q_weight, f32, (D,), at):
        _need(q_weight, "q_weight", f32, (D,), dev)
    if k_weight is not None and not _is(k_weight, f32, (D,), at):
        _need(k_weight, "k_weight", f32, (D,), dev)
    rot = 0
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be a 1-D tensor of rot_dim / 2 angles")
        half = inv_freq.shape[0]
        rot = 2 * half
        if not (_is(inv_freq, torch.float64, (half,), at) and _is(positions, i32, (M,), at)):
            _need(inv_freq, "inv_freq", torch.float64, None, dev)
            _need(positions, "positions", i32, (M,), dev)
    if rows is not None:
        if not _is(rows, i32, (M,), at):
            _need(rows, "rows", i32, (M,), dev)
        if out is None:
            raise ValueError("rows names rows of the k and v given in out")
    if out is None:
        q = torch.empty((M, heads, D), dtype=dtype, device=dev)
        k = torch.empty((M, kv_heads, D), dtype=dtype, device=dev)
        v = torch.empty((M, kv_heads, D), dtype=dtype, device=dev)
    else:
        q, k, v = out
    out_type = _type_of(q, "q", _TYPES)
    room = k.shape[0] if rows is not None and isinstance(k, torch.Tensor) and k.dim() == 3 else M
    dt, kv = q.dtype, (room, kv_heads, D)
    if not (_is(q, dt, (M, heads, D), at) and _is(k, dt, kv, at) and _is(v, dt, kv, at)):
        _need_strided(q, "q", dt, (M, heads, D), dev, output=True)
        _need_strided(k, "k", dt, kv, dev, output=True)
        _need_strided(v, "v", dt, kv, dev, output=True)
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    shape = _HEADS_SHAPE.pack(M, heads, kv_heads, D, rot, qkv.stride(0), room, qs[0], qs[1], ks[0], ks[1], vs[0],
                              vs[1], in_type, out_type, interleaved, eps)
    _call(dev, lib().bt_qk_norm_rope, shape, qkv.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(positions),
          _ptr(inv_freq), _ptr(rows), q.data_ptr(), k.data_ptr(), v.data_ptr())
    return q, k, v


_HEADS_SHAPE = struct.Struct("13q3if")  # bt_heads_shape
_ATTENTION_SHAPE = struct.Struct("7q3if12q")  # bt_attention_shape
_HALF = {torch.bfloat16: 1, torch.float16: 2}


def attention_workspace_bytes(tokens: int, keys: int, seqs: int, heads: int, kv_heads: int, head_dim: int,
                              prefix: int = 0) -> int:
    """bt_attention_workspace_bytes: the scratch of an attention call (0: none)."""
    return _workspace_bytes("bt_attention_workspace_bytes", tokens, keys, seqs, heads, kv_heads, head_dim, prefix)


def attention_workspace(q: torch.Tensor, k: torch.Tensor, seqs: int,
                        prefix_k: torch.Tensor | None = None) -> torch.Tensor | None:
    """A workspace for attention of these arrays in ``seqs`` sequences (its contents do not matter), or
    None where none is needed."""
    n = attention_workspace_bytes(q.shape[0], k.shape[0], seqs, q.shape[1], k.shape[1], q.shape[2],
                                  0 if prefix_k is None else prefix_k.shape[0])
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor, k_start: torch.Tensor,
              k_len: torch.Tensor, causal: bool = True, scale: float | None = None,
              prefix_k: torch.Tensor | None = None, prefix_v: torch.Tensor | None = None,
              out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
              lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """bt_attention: softmax attention of packed sequences with grouped heads.

    ``q`` [T, heads, D], ``k`` and ``v`` [rows, kv_heads, D] (bf16 or fp16, row and head strides of
    whole eights). Sequence b has queries q_start[b] .. q_start[b + 1] and keys k_start[b] .. + k_len[b]
    (int32, on the device); ``causal``: its last query sees all of them. With ``prefix_k`` / ``prefix_v`` [P, kv_heads,
    D] every query also sees the whole prefix. ``scale`` defaults to D ** -0.5. ``out`` [T, heads, D] in
    q's type or fp32 (``out_dtype``); ``lse`` [T, heads] fp32 receives the log of the softmax's sum.
    Rows of no sequence are not written. Returns (out, lse)."""
    kind = _type_of(q, "q", _HALF)
    if q.dim() != 3:
        raise ValueError(f"q must be [T, heads, D], got shape {tuple(q.shape)}")
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a tensor [rows, kv_heads, D]")
    if not isinstance(k_len, torch.Tensor) or k_len.dim() != 1:
        raise ValueError("k_len must be a 1-D tensor, one entry per sequence")
    (T, heads, D), (S, kv_heads), B, dev, dt = q.shape, k.shape[:2], k_len.shape[0], q.device, q.dtype
    if kv_heads < 1 or heads < 1 or heads % kv_heads:
        raise ValueError(f"{heads} heads are not a positive multiple of {kv_heads} key heads")
    kv, i32 = (S, kv_heads, D), torch.int32
    at = q.get_device()
    if not (_on_device(q) and q.is_contiguous() and _is(k, dt, kv, at) and _is(v, dt, kv, at)
            and _is(q_start, i32, (B + 1,), at) and _is(k_start, i32, (B,), at) and _is(k_len, i32, (B,), at)):
        _need_strided(q, "q", dt, q.shape, dev)
        _need_strided(k, "k", dt, kv, dev)
        _need_strided(v, "v", dt, kv, dev)
        _need(q_start, "q_start", i32, (B + 1,), dev)
        _need(k_start, "k_start", i32, (B,), dev)
        _need(k_len, "k_len", i32, (B,), dev)
    P, pk, pv = 0, (0, 0), (0, 0)
    if (prefix_k is None) != (prefix_v is None):
        raise ValueError("prefix_k and prefix_v come together")
    if prefix_k is not None:
        if not isinstance(prefix_k, torch.Tensor) or prefix_k.dim() != 3:
            raise ValueError("prefix_k must be a tensor [P, kv_heads, D]")
        P = prefix_k.shape[0]
        if not (_is(prefix_k, dt, (P, kv_heads, D), at) and _is(prefix_v, dt, (P, kv_heads, D), at)):
            _need_strided(prefix_k, "prefix_k", dt, (P, kv_heads, D), dev)
            _need_strided(prefix_v, "prefix_v", dt, (P, kv_heads, D), dev)
        pk, pv = prefix_k.stride(), prefix_v.stride()
    if out is None:
        out = torch.empty((T, heads, D), dtype=out_dtype or dt, device=dev)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    ot = out.dtype
    if ot is not dt and ot is not torch.float32:
        raise TypeError(f"out must be {dt} or torch.float32, got {out.dtype}")
    if not _is(out, ot, (T, heads, D), at):
        _need_strided(out, "out", ot, (T, heads, D), dev, output=True)
    if lse is not None and not _is(lse, torch.float32, (T, heads), at):
        _need(lse, "lse", torch.float32, (T, heads), dev)
    need = _workspace_bytes("bt_attention_workspace_bytes", T, S, B, heads, kv_heads, D, P)
    if workspace is not None:
        _need_bytes(workspace, "workspace", need, dev)
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    qs, ks, vs, os = q.stride(), k.stride(), v.stride(), out.stride()
    shape = _ATTENTION_SHAPE.pack(T, S, B, P, heads, kv_heads, D, kind, _TYPES[ot], causal,
                                  D ** -0.5 if scale is None else scale, qs[0], qs[1], ks[0], ks[1], vs[0], vs[1],
                                  pk[0], pk[1], pv[0], pv[1], os[0], os[1])
    _call(dev, lib().bt_attention, shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), q_start.data_ptr(),
          k_start.data_ptr(), k_len.data_ptr(), _ptr(prefix_k), _ptr(prefix_v), out.data_ptr(), _ptr(lse),
          _ptr(workspace))
    return out, lse
