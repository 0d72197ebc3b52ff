"""A cache of keys and values held in 4 bits, in pages, and the attention that reads it (bt_cache4_*,
bt_attention4, bt_pages_*): argument checks and marshalling only, as in api.py.

A decode step over such a cache: ``pages_grow`` gives the new tokens their places, ``qk_norm_rope`` their
queries, keys and values, ``cache4_write`` puts these in, ``attention4`` reads. ``pages_fork`` reorders beams,
shares prompts and drops what has ended; ``pages_compact`` brings the pages in use together.
"""
from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass, field

import torch

from . import api

from .api import _HALF, _TYPES, _call, _is, _need, _need_bytes, _need_strided, _ptr, _type_of, _workspace_bytes

_ROWS_SHAPE = struct.Struct("10q")  # bt_cache4_rows
_ATTENTION4_SHAPE = struct.Struct("9q3if4q")  # bt_attention4_shape
_PAGES_SHAPE = struct.Struct("8q")  # bt_pages_shape


def cache4_page_bytes(page_tokens: int, kv_heads: int, head_dim: int) -> int:
    """bt_cache4_page_bytes: bytes of one layer's page (0: a shape the cache does not take)."""
    return _workspace_bytes("bt_cache4_page_bytes", page_tokens, kv_heads, head_dim)


@dataclass(frozen=True, eq=False)
class Cache4:
    """Pages of keys and values in 4 bits: ``layers`` times ``pages`` pages of ``page_tokens`` places (a power of
    two, 16 to 1024). ``data`` [layers, pages, page_bytes] uint8 is made (zeros) where none is given."""

    pages: int
    page_tokens: int
    kv_heads: int
    head_dim: int
    layers: int = 1
    data: torch.Tensor | None = None
    device: str | torch.device = "cuda"

    def __post_init__(self):
        size = cache4_page_bytes(self.page_tokens, self.kv_heads, self.head_dim)
        if not size or self.pages < 0 or self.layers < 1 or self.pages * self.page_tokens > 1 << 30:
            raise ValueError(f"no cache of {self.layers} x {self.pages} pages of {self.page_tokens} tokens with "
                             f"{self.kv_heads} key heads of {self.head_dim}")
        if self.data is None:
            object.__setattr__(self, "data", torch.zeros((self.layers, self.pages, size), dtype=torch.uint8,
                                                         device=self.device))
        _need(self.data, "data", torch.uint8, (self.layers, self.pages, size))
        object.__setattr__(self, "device", self.data.device)
        object.__setattr__(self, "_layer_bytes", self.pages * size)

    def __setstate__(self, kept):  # perhaps loaded onto another device than it was saved from
        self.__dict__.update(kept, device=kept["data"].device)

    def _layer(self, layer: int) -> int:
        """The address of a layer's pages."""
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer {layer} of {self.layers}")
        return self.data.data_ptr() + layer * self._layer_bytes


def _check_cache(cache):
    if not isinstance(cache, Cache4):
        raise TypeError(f"cache must be a Cache4, got {type(cache).__name__}")


def _rows_shape(cache, k, v, M, kind):
    ks, vs = k.stride(), v.stride()
    return _ROWS_SHAPE.pack(cache.pages, cache.page_tokens, cache.kv_heads, cache.head_dim, M, ks[0], ks[1], vs[0],
                            vs[1], kind)


def cache4_write(cache: Cache4, k: torch.Tensor, v: torch.Tensor, rows: torch.Tensor, layer: int = 0) -> None:
    """bt_cache4_write: ``k`` and ``v`` [M, kv_heads, head_dim] (fp32, bf16 or fp16) into places ``rows`` [M] int32
    of the cache (outside it: not written; no place twice), rounded to 4 bits."""
    _check_cache(cache)
    kind, dev = _type_of(k, "k", _TYPES), cache.device
    if not isinstance(rows, torch.Tensor) or rows.dim() != 1:
        raise ValueError("rows must be a 1-D tensor, one place per token")
    M, at = rows.shape[0], cache.data.get_device()
    shape = (M, cache.kv_heads, cache.head_dim)
    if not (_is(k, k.dtype, shape, at) and _is(v, k.dtype, shape, at) and _is(rows, torch.int32, (M,), at)):
        _need_strided(k, "k", k.dtype, shape, dev)
        _need_strided(v, "v", k.dtype, shape, dev)
        _need(rows, "rows", torch.int32, (M,), dev)
    base = cache._layer(layer)
    _call(dev, api.lib().bt_cache4_write, _rows_shape(cache, k, v, M, kind), k.data_ptr(), v.data_ptr(),
          rows.data_ptr(), base)


def cache4_read(cache: Cache4, rows: torch.Tensor, layer: int = 0, out=None, dtype: torch.dtype = torch.bfloat16):
    """bt_cache4_read: the keys and values of places ``rows`` [M] int32 (outside the cache: zeros) as two tensors
    [M, kv_heads, head_dim] of ``dtype`` (bf16 holds them exactly), or into ``out`` = (k, v). Returns (k, v)."""
    _check_cache(cache)
    dev = cache.device
    if not isinstance(rows, torch.Tensor) or rows.dim() != 1:
        raise ValueError("rows must be a 1-D tensor, one place per token")
    M, at = rows.shape[0], cache.data.get_device()
    shape = (M, cache.kv_heads, cache.head_dim)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev), torch.empty(shape, dtype=dtype, device=dev)
    k, v = out
    kind = _type_of(k, "k", _TYPES)
    if not (_is(k, k.dtype, shape, at) and _is(v, k.dtype, shape, at) and _is(rows, torch.int32, (M,), at)):
        _need_strided(k, "k", k.dtype, shape, dev, output=True)
        _need_strided(v, "v", k.dtype, shape, dev, output=True)
        _need(rows, "rows", torch.int32, (M,), dev)
    base = cache._layer(layer)
    _call(dev, api.lib().bt_cache4_read, _rows_shape(cache, k, v, M, kind), base, rows.data_ptr(), k.data_ptr(),
          v.data_ptr())
    return k, v


def attention4_workspace_bytes(tokens: int, seqs: int, heads: int, kv_heads: int, head_dim: int, max_pages: int,
                               page_tokens: int) -> int:
    """bt_attention4_workspace_bytes: the scratch of an attention4 call (0: none)."""
    return _workspace_bytes("bt_attention4_workspace_bytes", tokens, seqs, heads, kv_heads, head_dim, max_pages,
                            page_tokens)


def attention4_workspace(q: torch.Tensor, cache: Cache4, table: torch.Tensor) -> torch.Tensor | None:
    """A workspace for attention4 of these arrays (its contents do not matter), or None where none is needed."""
    n = attention4_workspace_bytes(q.shape[0], table.shape[0], q.shape[1], cache.kv_heads, cache.head_dim,
                                   table.shape[1], cache.page_tokens)
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def attention4_plan(tokens: int, seqs: int, heads: int, kv_heads: int, head_dim: int, max_pages: int, page_tokens: int,
                    dtype: torch.dtype = torch.bfloat16, out_dtype: torch.dtype | None = None) -> str:
    """bt_attention4_plan: the kernel instances that such an attention4 call would launch (host-only query)."""
    for t in (dtype, out_dtype or dtype):
        if t not in _TYPES:
            raise TypeError(f"dtype and out_dtype must be of {[str(a) for a in _TYPES]}, got {t}")
    shape = _ATTENTION4_SHAPE.pack(tokens, seqs, max_pages, max_pages, 0, page_tokens, heads, kv_heads, head_dim,
                                   _TYPES[dtype], _TYPES[out_dtype or dtype], True, 1.0, 0, 0, 0, 0)
    buf = ctypes.create_string_buffer(128)
    api.check(api.lib().bt_attention4_plan(shape, buf, len(buf)))
    return buf.value.decode()


def attention4(q: torch.Tensor, cache: Cache4, table: torch.Tensor, k_len: torch.Tensor, q_start: torch.Tensor,
               layer: int = 0, causal: bool = True, scale: float | None = None, out: torch.Tensor | None = None,
               out_dtype: torch.dtype | None = None, lse: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None):
    """bt_attention4: softmax attention of packed sequences with grouped heads over a 4-bit cache.

    ``q`` [T, heads, D] (bf16 or fp16, row and head strides of whole eights). Sequence b has queries q_start[b] ..
    q_start[b + 1] and as keys the first k_len[b] tokens in pages ``table`` [seqs, max_pages] row b (int32, on the
    device: ``Pages.table`` and ``Pages.length``); ``causal``: its last query sees all of them. ``scale`` defaults to
    D ** -0.5. ``out`` [T, heads, D] in q's type or fp32 (``out_dtype``); ``lse`` [T, heads] fp32 receives the log of
    the softmax's sum. Rows of no sequence are not written. Returns (out, lse)."""
    _check_cache(cache)
    kind = _type_of(q, "q", _HALF)
    if q.dim() != 3:
        raise ValueError(f"q must be [T, heads, D], got shape {tuple(q.shape)}")
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a tensor [seqs, max_pages]")
    (T, heads, D), (B, W), dev, dt = q.shape, table.shape, cache.device, q.dtype
    if D != cache.head_dim or heads < 1 or heads % cache.kv_heads:
        raise ValueError(f"{heads} heads of {D} over a cache of {cache.kv_heads} key heads of {cache.head_dim}")
    i32, f32, at = torch.int32, torch.float32, cache.data.get_device()
    if not (_is(q, dt, q.shape, at) and _is(table, i32, table.shape, at) and _is(k_len, i32, (B,), at)
            and _is(q_start, i32, (B + 1,), at)):
        _need_strided(q, "q", dt, q.shape, dev)
        _need_strided(table, "table", i32, table.shape, dev)
        _need(k_len, "k_len", i32, (B,), dev)
        _need(q_start, "q_start", i32, (B + 1,), dev)
    if out is None:
        out = torch.empty((T, heads, D), dtype=out_dtype or dt, device=dev)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    ot = out.dtype
    if ot is not dt and ot is not f32:
        raise TypeError(f"out must be {dt} or torch.float32, got {out.dtype}")
    if not _is(out, ot, (T, heads, D), at):
        _need_strided(out, "out", ot, (T, heads, D), dev, output=True)
    if lse is not None and not _is(lse, f32, (T, heads), at):
        _need(lse, "lse", f32, (T, heads), dev)
    need = _workspace_bytes("bt_attention4_workspace_bytes", T, B, heads, cache.kv_heads, D, W, cache.page_tokens)
    if workspace is not None:
        _need_bytes(workspace, "workspace", need, dev)
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    qs, os, base = q.stride(), out.stride(), cache._layer(layer)
    shape = _ATTENTION4_SHAPE.pack(T, B, W, table.stride(0) if B > 1 else W, cache.pages, cache.page_tokens, heads,
                                   cache.kv_heads, D, kind, _TYPES[ot], causal, D ** -0.5 if scale is None else scale,
                                   qs[0], qs[1], os[0], os[1])
    _call(dev, api.lib().bt_attention4, shape, q.data_ptr(), base, table.data_ptr(),
          q_start.data_ptr(), k_len.data_ptr(), out.data_ptr(), _ptr(lse), _ptr(workspace))
    return out, lse


# ------------------------------------------------------------------------- the pages' bookkeeping


@dataclass(frozen=True, eq=False)
class Pages:
    """Which of ``seqs`` sequences holds which of ``pages`` pages of ``page_tokens`` tokens (a power of two up to
    1024), all of it on the device: ``table`` [seqs, max_pages] (-1 behind a sequence's pages), ``length`` [seqs] in
    tokens, ``refs`` [pages] (how many entries hold a page; 0: free) and ``first`` [1] (no page below it is free), int32
    views of one array ``state`` in this order, which can be copied to keep or go back to a state. Starts empty. A deep,
    pickled or saved copy is a second table with arrays of its own."""

    seqs: int
    max_pages: int
    pages: int
    page_tokens: int
    device: str | torch.device = "cuda"
    state: torch.Tensor = field(init=False)

    def __post_init__(self):
        need = _workspace_bytes("bt_pages_workspace_bytes", self.seqs, self.max_pages, self.pages)
        tokens = self.page_tokens
        if not need or not 1 <= tokens <= 1024 or tokens & (tokens - 1) or max(self.pages, self.max_pages) * tokens > 1 << 30:
            raise ValueError(f"no table of {self.seqs} x {self.max_pages} over {self.pages} pages of {tokens} tokens")
        cells = self.seqs * self.max_pages
        state = torch.zeros(cells + self.seqs + self.pages + 1, dtype=torch.int32, device=self.device)
        state[:cells] = -1
        self._hold(state)

    def _hold(self, state):
        """Makes ``state`` this object's, with views of it and a workspace."""
        cells = self.seqs * self.max_pages
        parts = state.split([cells, self.seqs, self.pages, 1])
        need = _workspace_bytes("bt_pages_workspace_bytes", self.seqs, self.max_pages, self.pages)
        for name, value in (("state", state), ("table", parts[0].view(self.seqs, self.max_pages)),
                            ("length", parts[1]), ("refs", parts[2]), ("first", parts[3]), ("device", state.device),
                            ("_need", need), ("_workspace", torch.empty(need, dtype=torch.uint8, device=state.device)),
                            ("_offsets", (4 * cells, 4 * (cells + self.seqs), 4 * (cells + self.seqs + self.pages)))):
            object.__setattr__(self, name, value)

    # A copy, by copy.deepcopy, pickle or torch.save, has its own state, and views and a workspace of it; copy.copy shares
    # the state.
    def __getstate__(self):
        return {name: getattr(self, name) for name in ("seqs", "max_pages", "pages", "page_tokens", "state")}

    def __setstate__(self, kept):
        for name, value in kept.items():
            object.__setattr__(self, name, value)
        self._hold(self.state)

    def _arrays(self):
        """The addresses of table, length, refs and first, asked for at every call: a copy's are its own."""
        at, (length, refs, first) = self.state.data_ptr(), self._offsets
        return at, at + length, at + refs, at + first

    def _shape(self, pool=None, tokens: int = 0):
        layers = stride = size = 0
        if pool is not None:
            layers, stride, size = pool
        return _PAGES_SHAPE.pack(self.seqs, self.max_pages, self.pages, self.page_tokens, layers, stride, size, tokens)

    def _scratch(self, workspace):
        if workspace is None:
            return self._workspace.data_ptr()
        _need_bytes(workspace, "workspace", self._need, self.device)
        return workspace.data_ptr()


def _check_pages(pages):
    if not isinstance(pages, Pages):
        raise TypeError(f"pages must be a Pages, got {type(pages).__name__}")


def _pool(pool, pages: int, dev, page_tokens: int | None = None):
    """((layers, bytes between layers, bytes of a page), address) of a pool: a Cache4 (of ``page_tokens``, where given),
    or a tensor [layers, pages, ...] of whole 16 bytes a page."""
    if isinstance(pool, Cache4):
        if page_tokens is not None and pool.page_tokens != page_tokens:
            raise ValueError(f"the pool is a Cache4 with pages of {pool.page_tokens} tokens, the table's have {page_tokens}")
        pool = pool.data
    if not isinstance(pool, torch.Tensor) or pool.dim() < 3:
        raise ValueError("pool must be a Cache4 or a tensor [layers, pages, ...]")
    if pool.get_device() != (-1 if dev.index is None else dev.index) or not pool.is_contiguous() or pool.shape[1] != pages:
        _need(pool, "pool", pool.dtype, (pool.shape[0], pages, *pool.shape[2:]), dev)
    each = pool.element_size()
    for n in pool.shape[2:]:
        each *= n
    if each % 16:
        raise ValueError(f"pages of {each} bytes: not whole 16 bytes")
    if not pool.numel():
        return (0, 0, 0), 0
    return (pool.shape[0], pages * each, each), pool.data_ptr()


def pages_grow(pages: Pages, q_start: torch.Tensor, pool, out=None, tokens: int | None = None,
               workspace: torch.Tensor | None = None):
    """bt_pages_grow: room for q_start[b + 1] - q_start[b] new tokens of every sequence b (``q_start`` [seqs + 1]
    int32 on the device, as attention4 takes it). A partly filled last page that others hold too is copied in ``pool``
    (a Cache4 of the same page_tokens, or a tensor [layers, pages, ...]). Returns (rows, positions, granted): the place of
    each new token (-1: refused), its number in its sequence, and the tokens each sequence got (all it asked for, or
    0). ``tokens``, the rows of the first two, is q_start's last entry where the host knows it; or pass ``out`` = (rows,
    positions, granted)."""
    _check_pages(pages)
    dev, i32, at = pages.device, torch.int32, pages.state.get_device()
    if not _is(q_start, i32, (pages.seqs + 1,), at):
        _need(q_start, "q_start", i32, (pages.seqs + 1,), dev)
    if out is None:
        if tokens is None:
            raise ValueError("tokens (the number of new tokens) or out is needed")
        out = tuple(torch.empty(n, dtype=i32, device=dev) for n in (tokens, tokens, pages.seqs))
    rows, positions, granted = out
    if not isinstance(rows, torch.Tensor) or rows.dim() != 1:
        raise ValueError("rows must be a 1-D tensor, one place per new token")
    T = rows.shape[0]
    if tokens is not None and tokens != T:
        raise ValueError(f"tokens = {tokens}, but rows has {T}")
    if not (_is(rows, i32, (T,), at) and _is(positions, i32, (T,), at) and _is(granted, i32, (pages.seqs,), at)):
        _need(rows, "rows", i32, (T,), dev)
        _need(positions, "positions", i32, (T,), dev)
        _need(granted, "granted", i32, (pages.seqs,), dev)
    over, base = _pool(pool, pages.pages, dev, pages.page_tokens)
    table, length, refs, first = pages._arrays()
    scratch = pages._scratch(workspace)
    _call(dev, api.lib().bt_pages_grow, pages._shape(over, T), table, length, refs, first, q_start.data_ptr(), base,
          rows.data_ptr(), positions.data_ptr(), granted.data_ptr(), scratch)
    return rows, positions, granted


def pages_fork(pages: Pages, parent: torch.Tensor, workspace: torch.Tensor | None = None) -> None:
    """bt_pages_fork: every sequence b becomes what sequence ``parent`` [seqs] int32 [b] was (itself: as it is;
    outside [0, seqs): nothing, its pages freed where no other sequence holds them). Nothing is copied."""
    _check_pages(pages)
    if not _is(parent, torch.int32, (pages.seqs,), pages.state.get_device()):
        _need(parent, "parent", torch.int32, (pages.seqs,), pages.device)
    scratch = pages._scratch(workspace)
    _call(pages.device, api.lib().bt_pages_fork, pages._shape(), *pages._arrays(), parent.data_ptr(), scratch)


def pages_compact(pages: Pages, pool, workspace: torch.Tensor | None = None) -> None:
    """bt_pages_compact: the pages in use, L of them, to places 0 .. L - 1 of ``pool`` (as in pages_grow), tables
    and counts with them. ``pages.first`` then holds L."""
    _check_pages(pages)
    over, base = _pool(pool, pages.pages, pages.device, pages.page_tokens)
    table, _, refs, first = pages._arrays()
    scratch = pages._scratch(workspace)
    _call(pages.device, api.lib().bt_pages_compact, pages._shape(over), table, refs, first, base, scratch)


def pages_copy(pool, src: torch.Tensor, dst: torch.Tensor) -> None:
    """bt_pages_copy: page dst[i] of ``pool`` (a Cache4, or a tensor [layers, pages, ...]) becomes a copy of page
    src[i], in all layers (``src`` and ``dst`` [n] int32 on the device; numbers outside the pool are left out)."""
    data = pool.data if isinstance(pool, Cache4) else pool
    if not isinstance(data, torch.Tensor) or data.dim() < 3:
        raise ValueError("pool must be a Cache4 or a tensor [layers, pages, ...]")
    dev = data.device
    if not isinstance(src, torch.Tensor) or src.dim() != 1:
        raise ValueError("src must be a 1-D tensor of page numbers")
    _need(src, "src", torch.int32, None, dev)
    _need(dst, "dst", torch.int32, src.shape, dev)
    (layers, stride, size), base = _pool(data, data.shape[1], dev)
    shape = _PAGES_SHAPE.pack(0, 0, data.shape[1], 1, layers, stride, size, 0)
    _call(dev, api.lib().bt_pages_copy, shape, base, src.data_ptr(), dst.data_ptr(), src.shape[0])
