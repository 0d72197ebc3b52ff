"""Refusals of the 4-bit cache, its attention, the pages' bookkeeping and the int8 product, by the C ABI and by the
wrapper: everything is checked on the host before a launch, so these run without a GPU."""
import struct

import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests.test_abi import BT_ERR_ALIGN, BT_ERR_NULL, BT_ERR_SHAPE, BT_ERR_UNSUPPORTED, BT_OK, FAKE
from tests.test_api_validation import host_ok  # noqa: F401  (fixture)

F32, BF16, F16 = 0, 1, 2
BIG = 1 << 40


# --------------------------------------------------------------------------- cache rows


def _rows(call="write", pages=4, page=16, kv=2, D=64, tokens=3, strides=(128, 64, 128, 64), type=BF16, shape=True, k=FAKE,
          v=FAKE, rows=FAKE, cache=FAKE):
    s = struct.pack("10q", pages, page, kv, D, tokens, *strides, type) if shape else None
    if call == "write":
        return bt.lib().bt_cache4_write(s, k, v, rows, cache, None)
    return bt.lib().bt_cache4_read(s, cache, rows, k, v, None)


@pytest.mark.parametrize("call", ["write", "read"])
def test_cache_rows_refusals(call):
    assert _rows(call, shape=False) == BT_ERR_NULL
    for page in (0, -16, 8, 24, 2048, BIG):
        assert _rows(call, page=page) == BT_ERR_SHAPE, page
    for D in (0, -8, 4, 60, 264):
        assert _rows(call, D=D) == BT_ERR_SHAPE, D
    assert _rows(call, kv=0) == BT_ERR_SHAPE and _rows(call, kv=40000) == BT_ERR_SHAPE and _rows(call, kv=BIG) == BT_ERR_SHAPE
    assert _rows(call, pages=-1) == BT_ERR_SHAPE and _rows(call, pages=(1 << 26) + 1) == BT_ERR_SHAPE
    assert _rows(call, pages=1 << 62) == BT_ERR_SHAPE
    assert _rows(call, tokens=-1) == BT_ERR_SHAPE and _rows(call, tokens=(1 << 23) + 1) == BT_ERR_SHAPE
    assert _rows(call, tokens=1 << 23, kv=64) == BT_ERR_SHAPE  # one launch's work-items
    assert _rows(call, type=3) == BT_ERR_UNSUPPORTED and _rows(call, type=-1) == BT_ERR_UNSUPPORTED
    for name in ("k", "v", "rows", "cache"):
        assert _rows(call, **{name: 0}) == BT_ERR_NULL, name
    for name, off in (("k", 4), ("v", 2), ("rows", 2), ("cache", 8)):
        assert _rows(call, **{name: FAKE + off}) == BT_ERR_ALIGN, name
    assert _rows(call, k=FAKE + 8, type=F32) == BT_ERR_ALIGN
    for i in range(4):
        bad = [128, 64, 128, 64]
        bad[i] = 66
        assert _rows(call, strides=bad) == BT_ERR_ALIGN
        bad[i] = -64
        assert _rows(call, strides=bad) == BT_ERR_ALIGN
    assert _rows(call, tokens=0, k=0, v=0, rows=0, cache=0) == BT_OK


def test_cache_writes_nothing_without_pages():
    assert _rows("write", pages=0, cache=0) == BT_OK


def test_cache_page_bytes():
    f = bt.cache4_page_bytes
    assert f(16, 1, 8) == 16 * 34 and f(64, 5, 128) == 64 * 5 * 4 * 34 and f(16, 3, 80) == 16 * 3 * 3 * 34
    assert f(17, 1, 64) == 0 and f(16, 0, 64) == 0 and f(16, 1, 260) == 0


# ---------------------------------------------------------------------------- attention


def _attention(tokens=2, seqs=1, W=3, row=3, pages=4, page=16, heads=4, kv=2, D=64, type=BF16, out_type=BF16, scale=0.1,
               strides=(256, 64, 256, 64), shape=True, q=FAKE, cache=FAKE, table=FAKE, q_start=FAKE, k_len=FAKE, out=FAKE,
               lse=0, ws=FAKE):
    s = struct.pack("9q3if4q", tokens, seqs, W, row, pages, page, heads, kv, D, type, out_type, 1, scale, *strides) if shape else None
    return bt.lib().bt_attention4(s, q, cache, table, q_start, k_len, out, lse, ws, None)


def test_attention4_refusals():
    assert _attention(shape=False) == BT_ERR_NULL
    for name in ("tokens", "seqs"):
        assert _attention(**{name: -1}) == BT_ERR_SHAPE and _attention(**{name: (1 << 23) + 1}) == BT_ERR_SHAPE
    assert _attention(heads=3) == BT_ERR_SHAPE and _attention(heads=0) == BT_ERR_SHAPE and _attention(heads=1 << 17) == BT_ERR_SHAPE
    assert _attention(kv=0) == BT_ERR_SHAPE and _attention(D=12) == BT_ERR_SHAPE and _attention(D=264) == BT_ERR_SHAPE
    assert _attention(tokens=1 << 23, heads=256) == BT_ERR_SHAPE
    assert _attention(page=48) == BT_ERR_SHAPE and _attention(page=8) == BT_ERR_SHAPE
    assert _attention(W=-1) == BT_ERR_SHAPE and _attention(W=(1 << 26) + 1, row=1 << 30) == BT_ERR_SHAPE and _attention(W=1 << 60) == BT_ERR_SHAPE
    assert _attention(pages=-1) == BT_ERR_SHAPE and _attention(pages=1 << 27) == BT_ERR_SHAPE
    assert _attention(row=2) == BT_ERR_SHAPE
    assert _attention(tokens=1 << 23, seqs=1 << 23, heads=64, kv=64) == BT_ERR_SHAPE  # work items
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert _attention(scale=scale) == BT_ERR_SHAPE
    assert _attention(type=F32, out_type=F32) == BT_ERR_UNSUPPORTED and _attention(type=F16, out_type=BF16) == BT_ERR_UNSUPPORTED
    for name in ("q", "cache", "table", "q_start", "k_len", "out"):
        assert _attention(**{name: 0}) == BT_ERR_NULL, name
    assert _attention(W=1000, row=1000, ws=0) == BT_ERR_NULL
    assert _attention(W=1000, row=1000, ws=FAKE + 64) == BT_ERR_ALIGN
    for name, off in (("q", 8), ("cache", 8), ("table", 2), ("q_start", 2), ("k_len", 2), ("out", 4), ("lse", 2)):
        assert _attention(**{name: FAKE + off}) == BT_ERR_ALIGN, name
    assert _attention(strides=(260, 64, 256, 64)) == BT_ERR_ALIGN and _attention(strides=(256, 64, 256, 66)) == BT_ERR_ALIGN
    assert _attention(strides=(256, -64, 256, 64)) == BT_ERR_ALIGN
    assert _attention(tokens=0, q=0, out=0) == BT_OK and _attention(seqs=0, q_start=0, k_len=0) == BT_OK


def test_attention4_workspace():
    f = bt.attention4_workspace_bytes
    assert f(1, 1, 4, 2, 64, 32, 16) == 0  # 512 keys go uncut
    assert f(1, 1, 4, 2, 64, 1000, 16) > 0 and f(1, 1, 4, 2, 64, 1000, 16) % 256 == 0
    assert f(0, 1, 4, 2, 64, 1000, 16) == 0 and f(1, 1, 3, 2, 64, 1000, 16) == 0


# -------------------------------------------------------------------------------- pages


def _pages(call, seqs=2, W=3, pages=8, page=16, layers=2, stride=8 * 64, size=64, tokens=4, shape=True, n=2, **ptr):
    s = struct.pack("8q", seqs, W, pages, page, layers, stride, size, tokens) if shape else None
    p = lambda name: ptr.get(name, FAKE)  # noqa: E731
    L = bt.lib()
    if call == "grow":
        return L.bt_pages_grow(s, p("table"), p("length"), p("refs"), p("first"), p("q_start"), p("pool"), p("rows"),
                               p("positions"), p("granted"), p("ws"), None)
    if call == "fork":
        return L.bt_pages_fork(s, p("table"), p("length"), p("refs"), p("first"), p("parent"), p("ws"), None)
    if call == "compact":
        return L.bt_pages_compact(s, p("table"), p("refs"), p("first"), p("pool"), p("ws"), None)
    return L.bt_pages_copy(s, p("pool"), p("src"), p("dst"), n, None)


POINTERS = {"grow": ["table", "length", "refs", "first", "q_start", "rows", "positions", "granted"],
            "fork": ["table", "length", "refs", "first", "parent"], "compact": ["table", "refs", "first"],
            "copy": ["src", "dst"]}


@pytest.mark.parametrize("call", ["grow", "fork", "compact", "copy"])
def test_pages_refusals(call):
    assert _pages(call, shape=False) == BT_ERR_NULL
    for page in (0, -1, 3, 2048):
        assert _pages(call, page=page) == BT_ERR_SHAPE
    assert _pages(call, pages=-1) == BT_ERR_SHAPE and _pages(call, pages=(1 << 24) + 1, page=1) == BT_ERR_SHAPE
    assert _pages(call, pages=(1 << 20) + 1, page=1024) == BT_ERR_SHAPE and _pages(call, pages=1 << 62) == BT_ERR_SHAPE
    assert _pages(call, W=-1) == BT_ERR_SHAPE and _pages(call, W=(1 << 26) + 1) == BT_ERR_SHAPE and _pages(call, W=1 << 62) == BT_ERR_SHAPE
    assert _pages(call, seqs=-1) == BT_ERR_SHAPE and _pages(call, seqs=1 << 16, W=1 << 15) == BT_ERR_SHAPE
    assert _pages(call, seqs=(1 << 23) + 1) == BT_ERR_SHAPE
    assert _pages(call, tokens=-1) == BT_ERR_SHAPE and _pages(call, tokens=(1 << 23) + 1) == BT_ERR_SHAPE
    for name in POINTERS[call]:
        assert _pages(call, **{name: 0}) == BT_ERR_NULL, name
        assert _pages(call, **{name: FAKE + 2}) == BT_ERR_ALIGN, name
    if call != "copy":
        assert _pages(call, ws=0) == BT_ERR_NULL and _pages(call, ws=FAKE + 8) == BT_ERR_ALIGN
    if call != "fork":
        for size in (0, 8, 24, -16, 1 << 31):
            assert _pages(call, size=size) == BT_ERR_SHAPE, size
        assert _pages(call, stride=8 * 64 - 16) == BT_ERR_SHAPE and _pages(call, stride=8 * 64 + 8) == BT_ERR_SHAPE
        assert _pages(call, layers=-1) == BT_ERR_SHAPE and _pages(call, layers=65537) == BT_ERR_SHAPE
        assert _pages(call, pool=0) == BT_ERR_NULL and _pages(call, pool=FAKE + 8) == BT_ERR_ALIGN
    if call == "copy":
        assert _pages(call, n=-1) == BT_ERR_SHAPE and _pages(call, n=1 << 25) == BT_ERR_SHAPE
        assert _pages(call, n=0, src=0, dst=0) == BT_OK and _pages(call, layers=0, pool=0) == BT_OK
    if call == "compact":
        assert _pages(call, pages=0, stride=0) == BT_OK
    if call == "fork":
        assert _pages(call, seqs=0) == BT_OK
    if call == "grow":
        assert _pages(call, seqs=0, tokens=0, table=0) == BT_OK


def test_pages_workspace():
    f = bt.lib().bt_pages_workspace_bytes
    assert f(2, 3, 8) >= 4 * (4 + 8 + 8) and f(-1, 3, 8) == 0 and f(2, 3, (1 << 24) + 1) == 0
    assert f(100, 500, 10) >= 4 * 100 * 501


# --------------------------------------------------------------------------------- int8


def _int8(M=3, N=5, K=100, type=F32, Wp=FAKE, sw=FAKE, X=FAKE, sx=FAKE, bias=0, Y=FAKE, acc=0, ws=FAKE):
    return bt.lib().bt_int8_gemm(Wp, sw, X, sx, M, N, K, bias, Y, type, acc, ws, None)


def test_int8_refusals():
    for bad in ({"M": -1}, {"M": (1 << 23) + 1}, {"N": -1}, {"N": (1 << 23) + 1}, {"K": -1}, {"K": 131073},
                {"M": 1 << 22, "N": (1 << 14) + 1}, {"N": 1 << 23, "K": 1 << 14}):
        assert _int8(**bad) == BT_ERR_SHAPE, bad
    assert _int8(type=3) == BT_ERR_UNSUPPORTED
    assert _int8(Y=0) == BT_ERR_NULL
    for name in ("Wp", "sw", "X", "sx"):
        assert _int8(**{name: 0}) == BT_ERR_NULL, name
    for name, off in (("Wp", 8), ("X", 8), ("sw", 2), ("sx", 2), ("bias", 2), ("Y", 2), ("acc", 2)):
        assert _int8(**{name: FAKE + off}) == BT_ERR_ALIGN, name
    assert _int8(type=BF16, Y=FAKE + 1) == BT_ERR_ALIGN
    assert _int8(M=0, Y=0) == BT_OK and _int8(N=0, Y=0) == BT_OK


def test_int8_pack_refusals():
    f = bt.lib().bt_int8_pack
    assert f(FAKE, 100, -1, 100, FAKE, None) == BT_ERR_SHAPE and f(FAKE, 99, 5, 100, FAKE, None) == BT_ERR_SHAPE
    assert f(FAKE, 1 << 18, 5, 131073, FAKE, None) == BT_ERR_SHAPE
    assert f(0, 100, 5, 100, FAKE, None) == BT_ERR_NULL and f(FAKE, 100, 5, 100, 0, None) == BT_ERR_NULL
    assert f(FAKE, 100, 5, 100, FAKE + 8, None) == BT_ERR_ALIGN
    assert f(0, 0, 0, 0, 0, None) == BT_OK
    assert bt.int8_weight_bytes(17, 65) == 32 * 128 and bt.int8_weight_bytes(0, 5) == 0 and bt.int8_weight_bytes(5, 131073) == 0


# ------------------------------------------------------------------------------ wrapper


def test_cpu_tensors_are_rejected():
    data = torch.zeros((1, 2, bt.cache4_page_bytes(16, 1, 64)), dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        bt.Cache4(2, 16, 1, 64, data=data)
    with pytest.raises(ValueError, match="device tensor"):
        bt.pack_int8(torch.zeros((2, 2), dtype=torch.int8), torch.ones(2))


def cache(layers=1):
    return bt.Cache4(4, 16, 2, 64, layers=layers, device="cpu")


def test_cache4_class(host_ok):  # noqa: F811
    for bad in ((4, 24, 2, 64), (4, 16, 0, 64), (4, 16, 2, 60), (-1, 16, 2, 64), (1 << 27, 16, 2, 64)):
        with pytest.raises(ValueError, match="no cache"):
            bt.Cache4(*bad, device="cpu")
    with pytest.raises(ValueError, match="no cache"):
        bt.Cache4(4, 16, 2, 64, layers=0, device="cpu")
    size = bt.cache4_page_bytes(16, 2, 64)
    with pytest.raises(ValueError, match="data must have shape"):
        bt.Cache4(4, 16, 2, 64, data=torch.zeros((4, size), dtype=torch.uint8))
    with pytest.raises(TypeError, match="data must be"):
        bt.Cache4(4, 16, 2, 64, data=torch.zeros((1, 4, size), dtype=torch.int8))
    with pytest.raises(ValueError, match="contiguous"):
        bt.Cache4(4, 16, 2, 64, data=torch.zeros((1, 4, size + 16), dtype=torch.uint8)[..., :size])
    assert cache(3).data.shape == (3, 4, size)


def test_cache4_write_and_read_refuse(host_ok):  # noqa: F811
    c, k, rows = cache(), torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError, match="Cache4"):
        bt.cache4_write(c.data, k, k, rows)
    with pytest.raises(TypeError, match="k must be one of"):
        bt.cache4_write(c, k.double(), k.double(), rows)
    with pytest.raises(TypeError, match="v must be"):
        bt.cache4_write(c, k, k.float(), rows)
    with pytest.raises(ValueError, match="k must have shape"):
        bt.cache4_write(c, k[:, :1], k, rows)
    with pytest.raises(ValueError, match="v must have shape"):
        bt.cache4_write(c, k, k[:2], rows)
    with pytest.raises(TypeError, match="rows must be"):
        bt.cache4_write(c, k, k, rows.long())
    with pytest.raises(ValueError, match="rows must be"):
        bt.cache4_write(c, k, k, rows.view(1, 3))
    with pytest.raises(ValueError, match="last dimension"):
        bt.cache4_write(c, torch.zeros((3, 2, 128), dtype=torch.bfloat16)[..., ::2], k, rows)
    with pytest.raises(ValueError, match="layer 1 of 1"):
        bt.cache4_write(c, k, k, rows, layer=1)
    with pytest.raises(ValueError, match="overlap"):
        bt.cache4_read(c, rows, out=(torch.zeros((1, 2, 64)).expand(3, 2, 64), torch.zeros((3, 2, 64))))
    with pytest.raises(ValueError, match="v must have shape"):
        bt.cache4_read(c, rows, out=(torch.zeros((3, 2, 64)), torch.zeros((3, 2, 32))))
    with pytest.raises(ValueError, match="layer -1"):
        bt.cache4_read(c, rows, layer=-1)


def test_attention4_wrapper_refuses(host_ok):  # noqa: F811
    c, q = cache(), torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    table, n, start = torch.zeros((2, 5), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)

    def call(q=q, table=table, k_len=n, q_start=start, **more):
        return bt.attention4(q, c, table, k_len, q_start, **more)

    for bad, kind, match in (({"q": q.float()}, TypeError, "q must be one of"), ({"q": q[0]}, ValueError, "q must be"),
                             ({"q": q[..., :32]}, ValueError, "over a cache"), ({"q": q[:, :3]}, ValueError, "over a cache"),
                             ({"table": table[0]}, ValueError, "table must be"), ({"table": table.long()}, TypeError, "table must be"),
                             ({"table": table.t().contiguous().t()}, ValueError, "last dimension"),
                             ({"k_len": n[:1]}, ValueError, "k_len must have shape"), ({"k_len": n.long()}, TypeError, "k_len must be"),
                             ({"q_start": n}, ValueError, "q_start must have shape"), ({"layer": 1}, ValueError, "layer"),
                             ({"out": torch.zeros((3, 4, 64), dtype=torch.float16)}, TypeError, "out must be"),
                             ({"out": q, "out_dtype": torch.float32}, TypeError, "out is"),
                             ({"out": torch.zeros((3, 4, 32), dtype=torch.bfloat16)}, ValueError, "out must have shape"),
                             ({"lse": torch.zeros((3, 2))}, ValueError, "lse must have shape"),
                             ({"table": torch.zeros((2, 500), dtype=torch.int32), "workspace": torch.zeros(64)}, ValueError, "workspace")):
        with pytest.raises(kind, match=match):
            call(**bad)


def test_pages_wrapper_refuses(host_ok):  # noqa: F811
    for bad in ((2, 3, 8, 24), (-1, 3, 8, 16), (2, 1 << 27, 8, 16), (2, 3, 1 << 25, 16)):
        with pytest.raises(ValueError, match="no table"):
            bt.Pages(*bad, device="cpu")
    p = bt.Pages(2, 3, 8, 16, device="cpu")
    assert p.table.tolist() == [[-1] * 3] * 2 and p.length.tolist() == [0, 0] and p.refs.tolist() == [0] * 8 and p.first.tolist() == [0]
    p.length[1] = 5
    assert p.state[6 + 1] == 5
    pool, start = torch.zeros((1, 8, 32), dtype=torch.uint8), torch.zeros(3, dtype=torch.int32)
    one = torch.zeros(2, dtype=torch.int32)
    for args, more, kind, match in (((p, start[:2], pool), {"tokens": 2}, ValueError, "q_start must have shape"),
                                    ((p, start.long(), pool), {"tokens": 2}, TypeError, "q_start must be"),
                                    ((p, start, pool), {}, ValueError, "tokens"),
                                    ((p, start, pool), {"out": (one, one, one), "tokens": 3}, ValueError, "tokens = 3"),
                                    ((p, start, pool), {"out": (one, one[:1], one)}, ValueError, "positions must have shape"),
                                    ((p, start, pool), {"out": (one, one, start)}, ValueError, "granted must have shape"),
                                    ((p, start, pool[:, :7]), {"tokens": 2}, ValueError, "pool must"),
                                    ((p, start, pool[..., :24]), {"tokens": 2}, ValueError, "contiguous"),
                                    ((p, start, pool[..., :24].contiguous()), {"tokens": 2}, ValueError, "whole 16 bytes"),
                                    ((p, start, pool[0]), {"tokens": 2}, ValueError, "pool must be"),
                                    ((p, start, pool), {"tokens": 2, "workspace": torch.zeros(2)}, ValueError, "workspace"),
                                    ((p.state, start, pool), {"tokens": 2}, TypeError, "Pages")):
        with pytest.raises(kind, match=match):
            bt.pages_grow(*args, **more)
    with pytest.raises(ValueError, match="parent must have shape"):
        bt.pages_fork(p, start)
    with pytest.raises(TypeError, match="parent must be"):
        bt.pages_fork(p, one.long())
    with pytest.raises(ValueError, match="pool must have shape"):
        bt.pages_compact(p, pool[:, :7].contiguous())
    with pytest.raises(ValueError, match="dst must have shape"):
        bt.pages_copy(pool, one, start)
    with pytest.raises(TypeError, match="src must be"):
        bt.pages_copy(pool, one.float(), one)


def test_int8_wrapper_refuses(host_ok):  # noqa: F811
    w = bt.Int8Weight(torch.zeros(bt.int8_weight_bytes(10, 300), dtype=torch.uint8), torch.ones(10), 10, 300)
    with pytest.raises(ValueError, match="packed weights holds"):
        bt.Int8Weight(torch.zeros(100, dtype=torch.uint8), torch.ones(10), 10, 300)
    with pytest.raises(ValueError, match="weight scale must have shape"):
        bt.Int8Weight(w.data, torch.ones(9), 10, 300)
    with pytest.raises(TypeError, match="codes must be"):
        bt.pack_int8(torch.zeros((10, 300)), torch.ones(10))
    with pytest.raises(ValueError, match="contiguous"):
        bt.pack_int8(torch.zeros((300, 10), dtype=torch.int8).t(), torch.ones(10))
    x, s = torch.zeros((3, 512), dtype=torch.int8), torch.ones(3)
    for bad, kind, match in (({"q": (x[:, :300].contiguous(), s)}, ValueError, "Xq must have shape"),
                             ({"q": (x.float(), s)}, TypeError, "Xq must be"), ({"q": (x, s[:2])}, ValueError, "Xq must have shape"),
                             ({"q": (x, s.double())}, TypeError, "s_x must be"), ({"bias": torch.ones(9)}, ValueError, "bias must have"),
                             ({"out": torch.zeros((3, 9))}, ValueError, "out must have shape"),
                             ({"out": torch.zeros((3, 10), dtype=torch.float64)}, TypeError, "out must be one of"),
                             ({"out": torch.zeros((3, 20))[:, ::2]}, ValueError, "contiguous"),
                             ({"out_acc": torch.zeros((3, 10))}, TypeError, "out_acc must be")):
        with pytest.raises(kind, match=match):
            bt.int8_gemm(w, **{"q": (x, s), **bad})
    with pytest.raises(ValueError, match="X must be"):
        bt.int8_linear(torch.zeros((3, 299)), w)
    with pytest.raises(TypeError, match="Int8Weight"):
        bt.int8_gemm(x, (x, s))
