"""Refusals of the attention-block operators, by the wrapper and by the C ABI: everything is checked
on the host before a launch, so these run without a GPU."""
import ctypes
import struct

import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests.test_abi import BT_ERR_ALIGN, BT_ERR_NULL, BT_ERR_SHAPE, BT_ERR_UNSUPPORTED, BT_OK, FAKE
from tests.test_api_validation import host_ok  # noqa: F401  (fixture)

F32, BF16 = 0, 1


def _groups(*rows):
    arr = (ctypes.c_int64 * len(rows))(*rows)
    return ctypes.addressof(arr), len(rows), arr


def _lora(A=FAKE, B=FAKE, w=BF16, scale=FAKE, ranks=0, L=2, R=8, groups=None, adapter=FAKE, X=FAKE, Y0=0, M=4, N=64,
          K=64, Y=FAKE, ws=FAKE):
    ptr, n, keep = groups or (0, 0, None)
    return bt.lib().bt_lora_apply(A, B, w, scale, ranks, L, R, ptr, n, adapter, X, Y0, M, N, K, Y, ws, None)


def test_lora_abi_refusals():
    assert _lora(M=-1) == BT_ERR_SHAPE
    assert _lora(N=(1 << 23) + 1) == BT_ERR_SHAPE
    assert _lora(M=1 << 23, N=1 << 14) == BT_ERR_SHAPE
    assert _lora(M=1 << 23, N=(1 << 12) + 1) == BT_ERR_SHAPE  # one launch's work-items
    assert _lora(K=131073) == BT_ERR_SHAPE
    assert _lora(R=0) == BT_ERR_SHAPE
    assert _lora(R=257) == BT_ERR_SHAPE
    assert _lora(L=-1) == BT_ERR_SHAPE
    assert _lora(L=1 << 31) == BT_ERR_SHAPE
    assert _lora(w=3) == BT_ERR_UNSUPPORTED
    assert _lora(groups=_groups(32, 31)) == BT_ERR_SHAPE
    assert _lora(groups=_groups(32, 0, 32)) == BT_ERR_SHAPE
    assert _lora(groups=_groups(*[8] * 9), N=72) == BT_ERR_SHAPE
    assert _lora(groups=_groups(2 ** 63 - 1, 2 ** 63 - 1)) == BT_ERR_SHAPE
    for name in ("A", "B", "scale", "adapter", "X", "Y", "ws"):
        assert _lora(**{name: 0}) == BT_ERR_NULL, name
    for name in ("A", "B"):
        assert _lora(**{name: FAKE + 1}) == BT_ERR_ALIGN, name
        assert _lora(**{name: FAKE + 2}, w=F32) == BT_ERR_ALIGN, name
    for name in ("scale", "ranks", "adapter", "X", "Y0", "Y"):
        assert _lora(**{name: FAKE + 2}) == BT_ERR_ALIGN, name
    assert _lora(ws=FAKE + 128) == BT_ERR_ALIGN
    assert _lora(M=0) == BT_OK and _lora(N=0) == BT_OK


def test_lora_workspace_bytes():
    f = bt.lib().bt_lora_workspace_bytes
    assert f(0, 64, 8, 1) == 0 and f(4, 64, 0, 1) == 0 and f(4, 64, 8, 9) == 0 and f(4, -1, 8, 1) == 0
    # a multiple of one fp32 value per token, group and rank (rounded up to 16)
    for M, K, R, G in ((1, 2560, 16, 3), (64, 11008, 64, 1), (2048, 2560, 32, 2), (5, 0, 1, 1), (300, 131072, 256, 8)):
        unit = M * G * -(-R // 16) * 16 * 4
        assert f(M, K, R, G) % unit == 0 and 1 <= f(M, K, R, G) // unit <= 32


def _adapters(N=64, K=32, R=8, L=3, groups=None, dtype=torch.bfloat16):
    n = 1 if groups is None else len(groups)
    return bt.LoraAdapters(torch.zeros((L, n * R, K), dtype=dtype), torch.zeros((L, N, R), dtype=dtype),
                           torch.zeros(L), group_rows=groups)


def test_lora_adapters_refuse(host_ok):  # noqa: F811
    with pytest.raises(ValueError, match="A must have shape"):
        bt.LoraAdapters(torch.zeros((3, 8, 32)), torch.zeros((3, 64, 4)), torch.zeros(3))
    with pytest.raises(TypeError, match="A must be"):
        bt.LoraAdapters(torch.zeros((3, 4, 32)), torch.zeros((3, 64, 4)).half(), torch.zeros(3))
    with pytest.raises(TypeError, match="A must be one of"):
        bt.LoraAdapters(torch.zeros((3, 4, 32)).double(), torch.zeros((3, 64, 4)).double(), torch.zeros(3))
    with pytest.raises(ValueError, match="group_rows"):
        _adapters(groups=(32, 31))
    with pytest.raises(ValueError, match="rank"):
        _adapters(R=257)
    with pytest.raises(ValueError, match="scale must have shape"):
        bt.LoraAdapters(torch.zeros((3, 4, 32)), torch.zeros((3, 64, 4)), torch.zeros(2))
    with pytest.raises(TypeError, match="ranks must be"):
        bt.LoraAdapters(torch.zeros((3, 4, 32)), torch.zeros((3, 64, 4)), torch.zeros(3), ranks=torch.zeros(3))


def test_lora_apply_refuses(host_ok):  # noqa: F811
    ad, X, ix = _adapters(), torch.zeros((5, 32)), torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="X must have shape"):
        bt.lora_apply(torch.zeros((5, 31)), ad, ix)
    with pytest.raises(TypeError, match="index must be"):
        bt.lora_apply(X, ad, ix.long())
    with pytest.raises(ValueError, match="index must have shape"):
        bt.lora_apply(X, ad, ix[:4])
    with pytest.raises(ValueError, match="base must have shape"):
        bt.lora_apply(X, ad, ix, base=torch.zeros((5, 63)))
    with pytest.raises(ValueError, match="contiguous"):
        bt.lora_apply(X, ad, ix, out=torch.zeros((64, 5)).t())
    with pytest.raises(ValueError, match="workspace holds"):
        bt.lora_apply(X, ad, ix, workspace=torch.zeros(16, dtype=torch.uint8))
    pw = bt.PackedWeight(torch.zeros(bt.packed_weight_bytes(64, 32), dtype=torch.uint8), torch.zeros(1), 64, 32)
    with pytest.raises(ValueError, match="come together"):
        bt.linear(X, pw, adapters=ad)
    with pytest.raises(ValueError, match="the adapters are for"):
        bt.linear(X, pw, adapters=_adapters(N=60), adapter_index=ix)
    with pytest.raises(ValueError, match="want_y"):
        bt.linear(X, pw, want_y=False, want_acc=True, adapters=ad, adapter_index=ix)
    with pytest.raises(ValueError, match="adapter_index must have shape"):
        bt.linear(X, pw, adapters=ad, adapter_index=ix[:2])


def _qk(qkv=FAKE, in_type=F32, ld=8 * 64, M=4, heads=4, kv=2, D=64, qw=0, kw=0, eps=1e-6, pos=FAKE, inv=FAKE, rot=64,
        inter=0, rows=0, kv_rows=4, q=FAKE, k=FAKE, v=FAKE, out_type=BF16, strides=(256, 64, 128, 64, 128, 64)):
    shape = struct.pack("13q3if", M, heads, kv, D, rot, ld, kv_rows, *strides, in_type, out_type, inter, eps)
    return bt.lib().bt_qk_norm_rope(shape, qkv, qw, kw, pos, inv, rows, q, k, v, None)


def test_qk_norm_rope_abi_refusals():
    assert _qk(M=-1) == BT_ERR_SHAPE
    assert _qk(heads=5) == BT_ERR_SHAPE and _qk(heads=0) == BT_ERR_SHAPE and _qk(kv=0) == BT_ERR_SHAPE
    assert _qk(D=60) == BT_ERR_SHAPE and _qk(D=520) == BT_ERR_SHAPE and _qk(D=0, rot=0) == BT_ERR_SHAPE
    assert _qk(rot=72) == BT_ERR_SHAPE and _qk(rot=4) == BT_ERR_SHAPE and _qk(rot=-8) == BT_ERR_SHAPE
    assert _qk(eps=-1.0) == BT_ERR_SHAPE and _qk(eps=float("nan")) == BT_ERR_SHAPE
    assert _qk(eps=float("inf")) == BT_ERR_SHAPE
    assert _qk(kv_rows=3) == BT_ERR_SHAPE and _qk(kv_rows=-1, rows=FAKE) == BT_ERR_SHAPE
    assert _qk(in_type=3) == BT_ERR_UNSUPPORTED and _qk(out_type=-1) == BT_ERR_UNSUPPORTED
    for name in ("qkv", "q", "k", "v", "pos", "inv"):
        assert _qk(**{name: 0}) == BT_ERR_NULL, name
    assert _qk(qkv=FAKE + 8) == BT_ERR_ALIGN and _qk(ld=514) == BT_ERR_ALIGN
    assert _qk(q=FAKE + 4) == BT_ERR_ALIGN and _qk(qw=FAKE + 8) == BT_ERR_ALIGN
    assert _qk(strides=(256, 66, 128, 64, 128, 64)) == BT_ERR_ALIGN
    assert _qk(strides=(256, 64, 128, 64, -128, 64)) == BT_ERR_ALIGN
    assert _qk(pos=FAKE + 2) == BT_ERR_ALIGN and _qk(inv=FAKE + 4) == BT_ERR_ALIGN
    assert _qk(M=0, kv_rows=0) == BT_OK
    assert bt.lib().bt_qk_norm_rope(None, *[FAKE] * 9, None) == BT_ERR_NULL


def test_qk_norm_rope_refuses(host_ok):  # noqa: F811
    qkv, pos = torch.zeros((3, 4 * 64)), torch.zeros(3, dtype=torch.int32)
    inv = torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="not 5 heads"):
        bt.qk_norm_rope(qkv, pos, inv, 3, 1)
    with pytest.raises(ValueError, match="multiple of kv_heads"):
        bt.qk_norm_rope(qkv, pos, inv, 2, 0)
    with pytest.raises(TypeError, match="inv_freq must be"):
        bt.qk_norm_rope(qkv, pos, inv.float(), 2, 1)
    with pytest.raises(TypeError, match="positions must be"):
        bt.qk_norm_rope(qkv, pos.long(), inv, 2, 1)
    with pytest.raises(TypeError, match="positions must be a"):
        bt.qk_norm_rope(qkv, None, inv, 2, 1)
    with pytest.raises(ValueError, match="q_weight must have shape"):
        bt.qk_norm_rope(qkv, pos, inv, 2, 1, q_weight=torch.ones(63))
    with pytest.raises(ValueError, match="rows names"):
        bt.qk_norm_rope(qkv, pos, inv, 2, 1, rows=pos)
    q, k = torch.zeros((3, 2, 64)), torch.zeros((3, 1, 64))
    with pytest.raises(TypeError, match="v must be"):
        bt.qk_norm_rope(qkv, pos, inv, 2, 1, out=(q, k, k.half()))
    with pytest.raises(ValueError, match="k must have shape"):
        bt.qk_norm_rope(qkv, pos, inv, 2, 1, out=(q, k[:2], k.clone()))
    with pytest.raises(ValueError, match="overlap itself"):
        bt.qk_norm_rope(qkv, pos, inv, 2, 1, out=(q, k[:1].expand(3, 1, 64), k))
    with pytest.raises(ValueError, match="last dimension"):
        bt.qk_norm_rope(qkv, pos, inv, 2, 1, out=(torch.zeros((3, 64, 2)).transpose(1, 2), k, k.clone()))
    with pytest.raises(TypeError, match="qkv must be one of"):
        bt.qk_norm_rope(qkv.double(), pos, inv, 2, 1)


# bt_attention_shape of a small valid call (with keys enough to need a workspace), and the call
ATT = dict(tokens=6, keys=2000, seqs=2, prefix=0, heads=4, kv_heads=2, head_dim=64, type=BF16, out_type=BF16, causal=1,
           scale=0.125, q_row=256, q_head=64, k_row=128, k_head=64, v_row=128, v_head=64, prefix_k_row=128,
           prefix_k_head=64, prefix_v_row=128, prefix_v_head=64, out_row=256, out_head=64)


def _attention(q=FAKE, k=FAKE, v=FAKE, q_start=FAKE, k_start=FAKE, k_len=FAKE, pk=0, pv=0, out=FAKE, lse=0, ws=FAKE,
               **change):
    shape = struct.pack("7q3if12q", *{**ATT, **change}.values())
    return bt.lib().bt_attention(shape, q, k, v, q_start, k_start, k_len, pk, pv, out, lse, ws, None)


def test_attention_abi_refusals():
    assert bt.lib().bt_attention(None, *[FAKE] * 11, None) == BT_ERR_NULL
    for change in (dict(tokens=-1), dict(tokens=(1 << 23) + 1), dict(keys=-1), dict(keys=2 ** 30 + 1), dict(seqs=-1),
                   dict(prefix=-1), dict(prefix=2 ** 30 + 1), dict(heads=5), dict(heads=0), dict(kv_heads=0), dict(heads=65537, kv_heads=65537),
                   dict(head_dim=60), dict(head_dim=264), dict(head_dim=0), dict(scale=0.0), dict(scale=-1.0),
                   dict(scale=float("nan")), dict(scale=float("inf")), dict(tokens=(1 << 22) + 1, heads=256, kv_heads=1),
                   dict(tokens=1 << 22, seqs=1 << 22, heads=64, kv_heads=64), dict(k_row=(1 << 23) + 8)):
        assert _attention(**change) == BT_ERR_SHAPE, change
    for change in (dict(type=F32), dict(type=3), dict(out_type=2), dict(out_type=7)):
        assert _attention(**change) == BT_ERR_UNSUPPORTED, change
    for name in ("q", "k", "v", "q_start", "k_start", "k_len", "out", "ws"):
        assert _attention(**{name: 0}) == BT_ERR_NULL, name
    assert _attention(prefix=5, pk=FAKE) == BT_ERR_NULL and _attention(prefix=5, pv=FAKE) == BT_ERR_NULL
    for name in ("q", "k", "v"):
        assert _attention(**{name: FAKE + 8}) == BT_ERR_ALIGN, name
    for name in ("q_start", "k_start", "k_len", "lse"):
        assert _attention(**{name: FAKE + 2}) == BT_ERR_ALIGN, name
    assert _attention(out=FAKE + 4) == BT_ERR_ALIGN and _attention(ws=FAKE + 128) == BT_ERR_ALIGN
    for name in ("q_row", "q_head", "k_row", "k_head", "v_row", "v_head"):
        assert _attention(**{name: 132}) == BT_ERR_ALIGN, name
        assert _attention(**{name: -8}) == BT_ERR_ALIGN, name
    assert _attention(out_row=258) == BT_ERR_ALIGN and _attention(out_head=-4) == BT_ERR_ALIGN
    assert _attention(prefix=5, pk=FAKE, pv=FAKE + 8) == BT_ERR_ALIGN
    assert _attention(prefix=5, pk=FAKE, pv=FAKE, prefix_k_row=12) == BT_ERR_ALIGN
    assert _attention(tokens=0) == BT_OK and _attention(seqs=0) == BT_OK


def test_attention_workspace_bytes():
    f = bt.lib().bt_attention_workspace_bytes
    assert f(0, 5, 1, 4, 4, 64, 0) == 0 and f(5, 5, 0, 4, 4, 64, 0) == 0 and f(5, 5, 1, 5, 4, 64, 0) == 0
    assert f(8192, 8192, 1, 32, 32, 128, 0) == 0  # tiles enough: keys are not cut
    assert f(1, 512, 1, 20, 5, 128, 0) == 0 and f(1, 513, 1, 20, 5, 128, 0) > 0  # few keys: one launch
    assert f(2, 1024, 2, 20, 5, 128, 0) == 0 and f(2, 1025, 2, 20, 5, 128, 0) > 0
    for sizes in ((1, 1024, 1, 20, 5, 128, 0), (64, 524288, 64, 20, 5, 128, 0), (64, 0, 64, 64, 8, 128, 16384)):
        n = f(*sizes)
        assert n > 0 and n % 256 == 0 and n < 1 << 28, sizes


def test_attention_refuses(host_ok):  # noqa: F811
    b16 = torch.bfloat16
    q, k, qs, ks = torch.zeros((6, 4, 64), dtype=b16), torch.zeros((9, 2, 64), dtype=b16), torch.zeros(
        3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="q must be one of"):
        bt.attention(q.float(), k, k, qs, ks, ks)
    with pytest.raises(ValueError, match="multiple of 3 key heads"):
        bt.attention(q, torch.zeros((9, 3, 64), dtype=b16), k, qs, ks, ks)
    with pytest.raises(TypeError, match="v must be"):
        bt.attention(q, k, k.half(), qs, ks, ks)
    with pytest.raises(ValueError, match="v must have shape"):
        bt.attention(q, k, k[:8], qs, ks, ks)
    with pytest.raises(ValueError, match="q_start must have shape"):
        bt.attention(q, k, k, ks, ks, ks)
    with pytest.raises(TypeError, match="k_start must be"):
        bt.attention(q, k, k, qs, ks.long(), ks)
    with pytest.raises(ValueError, match="k_len must be"):
        bt.attention(q, k, k, qs, ks, 5)
    with pytest.raises(ValueError, match="come together"):
        bt.attention(q, k, k, qs, ks, ks, prefix_k=k)
    with pytest.raises(ValueError, match="prefix_v must have shape"):
        bt.attention(q, k, k, qs, ks, ks, prefix_k=k, prefix_v=k[:4])
    with pytest.raises(TypeError, match="out must be"):
        bt.attention(q, k, k, qs, ks, ks, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="overlap itself"):
        bt.attention(q, k, k, qs, ks, ks, out=q[:1].expand(6, 4, 64))
    with pytest.raises(ValueError, match="last dimension"):
        bt.attention(q, k.transpose(1, 2).contiguous().transpose(1, 2), k, qs, ks, ks)
    with pytest.raises(ValueError, match="lse must have shape"):
        bt.attention(q, k, k, qs, ks, ks, lse=torch.zeros((4, 6)))
    far = torch.zeros((2000, 2, 64), dtype=b16)  # keys enough to be cut
    with pytest.raises(ValueError, match="workspace holds"):
        bt.attention(q, far, far, qs, ks, ks, workspace=torch.zeros(8, dtype=torch.uint8))
