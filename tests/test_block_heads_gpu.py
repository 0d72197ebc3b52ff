"""bt_qk_norm_rope against its definition in 64 bits.

Tolerance: one rounding to the output type (half a step, eps / 2 of the value; half the smallest
subnormal 2^-25 in fp16) and the fp32 arithmetic before it. That is, relative to the magnitude (the
head's value, or the sum of the pair's absolute values where it is rotated): the mean of squares and
its root (a sum of at most 512 squares in a tree of depth 12, halved by the root: 6 * 2^-24, plus 3
for division, root and eps), two products (2 * 2^-24), the rotation's products and sum (2 * 2^-24),
the sine and cosine (4 * 2^-24) and the turn's fraction rounded to fp32 (2^-26 of a turn, 2^-23.3
radians): below 20 * 2^-24. Positions stay under 2^31, where the fp64 angle is good to 2^-21 radians
(2^31 * 2^-52): 2^-20 covers both.
"""
import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests import block_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def note(msg):
    print(f"[gpu-case] {msg}", flush=True)


def close(y, ref, mag):
    half = torch.finfo(y.dtype).eps / 2
    tiny = 2.0 ** -25 if y.dtype == torch.float16 else 1e-38
    tol = half * (ref.abs() + 2.0 ** -19 * mag) + 2.0 ** -19 * mag + tiny
    d = (y.double() - ref).abs()
    assert bool((d <= tol).all()), float((d / tol).max())


def inputs(M, heads, kv, D, rot, in_kind, norm, max_pos, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    qkv = rnd(M, (heads + 2 * kv) * D).to(TYPES[in_kind])
    pos = torch.randint(0, max_pos, (M,), generator=g, device=DEV, dtype=torch.int32)
    inv = bt.rope_frequencies(rot, 10000.0, DEV) if rot else None
    return qkv, pos, inv, (1 + 0.2 * rnd(D) if norm else None), (1 - 0.2 * rnd(D) if norm else None)


def reference(qkv, pos, inv, qw, kw, heads, kv, D, interleaved, eps=1e-6):
    x = qkv.double().view(qkv.shape[0], heads + 2 * kv, D)
    rot = 0 if inv is None else 2 * inv.shape[0]
    angle = pos.double()[:, None] * inv if rot else None
    return (block_ref.norm_rope(x[:, :heads], qw, eps, angle, rot, interleaved),
            block_ref.norm_rope(x[:, heads: heads + kv], kw, eps, angle, rot, interleaved),
            (x[:, heads + kv:], x[:, heads + kv:].abs()))


CASES = [
    # M, heads, kv, D, rot, interleaved, norm, in, out, positions below
    (1, 20, 5, 128, 128, False, True, "fp32", "bf16", 4096),
    (1, 1, 1, 8, 8, False, True, "fp32", "fp32", 9),
    (2, 3, 1, 16, 8, True, True, "fp32", "fp32", 2 ** 31 - 1),
    (5, 8, 1, 256, 256, True, True, "fp32", "bf16", 100),
    (7, 6, 3, 80, 40, False, True, "bf16", "bf16", 131072),
    (9, 2, 2, 512, 128, False, True, "fp16", "fp32", 5000),
    (3, 4, 2, 504, 504, True, False, "fp32", "fp16", 5000),
    (37, 32, 32, 128, 64, True, True, "fp32", "fp16", 1000000),
    (65, 12, 4, 96, 96, False, False, "fp32", "bf16", 77),
    (33, 16, 2, 64, 0, False, True, "fp16", "fp16", 1),
    (40, 5, 5, 24, 24, False, True, "fp32", "fp32", 2 ** 31 - 1),
    (3, 3, 3, 200, 24, False, True, "fp32", "fp16", 100000),  # nine heads, two to a wave
    (5, 1, 1, 48, 48, True, True, "bf16", "fp32", 4096),  # three heads, eight to a wave
    (700, 20, 5, 128, 128, False, True, "fp32", "bf16", 8192),
    (2050, 7, 7, 72, 56, True, True, "fp32", "fp32", 8192),
]


@pytest.mark.parametrize("M,heads,kv,D,rot,inter,norm,in_kind,out_kind,max_pos", CASES)
def test_matches_definition(M, heads, kv, D, rot, inter, norm, in_kind, out_kind, max_pos):
    note(f"qk_norm_rope M={M} heads={heads}/{kv} D={D} rot={rot} inter={inter} norm={norm} {in_kind}->{out_kind}")
    qkv, pos, inv, qw, kw = inputs(M, heads, kv, D, rot, in_kind, norm, max_pos, M + D)
    got = bt.qk_norm_rope(qkv, pos, inv, heads, kv, qw, kw, interleaved=inter, dtype=TYPES[out_kind])
    for y, (ref, mag) in zip(got, reference(qkv, pos, inv, qw, kw, heads, kv, D, inter)):
        assert y.dtype == TYPES[out_kind]
        close(y, ref, mag)


def test_only_one_norm_and_negative_positions():
    note("qk_norm_rope one norm")
    qkv, pos, inv, qw, _ = inputs(6, 4, 2, 64, 64, "fp32", True, 3000, 3)
    pos = -pos
    got = bt.qk_norm_rope(qkv, pos, inv, 4, 2, q_weight=qw, dtype=torch.float32)
    for y, (ref, mag) in zip(got, reference(qkv, pos, inv, qw, None, 4, 2, 64, False)):
        close(y, ref, mag)


def test_zero_and_tiny_heads():
    """A zero head stays zero, a tiny one is held up by eps."""
    note("qk_norm_rope zero heads")
    qkv, pos, inv, qw, kw = inputs(3, 2, 1, 64, 64, "fp32", True, 50, 4)
    qkv[0] = 0
    qkv[1] *= 1e-12
    got = bt.qk_norm_rope(qkv, pos, inv, 2, 1, qw, kw, dtype=torch.float32)
    for y, (ref, mag) in zip(got, reference(qkv, pos, inv, qw, kw, 2, 1, 64, False)):
        close(y, ref, mag)
    assert bool((got[0][0] == 0).all())


@pytest.mark.parametrize("layout", ["rows", "heads first"])
def test_cache_rows_strides_and_padding_tokens(layout):
    note(f"qk_norm_rope cache {layout}")
    M, heads, kv, D, cap = 21, 6, 3, 80, 50
    qkv, pos, inv, qw, kw = inputs(M, heads, kv, D, 80, "fp32", True, 900, 5)
    wide = torch.zeros((M, qkv.shape[1] + 12), device=DEV)
    wide[:, 4: 4 + qkv.shape[1]] = qkv
    strided = wide[:, 4: 4 + qkv.shape[1]]
    rows = torch.randperm(cap, device=DEV)[:M].to(torch.int32)
    rows[3], rows[10], rows[20] = -1, cap, 2 ** 31 - 1
    if layout == "rows":
        kc = torch.full((cap, 2, kv, D), 7.0, dtype=torch.float16, device=DEV)
        k, v = kc[:, 0], kc[:, 1]
        q = torch.empty((M, heads, D), dtype=torch.float16, device=DEV)
    else:
        kc = torch.full((2, kv, cap, D), 7.0, dtype=torch.float16, device=DEV)
        k, v = kc[0].transpose(0, 1), kc[1].transpose(0, 1)
        q = torch.empty((heads, M, D), dtype=torch.float16, device=DEV).transpose(0, 1)
    got = bt.qk_norm_rope(strided, pos, inv, heads, kv, qw, kw, rows=rows, out=(q, k, v))
    assert got[0] is q
    (rq, mq), (rk, mk), (rv, mv) = reference(qkv, pos, inv, qw, kw, heads, kv, D, False)
    close(q, rq, mq)
    good = (rows >= 0) & (rows < cap)
    at = rows[good].long()
    close(k[at], rk[good], mk[good])
    close(v[at], rv[good], mv[good])
    left = torch.ones(cap, dtype=torch.bool, device=DEV)
    left[at] = False
    assert bool((k[left] == 7).all()) and bool((v[left] == 7).all())


def test_graph_replay():
    note("qk_norm_rope graph")
    M, heads, kv, D = 19, 8, 2, 128
    qkv, pos, inv, qw, kw = inputs(M, heads, kv, D, D, "fp32", True, 900, 6)
    out = tuple(torch.empty((M, h, D), dtype=torch.bfloat16, device=DEV) for h in (heads, kv, kv))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        bt.qk_norm_rope(qkv, pos, inv, heads, kv, qw, kw, out=out)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        bt.qk_norm_rope(qkv, pos, inv, heads, kv, qw, kw, out=out)
    for rep in range(3):
        qkv.normal_()
        pos.add_(1)
        eager = bt.qk_norm_rope(qkv, pos, inv, heads, kv, qw, kw)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), rep


def test_no_tokens():
    note("qk_norm_rope empty")
    qkv, pos, inv, qw, kw = inputs(0, 2, 1, 64, 64, "fp32", True, 50, 4)
    q, k, v = bt.qk_norm_rope(qkv, pos, inv, 2, 1, qw, kw)
    assert q.shape == (0, 2, 64) and k.shape == v.shape == (0, 1, 64)
