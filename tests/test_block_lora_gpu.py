"""bt_lora_apply against its definition in 64 bits.

Tolerance: operands are multiplied exactly (fp32 weights to 2^-30), so only fp32 sums round. A sum
of n terms in any order is within n * 2^-24 of the sum of their absolute values, and an inner product
nested in another adds their counts: (K + R + slices + 8) * 2^-24 * magnitude bounds it. The matrix
cores add the terms of an instruction without rounding each, and the partial sums are trees, so a
quarter of that count is asked for, at least 16.
"""
import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests import block_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def note(msg):
    print(f"[gpu-case] {msg}", flush=True)


def make(M, K, groups, R, L, dtype, seed, ranks=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    N = sum(groups)
    A = (rnd(L, len(groups) * R, K) / max(K, 1) ** 0.5).to(dtype)
    B = (rnd(L, N, R) / R ** 0.5).to(dtype)
    scale = torch.rand(L, generator=g, device=DEV) + 0.5
    index = torch.randint(-1, L + 1, (M,), generator=g, device=DEV, dtype=torch.int32)
    rk = torch.randint(0, R + 1, (L,), generator=g, device=DEV, dtype=torch.int32) if ranks else None
    return rnd(M, K), A, B, scale, index, rnd(M, N), rk


def close(y, ref, mag, K, R):
    tol = max(16, (K + R + 40) / 4) * 2.0 ** -24 * mag + 1e-37
    bad = (y.double() - ref).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), float(((y.double() - ref).abs() / tol).max()))


CASES = [
    # M, K, groups, R, L, type, ranks
    (1, 2560, (2560, 640, 640), 16, 4, "bf16", False),
    (1, 64, (64,), 8, 1, "fp16", False),
    (3, 1, (1,), 1, 2, "fp32", False),
    (7, 7, (5,), 3, 2, "bf16", True),
    (16, 130, (33, 67), 5, 3, "bf16", False),
    (17, 129, (1, 62, 200), 12, 5, "fp16", True),
    (33, 2564, (300,), 40, 33, "bf16", True),
    (64, 1100, (255, 258), 64, 48, "fp16", True),
    (128, 512, (640,), 16, 200, "bf16", False),
    (129, 513, (100, 3), 20, 2, "fp32", True),
    (300, 2560, (64, 64, 64, 64, 64, 64, 64, 64), 16, 3, "bf16", False),
    (515, 1024, (700, 324), 32, 9, "fp16", False),
    (200, 300, (130,), 256, 2, "bf16", True),
    (2048, 640, (1000,), 32, 8, "fp32", False),
    (300, 264, (500,), 24, 60, "bf16", True),  # many tokens, few of each adapter
    (1024, 96, (70,), 8, 200, "fp16", False),
    (1025, 96, (70,), 8, 200, "fp16", False),
    (513, 264, (500,), 24, 40, "bf16", True),
    (512, 264, (500,), 24, 3, "fp16", True),
    (5, 0, (20,), 4, 2, "bf16", False),
    (4, 28672, (512,), 16, 2, "bf16", False),
]
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.mark.parametrize("M,K,groups,R,L,kind,ranks", CASES)
def test_lora_matches_definition(M, K, groups, R, L, kind, ranks):
    note(f"lora M={M} K={K} groups={groups} R={R} L={L} {kind} ranks={ranks}")
    X, A, B, scale, index, base, rk = make(M, K, groups, R, L, TYPES[kind], 11 + M + K, ranks)
    ad = bt.LoraAdapters(A, B, scale, ranks=rk, group_rows=groups if len(groups) > 1 else None)
    ws = torch.full((max(bt.lora_workspace_bytes(M, ad), 256),), 255, dtype=torch.uint8, device=DEV)  # NaNs
    ref, mag = block_ref.lora(X, A, B, scale, index, base, rk, groups)
    y = bt.lora_apply(X, ad, index, base=base, workspace=ws)
    close(y, ref, mag, K, R)
    none = (index < 0) | (index >= L)
    assert torch.equal(y[none], base[none])  # no adapter: the base's row, bit for bit
    inplace = base.clone()
    assert bt.lora_apply(X, ad, index, base=inplace, out=inplace) is inplace
    assert torch.equal(inplace, y)
    z = bt.lora_apply(X, ad, index)
    refz, magz = block_ref.lora(X, A, B, scale, index, None, rk, groups)
    close(z, refz, magz, K, R)
    assert bool((z[none] == 0).all())


@pytest.mark.parametrize("M", [100, 400, 600])
def test_runs_and_mixed_orders_agree(M):
    """Tokens in mixed order and sorted by adapter, on both sides of the dispatch bound (128 tokens); with
    many tokens a token's result does not depend on its neighbours or its place at all."""
    note(f"lora orders M={M}")
    K, R, L = 512, 16, 6
    X, A, B, scale, index, base, _ = make(M, K, (320,), R, L, torch.bfloat16, 5)
    ad = bt.LoraAdapters(A, B, scale)
    ref, mag = block_ref.lora(X, A, B, scale, index, base)
    y = bt.lora_apply(X, ad, index, base=base)
    close(y, ref, mag, K, R)
    order = torch.argsort(index, stable=True)
    ys = bt.lora_apply(X[order].contiguous(), ad, index[order].contiguous(), base=base[order].contiguous())
    close(ys, ref[order], mag[order], K, R)
    if M > 128:
        assert torch.equal(ys, y[order])


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_tiles_with_every_share_of_an_adapter(kind):
    """Tiles in which an adapter has 1, 2, 4, 5, 11 and 16 tokens, with odd sizes and ranks in use."""
    note(f"lora shares {kind}")
    share = [1, 2, 4, 5, 4] + [11, 5] + [16] + [16 - 3, 3]
    M, K, groups, R, L = sum(share), 131, (30, 71), 20, len(share)
    X, A, B, scale, _, base, rk = make(M, K, groups, R, L, TYPES[kind], 15, True)
    index = torch.repeat_interleave(torch.arange(L, device=DEV), torch.tensor(share, device=DEV)).to(torch.int32)
    index[7] = -1
    ref, mag = block_ref.lora(X, A, B, scale, index, base, rk, groups)
    y = bt.lora_apply(X, bt.LoraAdapters(A, B, scale, ranks=rk, group_rows=groups), index, base=base)
    close(y, ref, mag, K, R)
    assert torch.equal(y[7], base[7])


@pytest.mark.parametrize("M,run", [(40, 1), (40, 6), (600, 5)])
def test_other_adapters_and_unused_ranks_never_leak(M, run):
    note(f"lora leaks M={M} run={run}")
    K, R, L = 200, 12, 4
    X, A, B, scale, _, base, _ = make(M, K, (70, 30), R, L, torch.float16, 6)
    index = (torch.arange(M, device=DEV) // run % L).to(torch.int32)
    ranks = torch.tensor([12, 5, 12, 0], dtype=torch.int32, device=DEV)
    ref, mag = block_ref.lora(X, A, B, scale, index, base, ranks, (70, 30))
    A2, B2 = A.clone(), B.clone()
    for a, r in ((1, 5), (3, 0)):
        for g in range(2):
            A2[a, g * R + r: (g + 1) * R] = float("nan")
        B2[a, :, r:] = float("inf")
    A2[2], B2[2] = float("nan"), float("inf")
    y = bt.lora_apply(X, bt.LoraAdapters(A2, B2, scale, ranks=ranks, group_rows=(70, 30)), index, base=base)
    fine = index != 2
    close(y[fine], ref[fine], mag[fine], K, R)
    assert bool(y[~fine].isnan().all())


def test_extreme_magnitudes():
    """fp32 values near the ends of the range, and weights of every size, keep fp32 accuracy."""
    note("lora magnitudes")
    M, K, R = 5, 96, 8
    X, A, B, scale, index, _, _ = make(M, K, (64,), R, 1, torch.float32, 8)
    index.zero_()
    X *= torch.tensor([1e30, 1e-25, 3.0e38 / 4, 1.0, 1e-30], device=DEV)[:, None] / X.abs().max()
    A *= 1e-3
    ref, mag = block_ref.lora(X, A, B, scale, index)
    close(bt.lora_apply(X, bt.LoraAdapters(A, B, scale), index), ref, mag, K, R)


def test_unaligned_views():
    note("lora unaligned")
    M, K, N, R = 9, 64, 48, 8
    X, A, B, scale, index, base, _ = make(M, K, (N,), R, 3, torch.bfloat16, 9)

    def shifted(t, by):
        flat = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
        v = flat[by:].view(t.shape)
        v.copy_(t)
        return v

    ref = bt.lora_apply(X, bt.LoraAdapters(A, B, scale), index, base=base)
    ad = bt.LoraAdapters(shifted(A, 1), shifted(B, 3), shifted(scale, 1))
    out = bt.lora_apply(shifted(X, 1), ad, shifted(index, 1), base=shifted(base, 2), out=shifted(base, 3))
    assert torch.equal(out, ref)


def test_empty_calls_and_no_adapters():
    note("lora empty")
    X, A, B, scale, index, base, _ = make(6, 32, (16,), 4, 2, torch.bfloat16, 10)
    ad = bt.LoraAdapters(A, B, scale)
    assert bt.lora_apply(X[:0], ad, index[:0]).shape == (0, 16)
    none = bt.LoraAdapters(A[:0], B[:0], scale[:0])
    assert torch.equal(bt.lora_apply(X, none, index, base=base), base)


@pytest.mark.parametrize("M", [2, 40, 300])
def test_linear_with_adapters(M):
    """The projection's own path: linear(..., adapters=) is the packed product plus the adapters'."""
    note(f"linear with adapters M={M}")
    K, groups, R, L = 512, (256, 64, 64), 16, 5
    X, A, B, scale, index, _, _ = make(M, K, groups, R, L, torch.bfloat16, 20 + M)
    pw = bt.pack_weights(torch.randn((sum(groups), K), device=DEV) * 0.02)
    ad = bt.LoraAdapters(A, B, scale, group_rows=groups)
    Y0, acc0 = bt.linear(X, pw, want_acc=True)
    Y, acc = bt.linear(X, pw, want_acc=True, adapters=ad, adapter_index=index)
    assert torch.equal(acc, acc0)
    ref, mag = block_ref.lora(X, A, B, scale, index, Y0, None, groups)
    close(Y, ref, mag, K, R)
    out = torch.empty_like(Y)
    assert bt.linear(X, pw, out_y=out, adapters=ad, adapter_index=index)[0] is out
    assert torch.equal(out, Y)


@pytest.mark.parametrize("M", [3, 200])
def test_graph_replays_and_streams(M):
    note(f"lora graph M={M}")
    K, groups, R, L = 640, (128, 72), 16, 5
    X, A, B, scale, index, base, _ = make(M, K, groups, R, L, torch.bfloat16, 30 + M)
    ad = bt.LoraAdapters(A, B, scale, group_rows=groups)
    ws, out = bt.lora_workspace(M, ad), torch.empty_like(base)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        bt.lora_apply(X, ad, index, base=base, out=out, workspace=ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        bt.lora_apply(X, ad, index, base=base, out=out, workspace=ws)
    for rep in range(3):
        X.normal_()
        index.copy_(torch.randint(-1, L, (M,), device=DEV, dtype=torch.int32))
        eager = bt.lora_apply(X, ad, index, base=base, workspace=ws)
        torch.cuda.synchronize()
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), rep
