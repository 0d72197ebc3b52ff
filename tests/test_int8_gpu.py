"""bt_int8_gemm: acc equal to the exact products, Y against the formula in 64 bits.

Tolerance of Y: fp32(acc) 2^-24, the product of the scales 2^-24, their product with acc 2^-24 (together below 3.1 *
2^-24 of |acc * scales|), the bias 2^-24 of the sum, one rounding to Y's type: eps / 2 (below its smallest normal
number: half its smallest step)."""
import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests import cache_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def note(msg):
    print(f"[gpu-case] {msg}", flush=True)


def codes(g, rows, K, low=-127):
    x = torch.randint(low, 128, (rows, K), generator=g, device=DEV, dtype=torch.int8)
    scale = torch.exp(torch.randn(rows, generator=g, device=DEV)) / 5000
    return x, scale


def padded(x, g):
    """Rows of bt_act_row_bytes(K); what lies past K may be anything."""
    M, K = x.shape
    out = torch.randint(-128, 128, (M, bt.act_row_bytes(K)), generator=g, device=DEV, dtype=torch.int8)
    out[:, :K] = x
    return out


def check(y, ref, acc, sx, sw, bias):
    t = y.dtype
    size = (acc.double() * (sx.double()[:, None] * sw.double())).abs()
    eps = torch.finfo(t).eps / 2
    tol = 3.1 * 2.0 ** -24 * size * (1 + eps) + (0 if bias is None else 2.0 ** -24 * ref.abs() * 1.01)
    tol = tol + eps * ref.abs() * (1 + 2.0 ** -20) + torch.finfo(t).smallest_normal * eps
    if t == torch.float16:  # beyond its largest number: infinity
        big = ref.abs() + tol >= 65504
        assert bool((y[big].isinf() | (y[big].abs() >= 65000)).all())
        y, ref, tol = y[~big], ref[~big], tol[~big]
    d = (y.double() - ref).abs()
    assert bool((d <= tol).all()), float((d / tol).max())


SHAPES = [(1, 1, 1), (1, 16, 64), (1, 32000, 2560), (2, 100, 300), (3, 2560, 6912), (4, 33, 70), (7, 4096, 4096), (8, 513, 1000),
          (15, 48, 64), (16, 640, 2560), (17, 1000, 129), (31, 777, 512), (32, 256, 8192), (33, 64, 64), (37, 2200, 4096),
          (48, 300, 700), (64, 4096, 1024), (65, 129, 257), (100, 2560, 2560), (127, 65, 4095), (128, 1024, 4096),
          (200, 6912, 2560), (255, 257, 640), (256, 256, 64), (300, 3000, 1100), (513, 515, 1025), (1000, 1111, 333),
          (1024, 2560, 2560), (2048, 4096, 512), (4096, 200, 300), (2, 5, 131072), (40, 20, 131072), (300, 260, 131072)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_int8_gemm(M, N, K):
    note(f"int8 {M} x {N} x {K}")
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N + K)
    X, sx = codes(g, M, K)
    W, sw = codes(g, N, K, low=-128)
    w = bt.pack_int8(W, sw)
    Xq = padded(X, g)
    ref, acc = cache_ref.int8(X, W, sx, sw, None)
    bias = torch.randn(N, generator=g, device=DEV)
    for t in TYPES:
        out_acc = torch.full((M, N), 9, dtype=torch.int32, device=DEV)
        y = bt.int8_gemm(w, (Xq, sx), out_dtype=t, out_acc=out_acc)
        assert torch.equal(out_acc.long(), acc)
        check(y, ref, acc, sx, sw, None)
        yb = bt.int8_gemm(w, (Xq, sx), bias=bias, out_dtype=t)
        check(yb, ref + bias.double(), acc, sx, sw, bias)


def test_packed_layout():
    """Byte for byte as the header says."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    for N, K in ((1, 1), (17, 65), (48, 128), (33, 1000)):
        W, sw = codes(g, N, K, low=-128)
        full = torch.zeros(-(-N // 16) * 16, -(-K // 64) * 64, dtype=torch.int8)
        full[:N, :K] = W.cpu()
        want = full.view(full.shape[0] // 16, 16, full.shape[1] // 64, 4, 16).permute(0, 2, 3, 1, 4).contiguous()
        data = bt.pack_int8(W, sw).data.cpu()
        assert torch.equal(data.view(torch.int8)[: want.numel()], want.flatten())


def test_extreme_codes():
    """The largest sums: K = 131072 with one side in +-127 and the other down to -128."""
    note("int8 extreme codes")
    K = 131072
    for M, N in ((1, 20), (20, 40), (260, 130)):
        X = torch.full((M, K), 127, dtype=torch.int8, device=DEV)
        X[1::2] = -127
        W = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
        W[::3] = 127
        sx, sw = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
        acc = torch.empty((M, N), dtype=torch.int32, device=DEV)
        y = bt.int8_gemm(bt.pack_int8(W, sw), (X, sx), out_acc=acc)
        ref, want = cache_ref.int8(X[:2], W, sx[:2], sw, None)
        want = want[torch.arange(M, device=DEV) % 2]
        assert torch.equal(acc.long(), want)
        assert bool(((y.double() - want).abs() <= 2.0 ** -24 * want.abs()).all())


def test_nothing_to_do_and_no_k():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    bias = torch.randn(5, device=DEV)
    w = bt.pack_int8(torch.zeros((5, 0), dtype=torch.int8, device=DEV), torch.ones(5, device=DEV))
    y = bt.int8_gemm(w, (torch.zeros((3, 0), dtype=torch.int8, device=DEV), torch.ones(3, device=DEV)), bias=bias)
    assert torch.equal(y, bias.expand(3, 5))
    W, sw = codes(g, 0, 64)
    assert bt.int8_gemm(bt.pack_int8(W, sw), (torch.zeros((3, 256), dtype=torch.int8, device=DEV), torch.ones(3, device=DEV))).shape == (3, 0)
    W, sw = codes(g, 7, 64)
    assert bt.int8_gemm(bt.pack_int8(W, sw), (torch.zeros((0, 256), dtype=torch.int8, device=DEV), torch.ones(0, device=DEV))).shape == (0, 7)


def test_from_weights_and_tokens():
    """fp32 weights and tokens: both sides quantized by bt_quant_act's rule, the product exact on its codes."""
    note("int8 linear")
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    for M, N, K in ((1, 500, 300), (40, 130, 2560), (150, 300, 1000)):
        X = torch.randn(M, K, generator=g, device=DEV)
        W = torch.randn(N, K, generator=g, device=DEV)
        w = bt.pack_weights_int8(W)
        xq, sx, _ = bt.quant_act(X)
        wq, sw, _ = bt.quant_act(W)
        assert torch.equal(w.scale, sw)
        ref, acc = cache_ref.int8(xq[:, :K], wq[:, :K], sx, sw, None)
        check(bt.int8_linear(X, w), ref, acc, sx, sw, None)
        check(bt.int8_linear(X, w, out_dtype=torch.bfloat16), ref, acc, sx, sw, None)
        # and near the unquantized product: half a step a side, steps of max / 127
        dense = X.double() @ W.double().t()
        bound = (X.abs().sum(1)[:, None] * sw + W.abs().sum(1) * sx[:, None]) / 2 + K * sx[:, None] * sw / 4
        assert bool(((bt.int8_linear(X, w).double() - dense).abs() <= bound.double() * 1.001).all())


def test_unaligned_outputs():
    """Outputs aligned to their element only."""
    note("int8 unaligned outputs")
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    for M, N, K in ((3, 70, 100), (40, 96, 256), (300, 512, 128)):
        X, sx = codes(g, M, K)
        W, sw = codes(g, N, K)
        w, Xq = bt.pack_int8(W, sw), padded(X, g)
        ref, acc = cache_ref.int8(X, W, sx, sw, None)
        for t in TYPES:
            room = torch.full((M * N + 2,), 3.0, dtype=t, device=DEV)
            racc = torch.full((M * N + 2,), 3, dtype=torch.int32, device=DEV)
            y = bt.int8_gemm(w, (Xq, sx), out=room[1:-1].view(M, N), out_acc=racc[1:-1].view(M, N))
            check(y, ref, acc, sx, sw, None)
            assert torch.equal(racc[1:-1].view(M, N).long(), acc)
            assert float(room[0]) == 3 and float(room[-1]) == 3 and int(racc[0]) == 3 and int(racc[-1]) == 3


def test_replays():
    note("int8 replays")
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    for M, N, K in ((1, 2560, 2560), (24, 4096, 1024), (300, 1024, 2560)):
        X, sx = codes(g, M, K)
        W, sw = codes(g, N, K)
        w, Xq = bt.pack_int8(W, sw), padded(X, g)
        ws = bt.int8_workspace(M, w)
        out, acc = torch.empty((M, N), device=DEV), torch.empty((M, N), dtype=torch.int32, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            bt.int8_gemm(w, (Xq, sx), out=out, out_acc=acc, workspace=ws)
            side.synchronize()
            with torch.cuda.graph(graph, stream=side):
                bt.int8_gemm(w, (Xq, sx), out=out, out_acc=acc, workspace=ws)
        torch.cuda.synchronize()
        for _ in range(3):
            X2, s2 = codes(g, M, K)
            Xq[:, :K] = X2
            sx.copy_(s2)
            graph.replay()
            ref, want = cache_ref.int8(X2, W, sx, sw, None)
            assert torch.equal(acc.long(), want)
            check(out, ref, want, sx, sw, None)
