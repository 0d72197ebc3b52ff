"""Calls of the 4-bit cache, its pages and the int8 products at the ends of what they allow: batches of more sequences
than a wave or a workgroup has lanes for, tables and workspaces that are shared, offsets that leave the arrays, every
tile of the int8 products. Tolerances are the operators' own, given with their tests."""
import math

import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests import cache_ref
from tests.test_cache4_gpu import Case, i32, note
from tests.test_int8_gpu import check as check_int8, codes, padded
from tests.test_pages_gpu import Both

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def lengths(n, most, every, long):
    """k lengths of n sequences: up to `most`, and `long` for each `every`-th."""
    return [long if b % every == every - 1 else (b * 7919 + 3) % (most + 1) for b in range(n)]


@pytest.mark.parametrize("q,k,heads,kv", [
    # single tokens, more than 64, 256 and 1024 sequences
    ([1] * 70, lengths(70, 200, 9, 1300), 8, 2),
    ([1] * 300, lengths(300, 90, 60, 700), 4, 1),
    ([1] * 1100, lengths(1100, 40, 550, 100), 2, 1),
    # most sequences without rows, the keys of the others cut into slices
    ([1 if b % 8 == 3 else 0 for b in range(1100)], lengths(1100, 60, 97, 1500), 4, 1),
    ([1 if b % 3 == 1 else 0 for b in range(260)], lengths(260, 60, 40, 1500), 16, 1),
    # tiles of 64 and of 128 rows
    ([1 if b % 6 == 3 else 0 for b in range(1100)], lengths(1100, 60, 97, 900), 32, 1),
    ([3 if b % 12 == 3 else 0 for b in range(1030)], lengths(1030, 60, 97, 900), 72, 1),
    ([2 if b % 2 else 0 for b in range(130)], lengths(130, 60, 27, 1100), 40, 2),
])
def test_many_sequences(q, k, heads, kv):
    note(f"attention4 {len(q)} sequences of {sum(q)} tokens, {heads}/{kv}")
    c = Case(q, k, heads, kv, 64, "bf16", page=32, seed=len(q), tail=1)
    for wide in (True, False):
        out, lse = c.run(out_dtype=torch.float32 if wide else None)
        c.check(out, lse)
        assert bool((lse[-1] == 77).all())


def test_shared_pages():
    """One page for several sequences and several times in one; a table that repeats its row is refused, not misread."""
    note("attention4 shared pages")
    c = Case([1, 4, 1], [100, 100, 100], 8, 2, 128, "bf16", page=16)
    row = c.table[0]
    row[3], row[5] = row[1], row[0]
    c.table = [row] * 3
    c.check(*c.run(out_dtype=torch.float32))
    one = i32(row)[None]
    with pytest.raises(bt.BTError):
        bt.attention4(c.q, c.cache, one.expand(3, -1), i32(c.k_len), i32(c.q_start))
    with pytest.raises(bt.BTError):
        bt.attention4(c.q, c.cache, i32(row * 3).as_strided((3, len(row)), (len(row) - 1, 1)), i32(c.k_len), i32(c.q_start))


def test_offsets_that_leave_the_arrays():
    note("attention4 offsets outside")
    c = Case([3, 0, 1], [40, 9, 700], 4, 2, 64, "fp16")
    table, k_len = i32(c.table).view(-1, c.W), i32(c.k_len)
    want = bt.attention4(c.q, c.cache, table, k_len, i32([0, 3, 3, 4]))[0]
    got = bt.attention4(c.q, c.cache, table, k_len, i32([-5, 3, 3, 10 ** 9]))[0]
    assert torch.equal(got, want)


def test_sequences_that_overlap():
    """A caller's mistake: more rows than tokens. What the rows hold is open; nothing beside them is touched."""
    note("attention4 sequences that overlap")
    c = Case([30], [900], 64, 8, 64, "bf16", page=32)
    T, B = 30, 200
    table, k_len = i32(c.table * B).view(B, c.W), i32([900] * B)
    room = torch.full((3 * T, 64, 64), 7.0, device=DEV)
    lse = torch.full((3 * T, 64), 7.0, device=DEV)
    need = bt.attention4_workspace_bytes(T, B, 64, 8, 64, c.W, 32)
    ws = torch.full((need + 8192,), 129, dtype=torch.uint8, device=DEV)  # notes of before: negative numbers
    before = c.cache.data.clone()
    for offsets in ([0, T] * (B // 2) + [0], [0, T, 0, 10] * (B // 4) + [T]):
        bt.attention4(c.q, c.cache, table, k_len, i32(offsets), out=room[T: 2 * T], lse=lse[T: 2 * T], workspace=ws[:need])
        torch.cuda.synchronize()
        for x in (room, lse):
            assert bool((x[:T] == 7).all()) and bool((x[2 * T:] == 7).all())
        assert bool((ws[need:] == 129).all()) and torch.equal(c.cache.data, before)
    bt.attention4(c.q, c.cache, table[:1], k_len[:1], i32([0, T]), out=room[T: 2 * T], lse=lse[T: 2 * T])
    c.check(room[T: 2 * T], lse[T: 2 * T])


def test_workspace_of_two_graphs():
    """Two captured calls that share a workspace, replayed one behind the other with other work in it in between."""
    note("attention4 one workspace")
    cases = [Case([1] * 3, [900, 700, 30], 20, 5, 128, "bf16"), Case([70], [900], 8, 2, 64, "bf16", page=32)]
    sizes = [bt.attention4_workspace(c.q, c.cache, i32(c.table).view(-1, c.W)).numel() for c in cases]
    ws = torch.full((max(sizes),), 255, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = []
    for c in cases:
        tensors = (i32(c.table).view(-1, c.W), i32(c.k_len), i32(c.q_start))
        out, lse = torch.empty(c.q.shape, device=DEV), torch.empty(c.q.shape[:2], device=DEV)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            bt.attention4(c.q, c.cache, *tensors, out=out, lse=lse, workspace=ws)
        runs.append((c, out, lse, graph, tensors))
    for turn in range(3):
        with torch.cuda.stream(side):
            for c, _, _, graph, _ in runs:
                c.q.neg_()
                graph.replay()
            ws.random_(0, 256)
        side.synchronize()
        for c, out, lse, _, _ in runs:
            c.check(out, lse)


def test_growth_with_falling_offsets():
    """Offsets that fall are a caller's mistake: places stay inside the pool all the same, and lengths what was granted."""
    note("grow, falling offsets")
    both = Both(4, 6, 40, 16)
    both.grow([20, 3, 16, 0])
    before = both.pages.length.tolist()
    rows, positions, granted = bt.pages_grow(both.pages, i32([0, 9, 4, 60, 20]), both.pool, tokens=64)
    assert all(-1 <= r < 40 * 16 for r in rows.tolist())
    assert [n + m for n, m in zip(before, granted.tolist())] == both.pages.length.tolist()
    table, refs = both.pages.table.tolist(), [0] * 40
    for held, n in zip(table, both.pages.length.tolist()):
        assert [p >= 0 for p in held] == [i < -(-n // 16) for i in range(6)]
        for p in held:
            refs[p] += p >= 0
    assert refs == both.pages.refs.tolist()


@pytest.mark.parametrize("M,N,K", [
    (16, 4096, 200), (16, 4100, 200), (3, 9000, 700),
    (17, 9000, 300), (40, 10000, 520), (64, 16384, 130), (49, 8200, 1100),
    (32, 17000, 300), (33, 16400, 520), (48, 20000, 64), (50, 17003, 130), (64, 24000, 640),
    (17, 2000, 1000), (40, 2560, 900), (64, 2560, 900), (64, 8192, 200), (128, 2560, 300), (200, 2560, 520), (70, 16384, 300),
    (128, 8192, 640), (256, 2560, 700), (256, 4096, 1300), (300, 2560, 300),
    (2048, 5120, 192), (4090, 2500, 100), (520, 20500, 70), (1024, 8192, 130),
])
def test_int8_tiles(M, N, K):
    note(f"int8 tiles {M} x {N} x {K}")
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N + K)
    X, sx = codes(g, M, K)
    W, sw = codes(g, N, K, low=-128)
    w, Xq = bt.pack_int8(W, sw), padded(X, g)
    ref, acc = cache_ref.int8(X, W, sx, sw, None)
    for t in (torch.bfloat16, torch.float32):
        out_acc = torch.full((M, N), 9, dtype=torch.int32, device=DEV)
        y = bt.int8_gemm(w, (Xq, sx), out_dtype=t, out_acc=out_acc)
        assert torch.equal(out_acc.long(), acc)
        check_int8(y, ref, acc, sx, sw, None)
        assert torch.equal(bt.int8_gemm(w, (Xq, sx), out_dtype=t), y)


def test_int8_without_k_for_many_outputs():
    note("int8 no k, many outputs")
    M, N = 1500, 1111
    w = bt.pack_int8(torch.zeros((N, 0), dtype=torch.int8, device=DEV), torch.ones(N, device=DEV))
    bias = torch.randn(N, device=DEV)
    y = torch.full((M, N), math.nan, device=DEV)
    bt.int8_gemm(w, (torch.zeros((M, 0), dtype=torch.int8, device=DEV), torch.ones(M, device=DEV)), bias=bias, out=y)
    assert torch.equal(y, bias.expand(M, N))


def test_int8_rows_at_odd_places():
    """Weights' codes whose rows start at any byte (a view of a larger array would be copied; one at an odd address is not)."""
    note("int8 pack from odd addresses")
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    for N, K in ((5, 33), (20, 64), (17, 131)):
        room = torch.randint(-128, 128, (N * K + 3,), generator=g, device=DEV, dtype=torch.int8)
        W = room[3:].view(N, K)
        a, b = bt.pack_int8(W, torch.ones(N, device=DEV)), bt.pack_int8(W.clone(), torch.ones(N, device=DEV))
        n = bt.int8_weight_bytes(N, K)
        assert torch.equal(a.data[:n], b.data[:n])
