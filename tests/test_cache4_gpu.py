"""The 4-bit cache: the write bit for bit against its rule, the read-back, and bt_attention4 against its definition
in 64 bits on the cache's own values.

Tolerance of the attention. Keys and values are exact (a code with its scale is a bf16), and so are the queries.
 - Probabilities are carried in two bf16 parts, each the nearest: a bf16 has 8 significant bits, so the rest is at most
   half a step, 2^-8 of a value in [1, 2) and so of any value, and 2^-16 is left after two parts; after three, for
   fp32 outputs, 2^-24; after one, for bf16 outputs of more than 16 rows of a sequence and key head, 2^-8.
   Parts below bf16's smallest are below 2^-126 of the largest.
 - Scores: fp32 sums of products of bf16 (two parts of an fp16 query: exact, twice the terms), off by at most
   2 * (D / 8 + 2) * 2^-24 * scale * sum |q k| (instructions add 16 products or more at once), and the roundings of the
   FMA with the reference. A score error e changes p_j by a factor within e, the output by at most 2 e * sum p_j |v_j|.
 - v_exp_f32 and the reciprocal: 2 * 2^-23. fp32 sums over n keys: n / 16 * 2^-24.
 - One rounding to the output type: eps / 2 of the value (fp16 outputs below 2^-14: 2^-25).
lse: the score error, the sum's n / 16 * 2^-24, and three roundings of the value itself.
"""
import math

import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests import block_ref, cache_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def note(msg):
    print(f"[gpu-case] {msg}", flush=True)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def random_data(g, *shape):
    return torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)


# ------------------------------------------------------------------ write and read


def check_write(pages, page, kv, D, rows, k, v):
    """Writes k, v to a cache of random bytes; every byte is as the rule has it."""
    g = torch.Generator(device=DEV)
    g.manual_seed(len(rows))
    size = bt.cache4_page_bytes(page, kv, D)
    cache = bt.Cache4(pages, page, kv, D, layers=2, data=random_data(g, 2, pages, size))
    want = cache.data.cpu().clone()
    flat = want[1].view(-1)
    for m, row in enumerate(rows):
        if 0 <= row < pages * page:
            cache_ref.put(flat, row, page, k[m].cpu(), v[m].cpu())
    bt.cache4_write(cache, k, v, i32(rows), layer=1)
    assert torch.equal(cache.data.cpu(), want)
    return cache


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("page,kv,D", [(16, 1, 8), (32, 3, 40), (16, 5, 128), (64, 2, 64), (128, 1, 80), (1024, 2, 256)])
def test_write_is_the_rule(kind, page, kv, D):
    note(f"write {kind} page {page} kv {kv} D {D}")
    g = torch.Generator(device=DEV)
    g.manual_seed(D)
    pages = 3
    n = 37
    rows = torch.randperm(pages * page, generator=torch.Generator().manual_seed(1))[:n].tolist()
    rows[3], rows[10 % len(rows)] = -1, pages * page  # outside: not written
    rows = rows + [-(2 ** 31), 2 ** 31 - 1]
    k, v = ((torch.randn(len(rows), kv, D, generator=g, device=DEV)
             * torch.exp2(torch.randint(-20, 12, (len(rows), kv, 1), generator=g, device=DEV).float())).to(TYPES[kind])
            for _ in range(2))
    check_write(pages, page, kv, D, rows, k, v)


def test_write_edges():
    """Ties, the scale's borders, zeros of both signs, subnormals, the largest values, infinities and NaNs."""
    tiny, big = 2.0 ** -149, torch.finfo(torch.float32).max
    groups = []
    for top in (7.0, 7.0000005, 6.9999995, 3.5, 1.75, 1.7500001, 1.9999999, 1.0, 6.0, 5.0):
        ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.25000003, 0.24999999, 0.7500001, 0.74999994, 5.0000005, 4.9999995]
        line = [top] + [t * (1 if top >= 4 else top / 7) for t in ties]
        groups.append(line + [-x for x in line] + [0.0, -0.0, 1e-30, -1e-30])
    groups += [[0.0] * 32, [-0.0] * 32, [tiny * (i - 16) for i in range(32)], [2.0 ** -126 * (i - 16) / 4 for i in range(32)],
               [2.0 ** -124 * (i - 16) / 9 for i in range(32)], [big * (i - 16) / 16 for i in range(32)],
               [2.0 ** 127 * (1.75 if i % 2 else 1.0) / (1 + i // 4) for i in range(32)],
               [math.inf] + [1.0] * 31, [1.0] * 31 + [-math.inf], [math.nan] + [2.0] * 31, [math.nan] * 32]
    x = torch.tensor(groups, dtype=torch.float32, device=DEV)
    x = torch.nn.functional.pad(x, (0, 32 - x.shape[1])) if x.shape[1] < 32 else x
    n = x.shape[0]
    note(f"write edges, {n} groups")
    for kind in ("fp32", "bf16"):
        y = x.to(TYPES[kind])[:, None]
        check_write(2, 16, 1, 32, list(range(n)), y, y.flip(0))


def test_write_strided():
    """Keys and values as views of one row of a projection, in heads that are apart."""
    note("write strided")
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    qkv = torch.randn(9, 4 + 3 + 3, 72, generator=g, device=DEV).bfloat16()
    k, v = qkv[:, 4:7, :64], qkv[:, 7:, 8:72].transpose(0, 1).contiguous().transpose(0, 1)
    check_write(2, 16, 3, 64, [30, 2, 7, 9, 31, 0, 16, 15, 4], k, v)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp16"])
@pytest.mark.parametrize("page,kv,D", [(16, 2, 128), (64, 3, 72), (32, 1, 256), (16, 2, 8)])
def test_read_back(kind, page, kv, D):
    """Any bytes: codes times scales, NaN above the largest scale, zeros for places outside."""
    note(f"read {kind} page {page} kv {kv} D {D}")
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    pages = 5
    cache = bt.Cache4(pages, page, kv, D, data=random_data(g, 1, pages, bt.cache4_page_bytes(page, kv, D)))
    rows = [0, pages * page - 1, -1, pages * page, 17, 17] + list(range(pages * page))
    k = torch.full((len(rows), kv + 1, D + 8), 7.0, dtype=TYPES[kind], device=DEV)
    v = torch.full((kv, len(rows), D), 7.0, dtype=TYPES[kind], device=DEV)
    bt.cache4_read(cache, i32(rows), out=(k[:, :kv, :D], v.transpose(0, 1)))
    want = cache_ref.get(cache.data[0], page, kv, D)
    at = torch.tensor([r if 0 <= r < pages * page else -1 for r in rows], device=DEV)
    for x, y in ((k[:, :kv, :D], want[0]), (v.transpose(0, 1), want[1])):
        y = torch.where((at < 0)[:, None, None], torch.zeros_like(y[at]), y[at])
        assert torch.equal(x.double().nan_to_num(nan=1.25e300), y.to(TYPES[kind]).double().nan_to_num(nan=1.25e300))
    assert bool((k[:, kv:] == 7).all()) and bool((k[..., D:] == 7).all())
    if kind == "bf16":  # what was written comes back from another place's values exactly
        again = bt.cache4_read(cache, i32(rows), dtype=torch.bfloat16)
        assert torch.equal(again[0].nan_to_num(nan=9.0), k[:, :kv, :D].nan_to_num(nan=9.0))


def test_nothing_to_do():
    cache = bt.Cache4(0, 16, 1, 64)
    none = torch.zeros((0, 1, 64), dtype=torch.bfloat16, device=DEV)
    bt.cache4_write(cache, none, none, i32([]))
    one = torch.ones((2, 1, 64), dtype=torch.bfloat16, device=DEV)
    bt.cache4_write(cache, one, one, i32([0, -1]))
    k, v = bt.cache4_read(cache, i32([0, 5]))
    assert bool((k == 0).all()) and bool((v == 0).all())


# ------------------------------------------------------------------------ attention


class Case:
    def __init__(self, q_len, k_len, heads, kv, D, kind, page=16, seed=0, tail=0, layers=1, spread=1.0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.kind, self.kv, self.D, self.page = TYPES[kind], kv, D, page
        self.q_start = [0]
        for n in q_len:
            self.q_start.append(self.q_start[-1] + n)
        self.k_len = list(k_len)
        need = [-(-n // page) for n in k_len]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.W = max(need + [1])
        self.table, at = [], 0
        for n in need:
            self.table.append(order[at: at + n] + [2 ** 31 - 1] * (self.W - n))  # what lies behind is not read
            at += n
        # pages hold anything but NaN scales where no key lies, and NaN scales in unused pages
        data = random_data(g, layers, pages, bt.cache4_page_bytes(page, kv, D))
        self.cache = bt.Cache4(pages, page, kv, D, layers=layers, data=data)
        self.layer = layers - 1
        rows = [self.table[b][j // page] * page + j % page for b, n in enumerate(k_len) for j in range(n)]
        k, v = (torch.randn(len(rows), kv, D, generator=g, device=DEV) * spread for _ in range(2))
        bt.cache4_write(self.cache, k, v, i32(rows), layer=self.layer)
        T = self.q_start[-1] + tail
        self.q = torch.randn(T, heads, D, generator=g, device=DEV).to(self.kind)

    def run(self, causal=True, **more):
        lse = torch.full(self.q.shape[:2], 77.0, device=DEV)
        out, _ = bt.attention4(self.q, self.cache, i32(self.table).view(-1, self.W), i32(self.k_len), i32(self.q_start),
                               layer=self.layer, causal=causal, lse=lse, **more)
        return out, lse

    def check(self, out, lse, causal=True, scale=None):
        data = self.cache.data[self.layer]
        k, v, start, left = cache_ref.gather(data, self.table, self.k_len, self.page, self.kv, self.D)
        assert left == self.k_len
        args = (self.q_start, start, self.k_len, causal, scale)
        ref, rlse = block_ref.attention(self.q.double(), k, v, *args)
        mag, _ = block_ref.attention(self.q.double(), k, v.abs(), *args)
        tol, ltol = tolerance(self.q, k, max(self.k_len + [0]), mag, ref, rlse, out.dtype, scale)
        self.tol = tol
        n = self.q_start[-1]
        d = (out.double() - ref).abs()
        assert not bool(ref[:n].isnan().any())
        assert bool((d[:n] <= tol[:n]).all()), float((d / tol)[:n].max())
        finite = torch.isfinite(rlse[:n])
        assert torch.equal(torch.isfinite(lse[:n]), finite) and bool((lse[:n][~finite] == -math.inf).all())
        assert bool(((lse.double() - rlse).abs() <= ltol)[:n][finite].all())
        return ref


def tolerance(q, k, keys, mag, ref, rlse, out_type, scale=None):
    """(of out, of lse); see the head of the file."""
    D = q.shape[-1]
    s = D ** -0.5 if scale is None else scale
    kmax = float(k.norm(dim=-1).max()) if k.numel() else 0.0
    qk = s * q.double().norm(dim=-1, keepdim=True) * kmax  # bounds scale * sum |q k|
    e = 2 * (D / 8 + 2) * 2.0 ** -24 * qk
    rest = (keys / 16 + 4) * 2.0 ** -24
    parts = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -16}.get(out_type, 2.0 ** -8)
    tol = (2 * e + parts + 2 * rest) * mag + torch.finfo(out_type).eps / 2 * ref.abs() * (1 + 2.0 ** -8) + 1e-30
    if out_type == torch.float16:
        tol = tol + 2.0 ** -25
    return tol, e[..., 0] + rest + 3 * 2.0 ** -24 * rlse.abs()


CASES = [
    # q lengths, k lengths, heads, kv, D, type, page, causal
    ([1], [1], 1, 1, 8, "bf16", 16, True),
    ([1], [777], 20, 5, 128, "bf16", 16, True),
    ([1] * 9, [0, 1, 15, 16, 17, 31, 33, 300, 64], 8, 2, 128, "bf16", 16, True),
    ([1] * 5, [1500, 0, 2300, 64, 65], 64, 8, 128, "fp16", 32, True),
    ([5, 1, 3, 0, 4], [400, 17, 3, 9, 2], 6, 3, 80, "fp16", 16, True),  # the last: rows that see nothing
    ([5, 1, 3, 0, 4], [400, 17, 3, 9, 2], 6, 3, 80, "bf16", 64, False),
    ([64], [64], 8, 2, 128, "bf16", 16, True),
    ([300, 1, 17, 0, 129], [300, 1, 17, 0, 129], 20, 5, 128, "bf16", 64, True),
    ([257, 31], [900, 31], 7, 1, 128, "fp16", 128, True),
    ([200, 90], [230, 1100], 8, 1, 256, "bf16", 16, True),
    ([33], [33], 5, 5, 32, "fp16", 16, False),
    ([90, 3], [50, 3], 12, 4, 96, "bf16", 32, True),  # more queries than keys
    ([1, 2, 150], [2100, 40, 2000], 16, 2, 64, "bf16", 1024, True),
    ([1], [4099], 4, 4, 256, "fp16", 16, True),
    ([700], [700], 4, 2, 64, "fp16", 32, True),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("q,k,heads,kv,D,kind,page,causal", CASES)
def test_attention4(q, k, heads, kv, D, kind, page, causal, wide):
    note(f"attention4 {q} over {k}, {heads}/{kv} x {D} {kind} page {page} causal {causal} wide {wide}")
    c = Case(q, k, heads, kv, D, kind, page, seed=len(q) + D, tail=2, layers=2)
    out, lse = c.run(causal, out=torch.full(c.q.shape, 5.0, dtype=torch.float32 if wide else c.kind, device=DEV))
    c.check(out, lse, causal)
    n = c.q_start[-1]
    assert bool((out[n:] == 5).all()) and bool((lse[n:] == 77).all())  # rows behind the last sequence
    again, lse2 = c.run(causal, out_dtype=out.dtype)
    assert torch.equal(again[:n], out[:n]) and torch.equal(lse2[:n], lse[:n])
    empty = (lse[:n] == -math.inf)
    assert bool((out[:n][empty] == 0).all())


@pytest.mark.parametrize("scale", [0.01, 1.7])
def test_attention4_scale_and_large_scores(scale):
    note(f"attention4 scale {scale}")
    c = Case([1, 40], [600, 100], 4, 2, 64, "bf16", spread=3.0)
    c.check(*c.run(scale=scale, out_dtype=torch.float32), scale=scale)


def test_attention4_strides():
    note("attention4 strides")
    c = Case([3, 40, 1], [30, 70, 600], 8, 2, 64, "bf16", tail=1)
    wide = torch.zeros(c.q.shape[0], 12, 72, dtype=torch.bfloat16, device=DEV)
    wide[:, 2:10, :64] = c.q
    c.q = wide[:, 2:10, :64]
    room = torch.full((8, c.q.shape[0], 68), 3.0, device=DEV)
    out = room.transpose(0, 1)[..., :64]
    table = torch.full((3, c.W + 5), -1, dtype=torch.int32, device=DEV)
    table[:, 1: 1 + c.W] = i32(c.table)
    lse = torch.empty(c.q.shape[:2], device=DEV)
    bt.attention4(c.q, c.cache, table[:, 1: 1 + c.W], i32(c.k_len), i32(c.q_start), out=out, lse=lse)
    c.check(out, lse)
    assert bool((room[..., 64:] == 3).all()) and bool((out[-1] == 3).all())


@pytest.mark.parametrize("q,k,heads,kv,D,kind", [([1, 3], [200, 40], 8, 2, 128, "bf16"), ([60], [150], 2, 1, 64, "fp16"),
                                                 ([40, 90], [40, 300], 2, 2, 256, "bf16"), ([4], [4], 4, 1, 32, "fp16"),
                                                 ([2], [2000], 4, 2, 64, "bf16"), ([150], [150], 2, 2, 128, "bf16")])
def test_attention4_nan(q, k, heads, kv, D, kind):
    """NaN groups: in V, NaN in that group of the rows that see the key; in K, NaN rows; unseen, nothing. Places past
    a sequence's end hold NaN scales, too."""
    note(f"attention4 nan {q} over {k} D {D}")
    c = Case(q, k, heads, kv, D, kind, page=16, seed=9)
    clean, clean_lse = c.run(out_dtype=torch.float32)
    c.check(clean, clean_lse)
    G = -(-D // 32)
    flat = c.cache.data[0].view(-1)

    def place(b, j):
        return c.table[b][j // 16] * 16 + j % 16

    ends = [cache_ref.places(place(b, n), 16, kv, D) for b, n in enumerate(k) if n % 16]
    for _, scales in ends:
        for at in scales:
            flat[at.flatten().to(DEV)] = 253
    out, lse = c.run(out_dtype=torch.float32)
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
    # a V group of head kv - 1 in the last key of every sequence, and one in the middle
    hit = [(0, k[0] - 1, G - 1), (0, k[0] // 2, 0)] + [(len(k) - 1, k[-1] - 1, 0)]
    saved = flat.clone()
    for b, j, group in hit:
        _, scales = cache_ref.places(place(b, j), 16, kv, D)
        flat[int(scales[1][kv - 1, group])] = 255
    for dtype in (torch.float32, c.kind):
        out, lse = c.run(out_dtype=dtype)
        want = torch.zeros(out.shape, dtype=torch.bool, device=DEV)
        for b, j, group in hit:
            first = max(0, j - (k[b] - q[b]))
            want[c.q_start[b] + first: c.q_start[b + 1], (kv - 1) * (heads // kv):, 32 * group: 32 * group + 32] = True
        assert torch.equal(out.isnan(), want)
        assert torch.equal(lse, clean_lse)
        if dtype == torch.float32:
            assert torch.equal(out[~want], clean[~want])
    flat.copy_(saved)
    b, j = 0, k[0] - 1
    _, scales = cache_ref.places(place(b, j), 16, kv, D)
    flat[int(scales[0][0, 0])] = 254
    out, lse = c.run(out_dtype=torch.float32)
    want = torch.zeros(lse.shape, dtype=torch.bool, device=DEV)
    want[c.q_start[1] - 1, : heads // kv] = True
    assert torch.equal(lse.isnan(), want) and torch.equal(out.isnan().any(-1), want)
    # rows beside it may be rescaled at other keys: each result within its tolerance
    assert bool(((out.double() - clean.double()).abs() <= 2 * c.tol)[~want].all())


@pytest.mark.parametrize("q,page", [(1, 16), (1, 64), (50, 16), (50, 128)])
def test_attention4_entries_outside(q, page):
    """The keys of entries that name no page are as if they were not there; k_len past the table is cut."""
    note(f"attention4 entries outside, q {q} page {page}")
    c = Case([q, 1], [600, 300], 4, 2, 64, "bf16", page=page)
    W = c.W
    c.table[0][1], c.table[0][3], c.table[1][0] = -1, c.cache.pages, -(2 ** 31)
    data = c.cache.data[0]
    out, lse = c.run(causal=False, out_dtype=torch.float32)
    k, v, start, left = cache_ref.gather(data, c.table, c.k_len, page, 2, 64)
    ref, rlse = block_ref.attention(c.q.double(), k, v, c.q_start, start, left, False)
    mag, _ = block_ref.attention(c.q.double(), k, v.abs(), c.q_start, start, left, False)
    tol, ltol = tolerance(c.q, k, 600, mag, ref, rlse, out.dtype)
    assert bool(((out.double() - ref).abs() <= tol).all())
    assert bool(((lse.double() - rlse).abs() <= ltol).all())
    full = i32(c.table)
    a = bt.attention4(c.q, c.cache, full[:, : W - 2], i32([10 ** 9, -5]), i32(c.q_start), causal=False)[0]
    b = bt.attention4(c.q, c.cache, full[:, : W - 2].contiguous(), i32([(W - 2) * page, 0]), i32(c.q_start), causal=False)[0]
    assert torch.equal(a, b) and bool((b[q:] == 0).all())


def test_attention4_without_keys():
    note("attention4 without keys")
    for pages, W in ((0, 4), (3, 0), (0, 0)):
        cache = bt.Cache4(pages, 16, 2, 64)
        q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device=DEV)
        lse = torch.zeros(3, 4, device=DEV)
        out, _ = bt.attention4(q, cache, torch.zeros((1, W), dtype=torch.int32, device=DEV), i32([50]), i32([0, 3]), lse=lse)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    out, _ = bt.attention4(q[:0], cache, torch.zeros((0, 0), dtype=torch.int32, device=DEV), i32([]), i32([0]))
    assert out.shape == (0, 4, 64)


def test_far_pages():
    """Pages past 4 GiB of a pool, for the write, the read and the attention."""
    page, kv, D = 1024, 8, 128
    size = bt.cache4_page_bytes(page, kv, D)
    pages = (5 << 30) // size
    note(f"far pages: {pages} of {size} bytes")
    cache = bt.Cache4(pages, page, kv, D)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    n = 1500
    table = [[pages - 1, 0], [pages - 2, pages - 3]]
    k, v = (torch.randn(2 * n, kv, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    rows = [t[j // page] * page + j % page for t in table for j in range(n)]
    bt.cache4_write(cache, k, v, i32(rows))
    kk, vv = bt.cache4_read(cache, i32(rows))
    for x, y in ((kk, k), (vv, v)):
        assert torch.equal(x.double(), cache_ref.decode(*cache_ref.encode(y), D))
    q = torch.randn(2, 16, D, generator=g, device=DEV).bfloat16()
    out, _ = bt.attention4(q, cache, i32(table), i32([n, n]), i32([0, 1, 2]), out_dtype=torch.float32)
    args = ([0, 1, 2], [0, n], [n, n], True)
    ref, rlse = block_ref.attention(q.double(), kk.double(), vv.double(), *args)
    mag, _ = block_ref.attention(q.double(), kk.double(), vv.double().abs(), *args)
    tol, _ = tolerance(q, kk.double(), n, mag, ref, rlse, out.dtype)
    assert bool(((out.double() - ref).abs() <= tol).all())


def test_two_streams_and_replays():
    """Two captured graphs with workspaces of their own, replayed on two streams with new inputs in between; and a
    call on a stream other than the one the inputs were made on."""
    note("attention4 graphs")
    cases = [Case([1] * 4, [900, 700, 30, 0], 20, 5, 128, "bf16"), Case([70], [900], 8, 2, 64, "fp16", page=32)]
    runs = []
    torch.cuda.synchronize()
    for c in cases:
        tensors = (i32(c.table).view(-1, c.W), i32(c.k_len), i32(c.q_start))
        out, lse = torch.empty(c.q.shape, device=DEV), torch.empty(c.q.shape[:2], device=DEV)
        ws = bt.attention4_workspace(c.q, c.cache, tensors[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            bt.attention4(c.q, c.cache, *tensors, out=out, lse=lse, workspace=ws)
            side.synchronize()
            with torch.cuda.graph(graph, stream=side):
                bt.attention4(c.q, c.cache, *tensors, out=out, lse=lse, workspace=ws)
        runs.append((c, tensors, out, lse, ws, side, graph))
    for turn in range(3):
        for c, tensors, out, lse, ws, side, graph in runs:
            c.q.copy_(torch.randn(c.q.shape, device=DEV))
            c.k_len[0] = 900 - 100 * turn
            tensors[1].copy_(i32(c.k_len))
        torch.cuda.synchronize()
        for *_, side, graph in runs:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for c, _, out, lse, *_ in runs:
            c.check(out, lse)
