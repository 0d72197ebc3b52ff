"""bt_attention against its definition in 64 bits: packed prompts, continued prompts, decode steps over
cache slabs, short drafts, shared prefixes, empty rows, strides, and infinities in unseen places.

Tolerance. The exact result is sum_j p_j v_j with p from the given q, k, v (their types are exact).
 - Probabilities are rounded to the type of V: eps / 2 each, so eps / 2 * sum_j p_j |v_j| in all, and the
   sum of probabilities is taken before that rounding. Below the smallest normal fp16 number the
   rounding is absolute, 2^-25 of the row's largest probability each (never above 2^8 of the reference):
   2^-25 * sum_j |v_j| at most. With fp32 outputs the probability is carried as two values: (eps / 2)^2
   in place of eps / 2 (fp16: still the 2^-25 of a subnormal rest).
 - Scores: fp32 sums of D exact products, off by at most D * 2^-24 * scale * sum |q k| (fewer in practice:
   instructions add 16 products at once; D / 8 is asked for) and two roundings more of the score itself
   (the FMA with the reference, in powers of two); a score error e changes p_j by a factor within e, so
   the output by at most 2 e * sum_j p_j |v_j| (p_j and the sum).
 - v_exp_f32 and the reciprocal: 2 * 2^-23. fp32 sums over n keys: taken as n / 16 * 2^-24, blocks being
   added by the matrix cores.
 - One rounding to the output type: eps / 2 of the value.
lse: the score error, the sum's n / 16 * 2^-24, and three roundings of the value itself.
"""
import math

import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests import block_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def note(msg):
    print(f"[gpu-case] {msg}", flush=True)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


class Case:
    def __init__(self, q_len, k_len, heads, kv, D, kind, slab=0, prefix=0, seed=0, tail=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.dt = TYPES[kind]
        rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(self.dt)  # noqa: E731
        self.q_start, self.k_start = [0], []
        for n in q_len:
            self.q_start.append(self.q_start[-1] + n)
        at = 0
        for b, n in enumerate(k_len):
            self.k_start.append(b * slab if slab else at)
            at += n
        self.k_len = list(k_len)
        T, S = self.q_start[-1] + tail, (len(k_len) * slab if slab else at)
        self.q, self.k, self.v = rnd(T, heads, D), rnd(S, kv, D), rnd(S, kv, D)
        self.pk = rnd(prefix, kv, D) if prefix else None
        self.pv = rnd(prefix, kv, D) if prefix else None

    def offsets(self):
        return i32(self.q_start), i32(self.k_start), i32(self.k_len)

    def run(self, causal=True, **more):
        lse = torch.full(self.q.shape[:2], 77.0, device=DEV)
        out, _ = bt.attention(self.q, self.k, self.v, *self.offsets(), causal=causal, prefix_k=self.pk,
                              prefix_v=self.pv, lse=lse, **more)
        return out, lse

    def check(self, out, lse, causal=True, scale=None):
        q, k, v = self.q.double(), self.k.double(), self.v.double()
        pk = None if self.pk is None else self.pk.double()
        pv = None if self.pv is None else self.pv.double()
        args = (self.q_start, self.k_start, self.k_len, causal, scale)
        ref, rlse = block_ref.attention(q, k, v, *args, prefix_k=pk, prefix_v=pv)
        absv = lambda t: None if t is None else t.abs()  # noqa: E731
        mag, _ = block_ref.attention(q, k, v.abs(), *args, prefix_k=pk, prefix_v=absv(pv))
        D = q.shape[-1]
        s = D ** -0.5 if scale is None else scale
        keys = max([0] + self.k_len) + (0 if pk is None else pk.shape[0])
        kmax = max([float(t.double().norm(dim=-1).max()) for t in (self.k, self.pk) if t is not None and t.numel()] or [0])
        qk = s * q.norm(dim=-1, keepdim=True) * kmax  # bounds scale * sum |q k|
        e = (D / 8 + 2) * 2.0 ** -24 * qk
        eps = torch.finfo(self.dt).eps / 2
        rest = (keys / 16 + 4) * 2.0 ** -24
        round_p = eps if out.dtype != torch.float32 else eps * eps
        tol = (2 * e + round_p + 2 * rest) * mag + torch.finfo(out.dtype).eps / 2 * ref.abs() * (1 + 2 * eps) + 1e-30
        if self.dt == torch.float16:
            vs = [t.double().abs().sum(0).max() for t in (self.v, self.pv) if t is not None and t.numel()]
            tol = tol + 2.0 ** -25 * float(max(vs or [0.0])) * (1.0 if keys else 0.0)
            if out.dtype == torch.float16:
                tol = tol + 2.0 ** -25
        d = (out.double() - ref).abs()
        n = self.q_start[-1]
        assert not bool(ref[:n].isnan().any())
        assert bool((d[:n] <= tol[:n]).all()), float((d / tol)[:n].max())
        finite = torch.isfinite(rlse[:n])
        assert torch.equal(torch.isfinite(lse[:n]), finite) and bool((lse[:n][~finite] == -math.inf).all())
        ltol = e[..., 0] + rest + 3 * 2.0 ** -24 * rlse.abs()
        assert bool(((lse.double() - rlse).abs() <= ltol)[:n][finite].all())
        return ref


PROMPTS = [
    # q lengths (= k lengths), heads, kv, D, type, causal
    ([1], 1, 1, 8, "bf16", True),
    ([5], 4, 4, 64, "fp16", True),
    ([64], 8, 2, 128, "bf16", True),
    ([65, 63, 1, 128], 6, 3, 80, "bf16", True),
    ([300, 1, 17, 0, 129], 20, 5, 128, "bf16", True),
    ([257, 31], 7, 1, 128, "fp16", True),
    ([200, 90], 8, 1, 256, "bf16", True),
    ([140, 33], 4, 2, 216, "fp16", True),
    ([500], 12, 4, 96, "fp16", True),
    ([130, 258], 5, 5, 40, "bf16", False),
    ([1030], 2, 1, 128, "bf16", False),
    ([2000, 100], 3, 1, 64, "bf16", True),
    ([33] * 70, 4, 2, 64, "fp16", True),
    ([700] * 4, 32, 8, 128, "bf16", True),  # enough tiles to go uncut
]


@pytest.mark.parametrize("q_len,heads,kv,D,kind,causal", PROMPTS)
def test_packed_prompts(q_len, heads, kv, D, kind, causal):
    note(f"attention prompts {q_len[:6]} heads={heads}/{kv} D={D} {kind} causal={causal}")
    c = Case(q_len, q_len, heads, kv, D, kind, seed=sum(q_len) + D)
    out, lse = c.run(causal)
    c.check(out, lse, causal)
    wide, lse32 = c.run(causal, out_dtype=torch.float32)
    c.check(wide, lse32, causal)


CACHED = [
    # q lengths, k lengths, slab, heads, kv, D, type
    ([1], [1], 1, 20, 5, 128, "bf16"),
    ([1], [777], 1024, 20, 5, 128, "bf16"),
    ([1], [512], 512, 20, 5, 128, "bf16"),  # uncut, and one key more
    ([1], [513], 513, 20, 5, 128, "bf16"),
    ([4, 1], [511, 300], 512, 8, 2, 96, "fp16"),
    ([4, 1], [513, 300], 513, 8, 2, 96, "fp16"),
    ([1] * 7, [0, 1, 31, 32, 33, 500, 64], 500, 32, 32, 128, "fp16"),
    ([1] * 5, [130, 4000, 3, 128, 127], 4000, 8, 1, 256, "bf16"),
    ([1] * 130, [(37 * i) % 300 for i in range(130)], 300, 16, 2, 64, "bf16"),
    ([4, 4, 3, 0, 1], [900, 4, 2, 7, 0], 1000, 12, 4, 96, "fp16"),  # drafts; fewer keys than queries
    ([2] * 9, [50 * i for i in range(9)], 420, 64, 8, 128, "bf16"),
    ([100, 3, 260], [1100, 50, 200], 1200, 20, 5, 128, "bf16"),  # prompts continued; rows with no key
    ([33, 64], [5000, 64], 5000, 6, 3, 80, "fp16"),
    ([5, 1], [9, 70000], 70000, 2, 1, 128, "bf16"),
    ([17] * 20, [40] * 20, 64, 3, 1, 64, "bf16"),
]


@pytest.mark.parametrize("q_len,k_len,slab,heads,kv,D,kind", CACHED)
def test_cached_keys(q_len, k_len, slab, heads, kv, D, kind):
    note(f"attention cached q={q_len[:8]} k={k_len[:8]} slab={slab} heads={heads}/{kv} D={D} {kind}")
    c = Case(q_len, k_len, heads, kv, D, kind, slab=slab, seed=len(q_len) + slab)
    # what a cache holds behind a request's keys is not read
    for b, n in enumerate(k_len):
        c.k[b * slab + n: (b + 1) * slab] = math.nan
        c.v[b * slab + n: (b + 1) * slab] = math.inf
    out, lse = c.run()
    clean = Case(q_len, k_len, heads, kv, D, kind, slab=slab, seed=len(q_len) + slab)
    clean.check(out, lse)
    out32, lse32 = c.run(out_dtype=torch.float32)
    clean.check(out32, lse32)
    plain, lsep = c.run(causal=False)
    clean.check(plain, lsep, causal=False)


PREFIXED = [
    # q lengths, k lengths, prefix, heads, kv, D, type
    ([1], [0], 1, 4, 4, 64, "bf16"),
    ([1] * 8, [1, 200, 0, 33, 64, 7, 129, 90], 1000, 32, 32, 128, "fp16"),
    ([1] * 64, [(31 * i + 5) % 90 for i in range(64)], 2050, 16, 2, 128, "bf16"),
    ([3, 1, 0, 5], [3, 40, 9, 2], 63, 8, 1, 256, "bf16"),
    ([150, 20], [150, 25], 400, 6, 3, 80, "fp16"),
    ([2] * 6, [8] * 6, 9000, 20, 5, 128, "bf16"),
    ([40, 300], [900, 300], 5000, 4, 1, 64, "bf16"),
]


@pytest.mark.parametrize("q_len,k_len,prefix,heads,kv,D,kind", PREFIXED)
def test_shared_prefix(q_len, k_len, prefix, heads, kv, D, kind):
    note(f"attention prefix={prefix} q={q_len[:8]} k={k_len[:8]} heads={heads}/{kv} D={D} {kind}")
    c = Case(q_len, k_len, heads, kv, D, kind, slab=max(k_len) + 3, prefix=prefix, seed=prefix)
    out, lse = c.run()
    c.check(out, lse)
    out32, lse32 = c.run(out_dtype=torch.float32)
    c.check(out32, lse32)


@pytest.mark.parametrize("prefix", [0, 70])
def test_rows_behind_the_last_sequence_stay(prefix):
    note(f"attention tail rows prefix={prefix}")
    c = Case([40, 0, 5], [40, 9, 5], 4, 2, 64, "bf16", prefix=prefix, seed=3, tail=30)
    out = torch.full(c.q.shape, 5.0, dtype=c.dt, device=DEV)
    lse = torch.full(c.q.shape[:2], 6.0, device=DEV)
    bt.attention(c.q, c.k, c.v, *c.offsets(), prefix_k=c.pk, prefix_v=c.pv, out=out, lse=lse)
    c.check(out, lse)
    assert bool((out[45:] == 5).all()) and bool((lse[45:] == 6).all())


@pytest.mark.parametrize("q_len,k_len", [([200], [200]), ([4, 3], [70, 3]), ([150], [400])])
def test_infinities_reach_only_rows_that_see_them(q_len, k_len):
    note(f"attention infinities {q_len} {k_len}")
    c = Case(q_len, k_len, 8, 2, 128, "bf16", seed=9)
    n = sum(k_len)
    where = [(n - 1, 3, math.inf), (n - 1, 5, math.nan), (n - 2, 3, -math.inf), (n - 2, 9, -math.inf)]
    if q_len[0] > 100:
        where += [(n - 70, 11, math.inf), (n - 100, 12, math.nan)]
    for j, d, value in where:
        c.v[j, :, d] = value
    out, lse = c.run()
    ref, _ = block_ref.attention(c.q.double(), c.k.double(), c.v.double(), c.q_start, c.k_start, c.k_len, True)
    for name, test in (("nan", torch.isnan), ("inf", lambda t: t == math.inf), ("-inf", lambda t: t == -math.inf)):
        assert torch.equal(test(out), test(ref)), name
    c.v[~torch.isfinite(c.v)] = 0.0
    zeroed, _ = c.run()
    fine = torch.isfinite(ref)
    assert torch.equal(out[fine], zeroed[fine])
    # keys that are not seen may hold anything
    k = c.k.clone()
    last = c.q_start[1] - 1
    c.k[c.k_start[0] + c.k_len[0] - 1] = math.nan
    out2, lse2 = c.run()
    assert torch.equal(out2[:last], out[:last]) or bool(torch.isnan(out[:last]).any())
    assert bool(torch.isnan(out2[last]).all()) and bool(torch.isnan(lse2[last]).all())
    assert torch.equal(lse2[:last], lse[:last])
    c.k = k


def test_strides_and_head_layouts():
    """Heads-first caches, K and V interleaved in one array, a slice of a fused row, a strided output."""
    note("attention strides")
    heads, kv, D, T, S = 6, 3, 80, 150, 170
    c = Case([150], [150], heads, kv, D, "fp16", seed=4)
    want, wlse = c.run()
    both = torch.zeros((S, 2, kv, D), dtype=c.dt, device=DEV)
    both[:150, 0], both[:150, 1] = c.k, c.v
    fused = torch.zeros((T, 2, heads * D), dtype=c.dt, device=DEV)
    fused[:, 1] = c.q.reshape(T, -1)
    out = torch.zeros((heads, T, 2 * D), dtype=c.dt, device=DEV)
    lse = torch.empty((T, heads), device=DEV)
    bt.attention(fused[:, 1].view(T, heads, D), both[:, 0], both[:, 1],
                 *c.offsets(), out=out[:, :, :D].transpose(0, 1), lse=lse)
    assert torch.equal(out[:, :, :D].transpose(0, 1), want) and torch.equal(lse, wlse)
    assert bool((out[:, :, D:] == 0).all())
    kh = c.k.transpose(0, 1).contiguous().transpose(0, 1)
    vh = c.v.transpose(0, 1).contiguous().transpose(0, 1)
    got, _ = bt.attention(c.q, kh, vh, *c.offsets())
    assert torch.equal(got, want)


def test_shared_rows_and_expanded_heads():
    """Sequences that name the same rows, and one key head expanded to several (stride 0)."""
    note("attention shared rows")
    c = Case([30, 1, 1], [40, 0, 0], 4, 4, 64, "bf16", seed=5)
    c.k_start, c.k_len = [0, 0, 10], [40, 40, 25]
    c.k, c.v = c.k[:, :1].expand(-1, 4, -1), c.v[:, :1].expand(-1, 4, -1)
    out, lse = c.run()
    c.check(out, lse)


def test_scale_and_large_scores():
    note("attention scale")
    for scale in (1.0, 0.01, 4.0):
        c = Case([90, 1], [90, 300], 4, 2, 128, "bf16", seed=6)
        out, lse = c.run(scale=scale)
        c.check(out, lse, scale=scale)
        wide, lse = c.run(scale=scale, out_dtype=torch.float32)
        c.check(wide, lse, scale=scale)


def test_rising_and_falling_maxima():
    """Scores that keep rising (every block rescales) and that fall (none does)."""
    note("attention maxima")
    for sign in (1.0, -1.0):
        for q_len in ([256], [1]):
            c = Case(q_len, [1500 if q_len == [1] else 256], 2, 1, 64, "bf16", seed=7)
            ramp = torch.linspace(-30, 30, c.k.shape[0], device=DEV) * sign
            c.k[:] = (ramp[:, None, None] * torch.ones((1, 1, 64), device=DEV) / 8).to(c.dt)
            c.q[:] = 1.0
            out, lse = c.run(out_dtype=torch.float32)
            c.check(out, lse)


def test_offsets_that_leave_the_arrays_stay_inside():
    """Wrong offsets are cut to the arrays: nothing outside is read or written."""
    note("attention bad offsets")
    room = torch.full((64, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    q, k, v = (torch.randn((16, 2, 64), device=DEV).to(torch.bfloat16) for _ in range(3))
    out = room[24:40]
    for qs, ks, kl in (([-5, 40], [-3], [500]), ([3, 99], [14], [2 ** 31 - 1]), ([9, 2], [2 ** 31 - 1], [7]),
                       ([0, 16, 0, 16, 0, 16], [0, 4, 8, 12, 99], [16, -2, 3, 9, 9])):
        bt.attention(q, k, v, i32(qs), i32(ks), i32(kl), out=out)
        torch.cuda.synchronize()
        assert bool((room[:24] == 3).all()) and bool((room[40:] == 3).all())


@pytest.mark.parametrize("q_len,k_len,prefix", [([1] * 6, [50, 700, 0, 3, 90, 300], 0), ([200, 33], [200, 60], 0),
                                               ([1] * 6, [50, 70, 0, 3, 90, 30], 600)])
def test_graph_replays(q_len, k_len, prefix):
    note(f"attention graph {q_len} {k_len} {prefix}")
    slab = max(k_len)
    c = Case(q_len, k_len, 8, 2, 128, "bf16", slab=slab, prefix=prefix, seed=8)
    qs, ks, kl = c.offsets()
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device=DEV)
    ws = bt.attention_workspace(c.q, c.k, len(q_len), prefix_k=c.pk)
    s = torch.cuda.Stream()

    def call(o, l):
        bt.attention(c.q, c.k, c.v, qs, ks, kl, prefix_k=c.pk, prefix_v=c.pv, out=o, lse=l, workspace=ws)

    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call(out, lse)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(out, lse)
    eager, elsed = torch.empty_like(out), torch.empty_like(lse)
    for rep in range(4):
        c.q.normal_()
        if max(q_len) == 1:  # the lengths are read by every replay
            kl.copy_(torch.randint(0, slab + 1, (len(q_len),), device=DEV, dtype=torch.int32))
        if ws is not None:
            ws.fill_(255)
        call(eager, elsed)
        torch.cuda.synchronize()
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(lse, elsed), rep


def test_no_tokens_no_sequences_no_keys():
    note("attention empty")
    q = torch.randn((3, 2, 64), device=DEV).to(torch.bfloat16)
    k = torch.zeros((0, 1, 64), dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 4.0)
    bt.attention(q, k, k, i32([0]), i32([]), i32([]), out=out)
    assert bool((out == 4).all())
    lse = torch.zeros((3, 2), device=DEV)
    bt.attention(q, k, k, i32([0, 3]), i32([0]), i32([0]), out=out, lse=lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    assert bt.attention(q[:0], k, k, i32([0, 0]), i32([0]), i32([0]))[0].shape == (0, 2, 64)
