"""bt_attention where sums and probabilities are at the ends of their ranges, in every form of the kernel:
few rows, 64-row and 128-row tiles, with and without a prefix."""
import math

import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests import block_ref
from tests.test_block_attention_gpu import Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LN2 = math.log(2.0)


def note(msg):
    print(f"[gpu-case] {msg}", flush=True)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


# One query sequence length each (all sequences see the same keys), key heads, sequences, keys, prefix
FORMS = {
    "few rows, uncut": (1, 1, 2, 1000, 0),
    "few rows, long slices": (1, 1, 512, 65536, 0),
    "64-row tiles, uncut": (8192, 1, 1, 131072, 0),
    "64-row tiles, slices": (200, 2, 1, 40000, 0),
    "128-row tiles, uncut": (2048, 32, 1, 30000, 0),
    "prefix, few rows": (1, 4, 3, 5, 9000),
    "prefix, tiles": (4096, 8, 1, 64, 20000),
}


@pytest.mark.parametrize("exponent", [16, 25, 26])
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("form", FORMS)
def test_one_large_probability_and_a_long_flat_tail(form, kind, exponent):
    """Key j0 has a score of e ln 2 above all others, so each of them has 2^-e of its probability.

    Tolerance. The scale is ln 2 to 2^-24 of itself, so scores in powers of two are whole but for
    26 * 2^-23, and exp is 2^-e but for 2^-18 relative. From there on sums are exact: eight tail products, which the
    matrix cores add at once, are 2^(3 - e) of the accumulator, at least one unit in its last place for
    e <= 26, and a block's tail, which is one term of the sum of probabilities, is a multiple of the
    same; the relative 2^-18 of a term may move each by half a unit, so 2^-18 of the tail's mass plus 2^-24
    per block of 64 keys (32 keys to a lane) in a sum that is 1 + n 2^-e. The probabilities, powers of two but
    for 2^-18, are rounded to the type or two of it: relative to the tail's mass by eps / 2. What is left
    is the division, the slices' joining (8 roundings), and the output's own rounding. None of it grows with
    the number of keys other than by 2^-24 per block."""
    n_q, kv, seqs, S, P = FORMS[form]
    note(f"attention tail {form} {kind} 2^-{exponent}")
    dt, D = TYPES[kind], 8
    j0 = (P or S) // 3  # in the prefix, where there is one
    scale = LN2
    q = torch.zeros((n_q * seqs, kv, D), dtype=dt, device=DEV)
    q[..., 0] = 1
    k = torch.zeros((S, kv, D), dtype=dt, device=DEV)
    v = torch.ones((S, kv, D), dtype=dt, device=DEV)
    pk = torch.zeros((P, kv, D), dtype=dt, device=DEV) if P else None
    pv = torch.ones((P, kv, D), dtype=dt, device=DEV) if P else None
    (pk if P else k)[j0, :, 0] = exponent
    (pv if P else v)[j0, :, 4:] = 0  # dimensions 4 .. 7: the tail's mass alone
    starts = i32([n_q * b for b in range(seqs + 1)])
    zeros, lens = i32([0] * seqs), i32([S] * seqs)
    n = S + P - 1
    tail = n * 2.0 ** -exponent
    for out_dtype in (dt, torch.float32):
        lse = torch.empty((n_q * seqs, kv), device=DEV)
        out, _ = bt.attention(q, k, v, starts, zeros, lens, causal=False, scale=scale, prefix_k=pk, prefix_v=pv,
                              out_dtype=out_dtype, lse=lse)
        eps, half = torch.finfo(dt).eps / 2, torch.finfo(out_dtype).eps / 2
        part = tail / (1 + tail)
        unit = (n / 64 + 12) * 2.0 ** -24
        p_err = (2.0 ** -18 + (eps if out_dtype == dt else eps * eps)) * part + unit
        one = (out[..., :4].double() - 1).abs().max()
        assert float(one) <= p_err + half * (1 + 2.0 ** -7), float(one)
        rest = (out[..., 4:].double() - part).abs().max()
        # an fp16 output below 2^-14 is rounded absolutely
        assert float(rest) <= p_err + half * part + (2.0 ** -25 if out_dtype == torch.float16 else 0), float(rest)
        want = exponent * LN2 + math.log1p(tail)
        assert float((lse.double() - want).abs().max()) <= p_err + 26 * 2.0 ** -23 + 4 * 2.0 ** -24 * want


# q lengths, k lengths, slab, heads, key heads, D, prefix
BAD_VALUES = {
    "few rows, uncut": ([1, 4], [400, 300], 500, 4, 1, 128, 0),
    "few rows, slices": ([1] * 3, [3000, 700, 2100], 3000, 8, 2, 64, 0),
    "64-row tiles, slices": ([200], [2000], 0, 8, 2, 128, 0),
    "64-row tiles, uncut": ([400] * 12, [400] * 12, 0, 8, 4, 80, 0),
    "128-row tiles, uncut": ([700] * 4, [700] * 4, 0, 32, 8, 128, 0),
    "128-row tiles, D 256": ([500] * 9, [500] * 9, 0, 16, 16, 256, 0),
    "prefix, few rows": ([1, 1, 2], [100, 0, 90], 100, 4, 4, 128, 1500),
    "prefix, tiles and few rows": ([1] * 40, [(7 * i) % 60 for i in range(40)], 64, 8, 2, 64, 1500),
    "prefix, tiles": ([150, 20], [150, 25], 160, 6, 3, 80, 700),
}


@pytest.mark.parametrize("scale", [0.1, 5.0])
@pytest.mark.parametrize("out_type", ["type", "fp32"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("form", BAD_VALUES)
def test_infinities_and_nans_that_a_row_sees_are_its_output(form, kind, out_type, scale):
    """In fully visible blocks as in masked ones, however small the probability (with a scale of 5 nearly
    all are 0 in fp32) and whatever its rest; and columns that hold none are as if there were none."""
    q_len, k_len, slab, heads, kv, D, P = BAD_VALUES[form]
    note(f"attention bad values {form} {kind} {out_type} scale={scale}")
    dt = TYPES[kind]
    g = torch.Generator(device=DEV)
    g.manual_seed(31)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(dt)  # noqa: E731
    q_start = [sum(q_len[:b]) for b in range(len(q_len) + 1)]
    k_start = [b * slab if slab else sum(k_len[:b]) for b in range(len(k_len))]
    S = len(k_len) * slab if slab else sum(k_len)
    q, k, v = rnd(q_start[-1], heads, D), rnd(S, kv, D), rnd(S, kv, D)
    pk, pv = (rnd(P, kv, D), rnd(P, kv, D)) if P else (None, None)

    def place(rows, first, n):
        """Early, middle and late keys of n from `first` on, each in dimensions of its own."""
        if n > 6:
            rows[first + 2, :, 1] = math.inf
            rows[first + 3, :, 2] = -math.inf
            rows[first + 4, :, D - 1] = math.nan
            rows[first + 2, :, 4] = math.inf
            rows[first + n // 2, :, 4] = -math.inf
            rows[first + n // 2, :, 5] = math.inf
            rows[first + n - 1, :, 6] = -math.inf
            rows[first + n - 2, :, 8 % D] = math.nan

    for b in range(len(k_len)):
        if b != 1:  # one sequence has none
            place(v, k_start[b], k_len[b])
    if P:
        pv[7, :, 9] = math.inf
        pv[P - 1, :, 10] = -math.inf
        pv[P // 2, :, 11] = math.nan
    args = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (q_start, k_start, k_len)]
    out_dtype = torch.float32 if out_type == "fp32" else dt

    def run(values, prefix_values):
        lse = torch.empty((q.shape[0], heads), device=DEV)
        out, _ = bt.attention(q, k, values, *args, scale=scale, prefix_k=pk, prefix_v=prefix_values, lse=lse,
                              out_dtype=out_dtype)
        return out, lse

    out, lse = run(v, pv)
    ref, _ = block_ref.attention(q, k, v, q_start, k_start, k_len, True, scale, prefix_k=pk, prefix_v=pv)
    for name, test in (("nan", torch.isnan), ("inf", lambda t: t == math.inf), ("-inf", lambda t: t == -math.inf)):
        assert torch.equal(test(out), test(ref)), (name, int((test(out) != test(ref)).sum()))
    zero = lambda t: None if t is None else torch.where(torch.isfinite(t), t, torch.zeros_like(t))  # noqa: E731
    plain, plain_lse = run(zero(v), zero(pv))
    fine = torch.isfinite(ref)
    assert torch.equal(out[fine], plain[fine]) and torch.equal(lse, plain_lse)


UNSEEN = {
    "few rows": ([4, 3], [70, 3], 8, 2, 128, 0),
    "few rows, slices": ([1, 2], [300, 4000], 8, 2, 64, 0),
    "64-row tiles, slices": ([150], [1400], 8, 2, 128, 0),
    "64-row tiles, uncut": ([400] * 12, [400] * 12, 8, 4, 80, 0),
    "128-row tiles, uncut": ([700] * 4, [700] * 4, 32, 8, 128, 0),
    "prefix, tiles and few rows": ([3] * 12, [20 + b for b in range(12)], 8, 2, 128, 900),
    "prefix, tiles": ([150, 20], [150, 25], 6, 3, 80, 700),
}


@pytest.mark.parametrize("out_type", ["type", "fp32"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("form", UNSEEN)
def test_keys_and_values_that_are_nan_reach_only_rows_that_see_them(form, kind, out_type):
    """The last key and value of every sequence, which its last query alone sees, are NaN: all other rows are
    bit for bit what they are without."""
    q_len, k_len, heads, kv, D, P = UNSEEN[form]
    note(f"attention unseen {form} {kind} {out_type}")
    c = Case(q_len, k_len, heads, kv, D, kind, prefix=P, seed=12)
    out_dtype = torch.float32 if out_type == "fp32" else c.dt
    want, want_lse = c.run(out_dtype=out_dtype)
    last = torch.tensor([n - 1 for n in c.q_start[1:]], device=DEV)
    for b, n in enumerate(k_len):
        c.k[c.k_start[b] + n - 1] = math.nan
        c.v[c.k_start[b] + n - 1] = math.nan
    out, lse = c.run(out_dtype=out_dtype)
    rest = torch.ones(out.shape[0], dtype=torch.bool, device=DEV)
    rest[last] = False
    assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])
    assert bool(out[last].isnan().all()) and bool(lse[last].isnan().all())


INSTANCES = [
    # q lengths, k lengths, heads, key heads, D, prefix: tiles of 128 rows go uncut in the first five, few rows
    # stand behind a tiled prefix in the others
    ([700] * 4, [700] * 4, 32, 8, 64, 0),
    ([900, 30, 800, 1000], [900, 30, 800, 1000], 32, 32, 40, 0),
    ([700] * 4, [700] * 4, 32, 8, 128, 0),
    ([500] * 9, [500] * 9, 16, 16, 256, 0),
    ([450] * 10, [450] * 10, 16, 16, 216, 0),
    ([1] * 40, [(7 * b) % 60 for b in range(40)], 8, 2, 64, 1500),
    ([2, 1] * 15, [(11 * b) % 50 for b in range(30)], 12, 4, 96, 700),
    ([1] * 40, [(7 * b) % 60 for b in range(40)], 8, 2, 128, 3001),
    ([1, 3] * 10, [(5 * b) % 90 for b in range(20)], 8, 4, 256, 800),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("q_len,k_len,heads,kv,D,P", INSTANCES)
def test_every_instance_of_the_large_tiles(q_len, k_len, heads, kv, D, P, kind):
    note(f"attention instances q={q_len[:4]} heads={heads}/{kv} D={D} prefix={P} {kind}")
    c = Case(q_len, k_len, heads, kv, D, kind, prefix=P, seed=D + P)
    assert P or bt.attention_workspace_bytes(sum(q_len), sum(k_len), len(q_len), heads, kv, D) == 0  # uncut
    for out_dtype in (c.dt, torch.float32):
        out, lse = c.run(out_dtype=out_dtype)
        c.check(out, lse)


FEW = [
    ([1], [777], 1024, 20, 5, 128, 0),
    ([1] * 20, [(331 * b) % 3000 for b in range(20)], 3000, 20, 5, 128, 0),
    ([4, 1, 2], [900, 300, 77], 900, 8, 2, 64, 0),
    ([1, 1], [5000, 4000], 5000, 8, 1, 256, 0),
    ([1, 1, 2], [90, 0, 60], 90, 4, 4, 96, 1500),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("q_len,k_len,slab,heads,kv,D,P", FEW)
def test_few_rows_round_once(q_len, k_len, slab, heads, kv, D, P, kind):
    """The 16-bit outputs of few rows are off by their own rounding and by what fp32 sums are: probabilities
    are carried to twice the type's precision. Tolerance: half a step of the output; eps / 2 squared of
    sum p |v| for the probabilities (fp16: at least 2^-34 of the largest for every key); an error e of a
    score counts twice (the probability and the sum), e being D / 8 + 2 roundings of scale * sum |q k|, and
    sums of n keys n / 16 + 4 roundings, both as for the other forms; joining slices 8 roundings."""
    note(f"attention few rows rounding q={q_len[:4]} heads={heads}/{kv} D={D} prefix={P} {kind}")
    c = Case(q_len, k_len, heads, kv, D, kind, slab=slab, prefix=P, seed=7 + D)
    out, _ = c.run()
    wide = lambda t: None if t is None else t.double()  # noqa: E731
    args = (c.q_start, c.k_start, c.k_len, True)
    ref, _ = block_ref.attention(c.q.double(), c.k.double(), c.v.double(), *args, prefix_k=wide(c.pk),
                                 prefix_v=wide(c.pv))
    mag, _ = block_ref.attention(c.q.double(), c.k.double(), c.v.double().abs(), *args, prefix_k=wide(c.pk),
                                 prefix_v=None if c.pv is None else c.pv.double().abs())
    eps = torch.finfo(c.dt).eps / 2
    n = max(k_len) + P
    kmax = max(float(t.double().norm(dim=-1).max()) for t in (c.k, c.pk) if t is not None)
    e = (D / 8 + 2) * 2.0 ** -24 * D ** -0.5 * c.q.double().norm(dim=-1, keepdim=True) * kmax
    tol = (2 * e + eps * eps + 2 * (n / 16 + 12) * 2.0 ** -24) * mag + eps * ref.abs() * (1 + 2.0 ** -7) + 1e-30
    if kind == "fp16":
        sums = [t.double().abs().sum(0).max() for t in (c.v, c.pv) if t is not None]
        tol = tol + 2.0 ** -34 * float(sum(sums)) + 2.0 ** -25
    d = (out.double() - ref).abs()
    assert bool((d <= tol).all()), float((d / tol).max())
