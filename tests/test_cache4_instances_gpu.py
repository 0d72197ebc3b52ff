"""bt_attention4 in every kernel instance: both types, outputs of the type and fp32, heads of up to 64, 128 and 256, tiles
of 16, 64 and 128 rows, keys whole and cut into slices; and over tables that are wider than their lengths, as a server's
are. tests/test_attention4_plan.py checks (on the CPU) that no instance is left out.

Tolerance: test_cache4_gpu.py's for fp32 outputs, whose probabilities are exact to 2^-24; for 16-bit outputs 2^-16 of
sum p |v| for two bf16 parts of a probability, and one rounding, eps / 2 of the value (fp16 below 2^-14: 2^-25)."""
import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests import block_ref, cache_ref
from tests.test_cache4_gpu import Case, i32, note, tolerance

pytestmark = pytest.mark.gpu

# form: (q lengths, k lengths, query heads of a key head, key heads)
FORMS = {
    "16 whole": ([1, 1, 2, 1], [300, 17, 200, 0], 4, 2),
    "16 cut": ([1, 1, 1, 1], [1500, 0, 700, 90], 4, 2),
    "64 whole": ([40], [300], 1, 3),
    "64 cut": ([5, 3, 6, 5], [1500, 3, 900, 60], 8, 2),
    "128 whole": ([150], [400], 3, 2),
    "128 cut": ([130, 1, 90], [1200, 600, 90], 4, 2),
}
DIMS = [64, 128, 256]
ODD_DIMS = [8, 40, 96, 136, 200]


def check(c, out, lse, causal=True):
    c.check(out, lse, causal)
    ks, vs, start, _ = cache_ref.gather(c.cache.data[c.layer], c.table, c.k_len, c.page, c.kv, c.D)
    args = (c.q_start, start, c.k_len, causal)
    ref, rlse = block_ref.attention(c.q.double(), ks, vs, *args)
    mag, _ = block_ref.attention(c.q.double(), ks, vs.abs(), *args)
    tol, _ = tolerance(c.q, ks, max(c.k_len), mag, ref, rlse, torch.float32)
    if out.dtype != torch.float32:
        tol = tol + 2.0 ** -16 * mag + torch.finfo(out.dtype).eps / 2 * ref.abs() * (1 + 2.0 ** -8)
    if out.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    d = (out.double() - ref).abs()
    assert bool((d <= tol).all()), float((d / tol).max())


def case(form, D, kind, seed=0):
    q, k, group, kv = FORMS[form]
    return Case(q, k, group * kv, kv, D, kind, page=16, seed=seed + D, layers=2)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("form", FORMS)
def test_instance(form, D, kind, wide):
    note(f"attention4 instance {form} D {D} {kind} wide {wide}")
    c = case(form, D, kind)
    out, lse = c.run(out_dtype=torch.float32 if wide else None)
    check(c, out, lse)
    again, lse2 = c.run(out_dtype=torch.float32 if wide else None)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("D", ODD_DIMS)
@pytest.mark.parametrize("form", FORMS)
def test_odd_heads(form, D, kind):
    note(f"attention4 odd heads {form} D {D} {kind}")
    c = case(form, D, kind, seed=1)
    for causal in (True, False):
        out, lse = c.run(causal)
        check(c, out, lse, causal)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("width", [128, 600])
@pytest.mark.parametrize("form", FORMS)
def test_a_table_wider_than_its_lengths(form, width, kind):
    """What lies behind a sequence's pages is not read; the plan goes by what the table could hold."""
    note(f"attention4 {form}, {width} entries a row, {kind}")
    c = case(form, 128, kind, seed=2)
    tight = c.run(out_dtype=torch.float32)
    c.table = [row + [2 ** 31 - 1] * (width - c.W) for row in c.table]
    c.W = width
    for dtype in (None, torch.float32):
        out, lse = c.run(out_dtype=dtype)
        check(c, out, lse)
    assert bool(((out.double() - tight[0].double()).abs() <= 2 * c.tol).all())


@pytest.mark.parametrize("width", [4, 128])
def test_idle_sequences(width):
    """One prompt in a table with idle rows, alone and among decoding ones."""
    note(f"attention4 idle rows, {width} entries")
    for q, k in (([0] * 20 + [60] + [0] * 43, [0] * 20 + [60] + [30] * 43), ([1, 0] * 10 + [60] + [0, 1] * 10, [33, 0] * 10 + [64] + [0, 7] * 10)):
        c = Case(q, k, 8, 2, 128, "bf16", page=16, seed=width)
        c.table = [row + [2 ** 31 - 1] * (max(width, c.W) - c.W) for row in c.table]
        c.W = max(width, c.W)
        check(c, *c.run())


def test_two_streams_at_once():
    """Calls of different forms that run side by side, each with its own workspace."""
    note("attention4 forms side by side")
    cases = [case(form, 128, "bf16", seed=3) for form in FORMS]
    tables = [(i32(c.table).view(-1, c.W), i32(c.k_len), i32(c.q_start)) for c in cases]
    torch.cuda.synchronize()
    streams, results = [torch.cuda.Stream() for _ in cases], []
    for turn in range(3):
        results.clear()
        for c, t, s in zip(cases, tables, streams):
            with torch.cuda.stream(s):
                lse = torch.empty(c.q.shape[:2], device=c.q.device)
                results.append(bt.attention4(c.q, c.cache, *t, layer=c.layer, lse=lse))
        torch.cuda.synchronize()
        for c, (out, lse) in zip(cases, results):
            check(c, out, lse)
