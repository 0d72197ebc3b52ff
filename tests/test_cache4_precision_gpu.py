"""bt_attention4 with bf16 outputs carries probabilities in 16 bits in every form (16, 64 and 128 rows, whole and cut
keys), so that a sequence's precision does not depend on what it is batched with.

Tolerance: that of test_cache4_gpu.py for fp32 outputs, whose probabilities are exact to 2^-24, plus what 16-bit outputs
add: 2^-16 of sum p |v| for two bf16 parts of a probability (8 significant bits each, the rest of the second at most half a
step: 2^-8 * 2^-8), and one rounding of the output, eps / 2 = 2^-8 of its value. Outputs near zero tell the two apart: with
one part alone a probability is off by up to 2^-8, for few keys hundreds of times this bound there."""
import pytest
import torch

from tests import block_ref, cache_ref
from tests.test_cache4_gpu import Case, note, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q,k,heads,kv,D,page", [
    # 16 rows a tile: one part fewer would not show within the tolerance of one
    ([1], [40], 8, 2, 64, 16),
    ([1] * 6, [30, 17, 64, 5, 33, 50], 32, 4, 128, 16),
    ([2], [24], 8, 1, 256, 16),
    ([1, 1], [40, 900], 16, 2, 128, 32),
    # 64 rows
    ([10], [60], 8, 2, 64, 16),
    ([9, 12], [31, 70], 20, 5, 128, 16),
    ([20], [40], 4, 2, 256, 16),
    ([8] * 3, [30, 700, 45], 16, 4, 128, 32),
    # 128 rows
    ([40], [100], 8, 1, 64, 16),
    ([30], [90], 32, 4, 128, 16),
    ([40], [100], 8, 2, 256, 16),
    ([30, 25], [60, 800], 32, 4, 128, 64),
])
def test_probabilities_in_16_bits(q, k, heads, kv, D, page):
    note(f"attention4 precision {q} over {k}, {heads}/{kv} x {D}")
    c = Case(q, k, heads, kv, D, "bf16", page=page, seed=D + len(q))
    out, lse = c.run()
    c.check(out, lse)
    assert out.dtype == torch.bfloat16
    ks, vs, start, _ = cache_ref.gather(c.cache.data[c.layer], c.table, c.k_len, page, kv, D)
    args = (c.q_start, start, c.k_len, True)
    ref, rlse = block_ref.attention(c.q.double(), ks, vs, *args)
    mag, _ = block_ref.attention(c.q.double(), ks, vs.abs(), *args)
    tol, _ = tolerance(c.q, ks, max(k), mag, ref, rlse, torch.float32)
    tol = tol + 2.0 ** -16 * mag + 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8)
    d = (out.double() - ref).abs()
    assert bool((d <= tol).all()), float((d / tol).max())
