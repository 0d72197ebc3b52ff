"""bt_lora_apply with infinities and NaNs in tokens and weights, in every form of the kernels."""
import math

import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests import block_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# tokens, run of tokens on one adapter: at most four of a tile share an adapter (FMA), more do (matrix
# cores), many tokens in runs and in mixed order
FORMS = {"few": (14, 1), "few, shared": (48, 16), "many, runs": (600, 40), "many, mixed": (600, 1)}


@pytest.mark.parametrize("R", [12, 16, 40])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("form", FORMS)
def test_infinities_and_nans_as_the_formula_has_them(form, kind, R):
    """Tokens, A and B with infinities and NaNs, adapters of rank 0, 1, part and all of R: the class of every
    output (finite, inf, -inf, NaN) is the definition's, and the finite ones are within its fp32 sums."""
    M, run = FORMS[form]
    print(f"[gpu-case] lora infinities {form} {kind} R={R}", flush=True)
    K, groups, L = 200, (30, 71), 7
    N = sum(groups)
    g = torch.Generator(device=DEV)
    g.manual_seed(41)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    X, base = rnd(M, K), rnd(M, N)
    A = (rnd(L, 2 * R, K) / K ** 0.5).to(TYPES[kind])
    B = (rnd(L, N, R) / R ** 0.5).to(TYPES[kind])
    scale = torch.rand(L, generator=g, device=DEV) + 0.5
    ranks = torch.tensor([R, 0, 5, 1, R, R, 11], dtype=torch.int32, device=DEV)
    index = (torch.arange(M, device=DEV) // run % (L + 1) - 1).to(torch.int32)
    for m in range(M):
        where = m % 9
        if where == 2:
            X[m, 7 * m % K] = math.inf
        elif where == 5:
            X[m, K - 1] = -math.inf
            X[m, 3] = math.inf
        elif where == 7:
            X[m, 100] = math.nan
    A[4, 2, 50] = math.inf  # one rank of the first group, and nothing of the second
    A[5, R + 1, 199] = math.nan
    B[5, 12, 0] = -math.inf
    B[6, 100, 3] = math.nan
    B[6, 40, 10] = math.inf
    ad = bt.LoraAdapters(A, B, scale, ranks=ranks, group_rows=groups)
    ws = torch.full((max(bt.lora_workspace_bytes(M, ad), 256),), 255, dtype=torch.uint8, device=DEV)  # NaNs
    y = bt.lora_apply(X, ad, index, base=base, workspace=ws)
    ref, mag = block_ref.lora(X, A, B, scale, index, base, ranks, groups)
    for name, test in (("nan", torch.isnan), ("inf", lambda t: t == math.inf), ("-inf", lambda t: t == -math.inf)):
        assert torch.equal(test(y), test(ref)), (name, int((test(y) != test(ref)).sum()))
    fine = torch.isfinite(ref)
    assert bool(fine.any()) and not bool(fine.all())
    # every fp32 sum of n terms is within n * 2^-24 of its terms' magnitude, and one is inside the other
    tol = (K + R + 40) * 2.0 ** -24 * mag + 1e-37
    assert bool(((y.double() - ref).abs() <= tol)[fine].all())
    off = (index < 0) | (ranks[index.clamp(min=0).long()] == 0)
    assert torch.equal(y[off], base[off])  # no adapter, or one of rank 0: the base's row
