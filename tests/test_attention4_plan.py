"""Every kernel instance of bt_attention4 is run by a case of tests/test_cache4_instances_gpu.py, with its keys whole and cut
into slices. The query makes no device call, so this runs on the CPU."""
import pytest
import torch

import bit_ternary_weight_absmean_amd as bt
from tests import test_cache4_instances_gpu as instances

KINDS = {"bf16": torch.bfloat16, "fp16": torch.float16}


def plan(form, D, kind, wide):
    q, k, group, kv = instances.FORMS[form]
    pages = max(-(-n // 16) for n in k)
    return bt.attention4_plan(sum(q), len(q), group * kv, kv, D, pages, 16, KINDS[kind],
                              torch.float32 if wide else None)


def expected(rows, cut, D, kind, out):
    dp = 64 if D <= 64 else 128 if D <= 128 else 256
    name = f"k_attn4_few<{kind},{dp},{out}>" if rows == 16 else f"k_attn4_tile<{kind},{dp},{out},{rows}>"
    return name + (f" + k_attn4_join<{out}>" if cut else "")


def test_every_instance_has_a_case():
    found = {plan(f, D, kind, wide) for f in instances.FORMS for D in instances.DIMS for kind in KINDS for wide in (0, 1)}
    want = {expected(rows, cut, D, kind, out) for rows in (16, 64, 128) for cut in (0, 1) for D in (64, 128, 256)
            for kind in KINDS for out in (kind, "fp32")}
    assert len(want) == 72 and found == want


@pytest.mark.parametrize("form", instances.FORMS)
def test_a_form_is_what_it_is_called(form):
    rows, cut = form.split()
    for D in instances.DIMS + instances.ODD_DIMS:
        assert plan(form, D, "bf16", False) == expected(int(rows), cut == "cut", D, "bf16", "bf16")


def test_plan_query():
    assert bt.attention4_plan(0, 3, 4, 2, 64, 10, 16) == "" and bt.attention4_plan(3, 0, 4, 2, 64, 10, 16) == ""
    for bad in ((-1, 1, 4, 2, 64, 10, 16), (1, 1, 3, 2, 64, 10, 16), (1, 1, 4, 2, 60, 10, 16), (1, 1, 4, 2, 64, 10, 24)):
        with pytest.raises(bt.BTError):
            bt.attention4_plan(*bad)
    with pytest.raises(bt.BTError):
        bt.attention4_plan(1, 1, 4, 2, 64, 10, 16, torch.float32)
    with pytest.raises(bt.BTError):
        bt.attention4_plan(1, 1, 4, 2, 64, 10, 16, torch.float16, torch.bfloat16)
    for bad in ((torch.float64,), (torch.bfloat16, torch.int8)):
        with pytest.raises(TypeError, match="out_dtype must be"):
            bt.attention4_plan(1, 1, 4, 2, 64, 10, 16, *bad)
    # agrees with the workspace: joined where there is one
    for shape in ((1, 1, 4, 2, 64, 32, 16), (1, 1, 4, 2, 64, 1000, 16), (300, 300, 4, 2, 64, 40, 64), (2048, 1, 20, 5, 128, 512, 64)):
        assert ("join" in bt.attention4_plan(*shape)) == (bt.attention4_workspace_bytes(*shape) > 0)
