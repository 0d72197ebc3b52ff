"""The package imports, and answers host-only queries, under a torch that was built without a GPU."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)  # such a torch has none of them
import bit_ternary_weight_absmean_amd as bt
assert bt.packed_weight_bytes(64, 64) > 0
assert bt.attention_workspace_bytes(1, 4096, 1, 20, 5, 128) > 0
print(bt.kernel_plan(0, 1, 256, 256))
"""


def test_imports_without_gpu_bindings_in_torch():
    res = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr
    assert res.stdout.strip()
