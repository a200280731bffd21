"""The binding imports, and its host-side calls work, on a torch that was
built without CUDA."""

import os
import subprocess
import sys


def test_import_with_a_torch_built_without_cuda():
    """Such a torch has no torch._C._cuda_* functions."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
from nvfp4_w4a4_quantized_smooth_b200 import svdq
assert svdq.abi_version() == svdq.ABI_VERSION
plan = svdq.RopePlan((16, 24, 24), 256.0, 64)
assert len(plan._turns) == 32
x = torch.zeros(4, 64, dtype=torch.bfloat16)
q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
calls = (lambda: svdq.norm_gate_residual(x, x), lambda: svdq.attention(q, q, q),
         lambda: svdq.rope_qk(q, q, torch.zeros(4, 3, dtype=torch.int32), plan))
for call in calls:
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise AssertionError("taken")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
