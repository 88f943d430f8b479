"""The binding on a torch built without CUDA: it imports, and refuses host tensors."""
from __future__ import annotations

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from w4_gemm_error_b200 import build
build.build(quiet=True)
from w4_gemm_error_b200 import spear
try:
    spear.quantize_q8(torch.zeros(2, 64, dtype=torch.bfloat16))
except ValueError:
    print("refused")
"""


def test_the_binding_imports_without_torchs_private_cuda_functions():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr[-2000:]
