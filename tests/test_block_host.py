"""The decode-step binding on a machine or a torch build without CUDA (no GPU)."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_on_a_torch_without_cuda():
    """The import works, tensors that are not on a GPU are refused as such."""
    pytest.importorskip("torch")
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from calibration_free_sparse_gb300 import block
h = torch.zeros(4, 64)
for bad in (h, 3):
    try:
        block.residual_norm(bad, h)
    except TypeError as e:
        assert "CUDA tensor" in str(e)
    else:
        raise SystemExit("not refused")
try:
    block._current(0)
except RuntimeError as e:
    assert "no CUDA" in str(e)
    print("fine")
"""
    got = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert got.returncode == 0 and got.stdout.strip() == "fine", got.stderr
