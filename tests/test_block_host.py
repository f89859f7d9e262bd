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


FAKE = 1 << 24      # aligned addresses that are never dereferenced
NORM = ("h", "y", "gate", "post", "pre", "h_out", "x", "hs", "ys", "os", "xs", "grow", "gcol",
        "rows", "hidden", "ht", "yt", "xt", "gt", "wt", "scale", "eps")


@pytest.mark.parametrize("over", [
    # rows of an output that overlap one another
    dict(xs=0), dict(xs=248), dict(xs=-248), dict(os=0, h_out=4 * FAKE), dict(h_out=FAKE, hs=0, os=0),
    # an output over the gate or a weight, wholly or in part
    dict(gate=3 * FAKE, gcol=1, grow=256), dict(gate=3 * FAKE + 7 * 1024 + 512, gcol=1),
    dict(gate=3 * FAKE + 512, grow=1), dict(post=3 * FAKE + 4096), dict(pre=3 * FAKE + 7 * 1024 + 1008),
    dict(h_out=4 * FAKE, pre=4 * FAKE - 512), dict(h_out=4 * FAKE, gate=4 * FAKE + 4),
    dict(h_out=4 * FAKE, gate=4 * FAKE - 4096, gcol=1, grow=256),
    # column slices that run into one another
    dict(hs=512, xs=512, x=FAKE + 512), dict(hs=512, xs=512, x=FAKE + 1536),
    dict(ys=512, os=512, h_out=2 * FAKE + 1008)])
def test_residual_norm_refuses_outputs_that_overlap(over):
    """Argument errors that return before any device work."""
    pytest.importorskip("torch")
    from calibration_free_sparse_gb300 import block, build, reader
    build.build()
    a = dict(h=FAKE, y=2 * FAKE, gate=0, post=0, pre=0, h_out=0, x=3 * FAKE, hs=256, ys=256, os=256,
             xs=256, grow=0, gcol=0, rows=8, hidden=256, ht=0, yt=0, xt=0, gt=0, wt=0, scale=1.0,
             eps=1e-6)
    a.update(over)
    call = reader.library().moe_reader_residual_norm
    assert call(block._NORM.pack(*(a[n] for n in NORM)), None) == reader.EINVAL
