"""What a failed call leaves behind: nothing that a later one trips over."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu


FIRST_IN_A_CAPTURE = """
import torch
import mixed_precision_dense_mat_gb300 as cr
x, g = torch.randn(4, 64, device="cuda").T, torch.ones(64, device="cuda")
cr.load()
graph = torch.cuda.CUDAGraph()
first = None
try:
    with torch.cuda.graph(graph):
        try:
            cr.rmsnorm(x, g)
        except cr.CrError as e:
            first = e
except RuntimeError:   # the capture ends invalid
    pass
y, _ = cr.rmsnorm(x, g)
torch.cuda.synchronize()
assert torch.isfinite(y).all()
print("first call in the capture:", first and first.name)
"""


def test_a_first_call_inside_a_capture_spoils_no_later_one(lib):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_IN_A_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
