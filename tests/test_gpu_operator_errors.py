"""What a failed call leaves behind: nothing that a later one trips over."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_refused_scratch_leaves_nothing_behind(lib):
    """Scratch beyond the device's memory is refused before any launch; the error is this call's alone."""
    D, T = 3 * 2 ** 21, 2 ** 20   # 8 bytes per feature and 128 columns: 412 GB
    x = torch.zeros(16, device="cuda")
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    code = lib._lib.cr_gated_scan(1, 1, x.data_ptr(), D, x.data_ptr(), D, D, T, None, 1, None, 0, None, 0, None, 0, None,
                                  torch.cuda.current_stream().cuda_stream)
    assert lib.STATUS[code] == "CR_ERR_NOMEM"
    assert torch.cuda.mem_get_info()[0] >= free - 2 ** 28   # nor does the library's pool keep the memory
    y = torch.randn(4, 64, device="cuda").T
    a, _ = lib.rmsnorm(y, torch.ones(64, device="cuda"))   # its own check of the launch finds no error
    assert torch.isfinite(a).all()
    assert float((y + 1).sum()) == float((y + 1).sum())    # nor do PyTorch's


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
