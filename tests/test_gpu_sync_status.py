"""What sync_status costs a program: one read of an error word for each kind of kernel that may
wait or fail, and none for 8-bit products before the first of them."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
from torch.profiler import ProfilerActivity, profile
import matrix_aware_optimizers_gb300 as mao

def reads():
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        mao.sync_status()
        torch.cuda.synchronize()
    return sum(e.count for e in p.key_averages() if "DtoH" in e.key)

W = torch.randn(64, 64, device="cuda")
mao.apply_update(W, 0.1, U=W.clone())
reads()  # the profiler's first use
print("reads", reads())
x = mao.fp8_quantize(W, "row")
mao.fp8_product(*x, *mao.fp8_quantize(W, "tile"), "nt")
print("reads", reads())
mao.set_wait_limit(0)
mao.fp8_product(*x, *mao.fp8_quantize(W, "tile"), "nt")
try:
    mao.sync_status()
    print("no error")
except mao.MaoError as e:
    print("error", e)
"""


def test_reads_of_error_words(cuda):
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    lines = [ln for ln in r.stdout.splitlines() if ln.startswith(("reads", "error", "no error"))]
    assert lines[:2] == ["reads 3", "reads 4"]
    assert lines[2].startswith("error") and "TIMEOUT" in lines[2]
