"""The library is loaded before torch: the process still has one HIP runtime (with two, kernels
launched through one would not know the other's device, streams and memory)."""
import subprocess
import sys

import pytest

from tests.conftest import ROOT

EARLY = """
from log_prob_amd import flce
flce.linear_workspace(4, 64, 64)
import torch
"""
RUNTIMES = """
found = {line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line}
assert len(found) == 1, found
"""
LAUNCH = """
x = torch.ones(4, 64, device="cuda")
assert torch.equal(flce.dropout(x, 0.0, 1), x)
"""


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_one_hip_runtime():
    run(EARLY + RUNTIMES)


@pytest.mark.gpu
def test_a_launch_after_a_query_before_torch():
    run(EARLY + LAUNCH + RUNTIMES)
