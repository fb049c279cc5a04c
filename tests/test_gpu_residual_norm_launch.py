"""Launches of the residual between two norms whose shared memory, factors and
the kernel's own arrays together, passes 48 KB while the factors alone do not:
widths of 3944 to 4096 whose rows take several rounds.  Each type in a process
of its own, where no wider call has come before."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

SCRIPT = """
import sys
sys.path[:0] = [{root!r}, {here!r}]
import torch
import diffusion_transformer_denoising_auraflow_b200 as af
import test_gpu_residual_norm as t
for B, N, D in ((1, 1000, 3944), (1, 400, 4096), (2, 2100, 4096)):
    for post, pre, branch in (("none", "layer", True), ("none", "rms", False)):
        t.test_many_rows(af, B, N, D, torch.{dtype}, {y8}, post, pre, branch)
print("all ran")
"""


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("y8", [False, True])
def test_staged_factors_next_to_48_kb(dtype, y8):
    code = SCRIPT.format(root=os.path.dirname(HERE), here=HERE, dtype=dtype, y8=y8)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "all ran" in r.stdout, r.stderr[-2000:]
