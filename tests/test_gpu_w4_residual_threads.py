"""The first calls of a process from several host threads at once, each on a stream of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

SCRIPT = """
import sys, threading
sys.path.insert(0, {root!r})
import torch
import diffusion_transformer_denoising_auraflow_b200 as af
BF, N, K, D = torch.bfloat16, 600, 1024, 4096
g = torch.Generator(device="cuda").manual_seed(5)
w = torch.randn(N, K, device="cuda", generator=g)
x = torch.randn(2, K, device="cuda", generator=g)
rows = torch.randn(1, 700, D, device="cuda", generator=g).to(BF)
outs, errors, barrier = [None] * 8, [], threading.Barrier(8)
torch.cuda.synchronize()

def work(i):
    try:
        cs, ss = af.w4_shapes(N, K, 64)
        codes, scales = torch.zeros(cs, dtype=torch.uint8, device="cuda"), torch.zeros(ss, dtype=BF, device="cuda")
        out, xo, y = torch.empty(2, N, device="cuda"), torch.empty_like(rows), torch.empty_like(rows)
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        barrier.wait()
        for k in range(3):
            af.quantize_rows_w4(w, 64, codes, scales, stream=st)
            af.linear_w4(x, codes, scales, 64, out, stream=st)
            af.residual_norm(rows, rows, xo, y, 1e-6, post="rms" if i & 1 else "none", stream=st)
        st.synchronize()
        outs[i] = (out, xo, y)
    except Exception as e:
        errors.append(e)

threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not errors, errors
for i in range(8):
    assert all(torch.equal(a, b) for a, b in zip(outs[i], outs[i & 1]))
assert torch.equal(outs[0][0], outs[1][0]) and torch.isfinite(outs[0][0]).all()
print("all equal")
"""


def test_first_calls_from_threads():
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=os.path.dirname(HERE))], capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and "all equal" in r.stdout, r.stderr[-2000:]
