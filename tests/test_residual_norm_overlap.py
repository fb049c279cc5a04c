"""Codes of residual_norm_e4m3 over the rows they come from: refused at the C
entry (no GPU needed), and what lies beside them is no overlap."""
import pytest
import torch

import diffusion_transformer_denoising_auraflow_b200 as af

INVALID = 1
X, B, O, Y, S = ((i + 1) << 24 for i in range(5))  # stand for device addresses; no refused call reads them
ROWS, D = 6, 16


def _call(x=X, b=B, xo=O, y=Y, s=S, dt=0):
    return af.lib.af_residual_norm_e4m3(x, b, dt, 1.0, None, None, None, 0, 0, None, 1, None, xo, y, s, 2, 3, D, 1e-6,
                                        None)


@pytest.mark.parametrize("dt,size", [(0, 2), (1, 4)])
def test_codes_and_scales_over_rows_are_refused(dt, size):
    for t in (X, B, O):
        for at in (t, t + ROWS * D * size - 1, t - ROWS * D + 1):
            assert _call(y=at, dt=dt) == INVALID
        for at in (t, t + ROWS * D * size - 4, t - 4 * ROWS + 4):
            assert _call(s=at, dt=dt) == INVALID
    assert _call(y=S, dt=dt) == INVALID and _call(y=S - ROWS * D + 1, dt=dt) == INVALID
    assert _call(y=B, xo=None, dt=dt) == INVALID and _call(y=X, b=None, dt=dt) == INVALID


@pytest.mark.gpu
def test_codes_beside_the_rows_run():
    """One buffer with x, the codes and the scales next to each other, x' in place of x."""
    g = torch.Generator(device="cuda").manual_seed(11)
    n = ROWS * D
    buf = torch.zeros(n * 3 + 4 * ROWS, dtype=torch.uint8, device="cuda")
    x = buf[:2 * n].view(torch.bfloat16).view(2, 3, D)
    y8, ys = buf[2 * n:3 * n].view(2, 3, D), buf[3 * n:].view(torch.float32)
    src = torch.randn(2, 3, D, device="cuda", generator=g).bfloat16()
    b = torch.randn(2, 3, D, device="cuda", generator=g).bfloat16()
    x.copy_(src)
    af.residual_norm_e4m3(x, b, x, y8, ys, 1e-6, post="rms")
    xo, y2, s2 = torch.empty_like(src), torch.empty(2, 3, D, dtype=torch.uint8, device="cuda"), torch.empty(ROWS, device="cuda")
    af.residual_norm_e4m3(src, b, xo, y2, s2, 1e-6, post="rms")
    assert torch.equal(x, xo) and torch.equal(y8, y2) and torch.equal(ys, s2)
