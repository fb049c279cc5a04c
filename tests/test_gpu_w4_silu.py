"""SiLU within the 4-bit product.  One column of x is held exactly, so with a
weight of 1 the product is the function itself: x / (1 + exp(-x)) with exp good
to one fp32 step (2^-23 relative), half a step for the sum and half for the
division: 2 steps.  Below -88.7 exp(-x) is past fp32's largest number and the
result 0, where the function is below 4e-37."""
import pytest
import torch

import diffusion_transformer_denoising_auraflow_b200 as af

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F32, BF])
def test_silu_to_two_steps(dtype):
    x = torch.cat([torch.linspace(-88, 88, 20001), torch.linspace(-3, 3, 20001), torch.logspace(-30, 2, 3000),
                   -torch.logspace(-30, 1.9, 3000)]).cuda().to(dtype).view(-1, 1)
    codes = torch.full((3, 16), 0x88, dtype=torch.uint8, device="cuda")
    codes[:, 0] = 0x89
    scales = torch.ones(1, 8, dtype=BF, device="cuda")
    out = torch.empty(len(x), 3, device="cuda")
    af.linear_w4(x, codes, scales, 32, out, silu=True)
    want = x.double() * torch.sigmoid(x.double())
    assert torch.all((out.double() - want).abs() <= 2 * 2.0 ** -23 * want.abs() + 2.0 ** -149)


def test_silu_far_out():
    x = torch.tensor([-88.5, -88.8, -100.0, -1e30, 88.8, 1e30, 3e38], device="cuda").view(-1, 1)
    codes = torch.full((1, 16), 0x88, dtype=torch.uint8, device="cuda")
    codes[:, 0] = 0x89
    scales = torch.ones(1, 8, dtype=BF, device="cuda")
    out = torch.empty(7, 1, device="cuda")
    af.linear_w4(x, codes, scales, 32, out, silu=True)
    want = x.double() * torch.sigmoid(x.double())
    assert torch.all((out.double() - want).abs() <= 4e-37 + 2.0 ** -22 * want.abs())
    assert torch.equal(out[4:], x[4:])
