"""One vector per sample given as a [B, D] tensor is read one row per sample:
a mod_stride that says otherwise (0, the default, is one vector for all) is
refused instead of using other rows (no GPU needed)."""
import pytest
import torch

import diffusion_transformer_denoising_auraflow_b200 as af

SHAPE = 2
B, N, D = 3, 4, 16


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def _calls(**kw):
    x = z(B, N, D)
    yield lambda: af.residual_norm(x, z(B, N, D), z(B, N, D), z(B, N, D), 1e-6, **kw)
    yield lambda: af.residual_norm_e4m3(x, z(B, N, D), z(B, N, D), z(B, N, D, dtype=torch.uint8), z(B * N), 1e-6, **kw)


def _reaches_the_tensors(call):
    # sizes and strides pass: what is left to refuse is that these are CPU tensors
    with pytest.raises(TypeError, match="CUDA tensor"):
        call()


@pytest.mark.parametrize("name", ["gate", "shift", "scale"])
def test_rows_not_at_mod_stride_are_refused(name, monkeypatch):
    # CPU tensors would be refused as such first: let sizes be looked at
    monkeypatch.setattr(af, "_dev_rows", lambda t, *a: 0)
    monkeypatch.setattr(af, "_ptr", lambda t, *a: 0)
    monkeypatch.setattr(af, "_on_device", lambda t, *a: 0)
    table = z(B, 3 * D)
    for t, stride in ((z(B, D), 0), (table[:, D:2 * D], 0), (table[:, D:2 * D], D), (z(B, 1, D), 0), (z(B, D), 2 * D)):
        with pytest.raises(af.AFError, match="mod_stride") as e:
            af._residual_norm_args("w", z(B, N, D), z(B, N, D), None, *_three(name, t), stride, 1.0, "none", None, "layer",
                                   None, 0)
        assert e.value.status == SHAPE
    for t, stride in ((z(B, D), D), (table[:, D:2 * D], 3 * D), (table, 0), (z(D), 0), (z(1, D), 0),
                      (z(1, D).expand(B, D), 0), (table.view(-1), 3 * D), (z(B, 1, D), D)):
        af._residual_norm_args("w", z(B, N, D), z(B, N, D), None, *_three(name, t), stride, 1.0, "none", None, "layer",
                               None, 0)


def _three(name, t):
    return tuple(t if n == name else None for n in ("gate", "shift", "scale"))


def test_cpu_tensors_are_still_refused_as_such():
    for call in _calls(gate=z(B, D), mod_stride=D):
        _reaches_the_tensors(call)


@pytest.mark.gpu
def test_refused_on_the_gpu_and_right_with_the_stride():
    x = torch.randn(B, N, D, device="cuda")
    b, g = torch.randn_like(x), torch.randn(B, D, device="cuda")
    xo, y = torch.empty_like(x), torch.empty_like(x)
    with pytest.raises(af.AFError, match="mod_stride"):
        af.residual_norm(x, b, xo, y, 1e-6, gate=g)
    with pytest.raises(af.AFError, match="mod_stride"):
        af.residual_norm_e4m3(x, b, xo, y.to(torch.uint8), torch.empty(B * N, device="cuda"), 1e-6, gate=g)
    af.residual_norm(x, b, xo, y, 1e-6, gate=g, mod_stride=D)
    want = x.double() + g.double()[:, None] * b.double()
    # one product and one sum in fp32
    assert torch.all((xo.double() - want).abs() <= 2.0 ** -23 * (want.abs() + (g[:, None] * b).abs().double()))
    # one vector for all: the same as its expansion, strides 0
    af.residual_norm(x, b, xo, y, 1e-6, gate=g[0])
    x2, y2 = torch.empty_like(x), torch.empty_like(x)
    af.residual_norm(x, b, x2, y2, 1e-6, gate=g[:1].expand(B, D))
    assert torch.equal(xo, x2) and torch.equal(y, y2)
