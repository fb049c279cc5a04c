"""Refusals of the 4-bit and residual-norm calls (no GPU needed): sizes in the
binding, everything else at the C entries, before anything is launched."""
import ctypes

import pytest
import torch

import diffusion_transformer_denoising_auraflow_b200 as af

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
INVALID, SHAPE, UNSUPPORTED = 1, 2, 3
P = 1 << 20  # stands for a device address; no refused call reads it


def z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def _ok(fn, *a, **k):
    with pytest.raises(TypeError, match="CUDA tensor"):
        fn(*a, **k)


def _bad(status, fn, *a, **k):
    with pytest.raises(af.AFError) as ei:
        fn(*a, **k)
    assert ei.value.status == status


def test_w4_shapes():
    assert af.w4_shapes(5, 100, 32) == ((5, 64), (4, 8))
    assert af.w4_shapes(16, 128, 128) == ((16, 64), (1, 16))
    assert af.w4_shapes(1, 1, 64) == ((1, 32), (1, 8))
    _bad(UNSUPPORTED, af.w4_shapes, 5, 100, 48)


def test_linear_w4_sizes():
    x, codes, scales, out = z(3, 100), z(5, 64, dtype=U8), z(4, 8, dtype=BF), z(3, 5)
    _ok(af.linear_w4, x, codes, scales, 32, out)
    _ok(af.linear_w4, x.to(BF), codes, scales, 32, out, silu=True, bias=z(5))
    _ok(af.linear_w4, x, codes, z(4, 16, dtype=BF)[:, :8], 32, out)      # a range of wider scales
    _bad(SHAPE, af.linear_w4, x, codes, scales, 64, out)
    _bad(SHAPE, af.linear_w4, x, z(5, 63, dtype=U8), scales, 32, out)
    _bad(SHAPE, af.linear_w4, x, codes, z(3, 8, dtype=BF), 32, out)
    _bad(SHAPE, af.linear_w4, x, codes, z(4, 4, dtype=BF), 32, out)
    _bad(SHAPE, af.linear_w4, x, codes, z(8, 4, dtype=BF).t(), 32, out)
    _bad(SHAPE, af.linear_w4, x, codes, scales, 32, z(3, 6))
    _bad(SHAPE, af.linear_w4, x, codes, scales, 32, out, bias=z(6))
    _bad(UNSUPPORTED, af.linear_w4, x, codes, scales, 16, out)
    _bad(UNSUPPORTED, af.linear_w4, x, codes, z(4, 5, dtype=BF), 32, out)  # row stride not a multiple of 8
    with pytest.raises(TypeError):
        af.linear_w4(x.to(torch.float16), codes, scales, 32, out)
    with pytest.raises(TypeError):
        af.linear_w4(x, codes, scales, 32, out.to(torch.float64))


def test_quantize_rows_w4_sizes():
    codes, scales = z(5, 64, dtype=U8), z(4, 8, dtype=BF)
    _ok(af.quantize_rows_w4, z(5, 100), 32, codes, scales)
    _ok(af.dequantize_rows_w4, codes, scales, 32, z(5, 100, dtype=BF))
    _bad(SHAPE, af.quantize_rows_w4, z(5, 130), 32, codes, scales)
    _bad(SHAPE, af.dequantize_rows_w4, codes, scales, 32, z(6, 100))


def test_residual_norm_sizes():
    x, b, y = z(2, 3, 16), z(2, 3, 16), z(2, 3, 16)
    m = z(2, 48)
    _ok(af.residual_norm, x, b, x, y, 1e-6, gate=m[:, :16], shift=m[:, 16:32], scale=m[:, 32:], mod_stride=48)
    _bad(SHAPE, af.residual_norm, x, z(2, 3, 15), x, y, 1e-6)
    _bad(SHAPE, af.residual_norm, x, b, z(2, 4, 16), y, 1e-6)
    _bad(SHAPE, af.residual_norm, x, b, x, z(1, 3, 16), 1e-6)
    _bad(SHAPE, af.residual_norm, x, b, x, y, 1e-6, post_weight=z(15))
    _bad(SHAPE, af.residual_norm, x, b, x, y, 1e-6, pre_weight=z(17))
    _bad(SHAPE, af.residual_norm_e4m3, x, b, x, z(2, 3, 15, dtype=U8), z(6), 1e-6)
    _bad(SHAPE, af.residual_norm_e4m3, x, b, x, z(2, 3, 16, dtype=U8), z(5), 1e-6)
    with pytest.raises(ValueError):
        af.residual_norm(x, b, x, y, 1e-6, post="batch")


def _lin(x=P, xt=0, silu=0, codes=P, scales=P, ss=8, bias=None, out=P, ot=1, M=1, N=8, K=32, g=32):
    return af.lib.af_linear_w4(x, xt, silu, codes, scales, ss, bias, out, ot, M, N, K, g, None)


def test_linear_w4_entry_refuses():
    for k in ("x", "codes", "scales", "out"):
        assert _lin(**{k: None}) == INVALID
    for k in ("M", "N", "K"):
        assert _lin(**{k: 0}) == INVALID and _lin(**{k: -1}) == INVALID
    assert _lin(xt=2) == INVALID and _lin(ot=-1) == INVALID
    assert _lin(ss=7) == INVALID                    # fewer scales than rows
    assert _lin(g=0) == UNSUPPORTED and _lin(g=256) == UNSUPPORTED
    assert _lin(ss=12) == UNSUPPORTED               # not a multiple of 8
    assert _lin(codes=P + 8) == UNSUPPORTED and _lin(scales=P + 2) == UNSUPPORTED
    assert _lin(K=65537) == UNSUPPORTED
    assert _lin(N=(1 << 30) + 8, ss=(1 << 30) + 8) == UNSUPPORTED
    assert _lin(M=655351) == UNSUPPORTED and _lin(M=2**31 - 1) == UNSUPPORTED  # 65535 CTAs of ten rows of x


def test_quantize_entries_refuse():
    q, d = af.lib.af_quantize_rows_w4, af.lib.af_dequantize_rows_w4
    assert q(None, 0, 8, 32, 32, P, P, 8, None) == INVALID
    assert q(P, 3, 8, 32, 32, P, P, 8, None) == INVALID
    assert q(P, 0, 8, 32, 33, P, P, 8, None) == UNSUPPORTED
    assert q(P, 0, 8, 32, 32, P + 1, P, 8, None) == UNSUPPORTED
    assert q(P, 0, 9, 32, 32, P, P, 8, None) == INVALID
    assert d(P, P, 8, 8, 32, 32, None, 0, None) == INVALID
    assert d(P, P, 8, 0, 32, 32, P, 0, None) == INVALID
    assert d(P, P, 8, 8, 32, 16, P, 0, None) == UNSUPPORTED


def _rn(x=P, b=P, dt=0, g=None, sh=None, sc=None, ms=0, post=0, pw=None, pre=1, qw=None, xo=P, y=P, B=1, N=1, D=8,
        eps=1e-6):
    return af.lib.af_residual_norm(x, b, dt, 1.0, g, sh, sc, ms, post, pw, pre, qw, xo, y, B, N, D, eps, None)


def test_residual_norm_entry_refuses():
    assert _rn(x=None) == INVALID and _rn(xo=None, y=None) == INVALID
    assert _rn(dt=2) == INVALID and _rn(ms=-1) == INVALID
    for k in ("B", "N", "D"):
        assert _rn(**{k: 0}) == INVALID
    assert _rn(post=3) == INVALID and _rn(pre=-1) == INVALID
    assert _rn(eps=-1.0) == INVALID and _rn(eps=float("nan")) == INVALID
    # nothing for these to act on
    for kw in (dict(g=P), dict(pw=P), dict(post=2)):
        assert _rn(b=None, **kw) == INVALID
    for kw in (dict(sh=P), dict(sc=P), dict(qw=P)):
        assert _rn(y=None, **kw) == INVALID
    assert _rn(D=16385) == UNSUPPORTED
    assert _rn(B=1 << 16, N=1 << 16) == UNSUPPORTED
    assert _rn(B=2, N=(1 << 29) + 1) == UNSUPPORTED
    e = af.lib.af_residual_norm_e4m3
    assert e(P, P, 0, 1.0, None, None, None, 0, 0, None, 1, None, P, None, P, 1, 1, 8, 1e-6, None) == INVALID
    assert e(P, P, 0, 1.0, None, None, None, 0, 0, None, 1, None, P, P, None, 1, 1, 8, 1e-6, None) == INVALID
