"""GPU parity of the residual between two norms with the oracle, and a run of
it together with the 4-bit modulations.

Tolerances are elementwise, from the formula.  A row sum over D terms passes
at most D / 256 + 24 additions (256 threads at least, or 32 with D at most
4096: 4096 / 32 = 128; taken together d = 160), each off by at most half an
fp32 step, u = 2^-24, of the sum of magnitudes; the root and the products add
a few u.  With c = (d + 24) u and v the normed vector, rstd its factor:
  |error of n(v)| <= c (|n(v)| + rstd mean|v|) + rstd (error of v + its mean)
                     + |n(v)| rstd (root mean square of v's error).
Storage adds half a step: 2^-8 relative in bf16, u in fp32; e4m3 codes 2^-4
relative or half the subnormal step 2^-10, in units of the row scale.
"""
import numpy as np
import pytest
import torch

import oracle as O
import synth
from helpers import e4m3_lut, to_bf16, to_f32

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
C = (160 + 24) * U
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32
STEP = {BF: 2.0 ** -8, F32: U}
LUT = e4m3_lut()


@pytest.fixture(scope="module")
def af():
    import diffusion_transformer_denoising_auraflow_b200 as m
    return m


def _dev(a, dtype):
    return to_bf16(a) if dtype == BF else to_f32(a)


def _norm_err(v, kind, ev):
    """Bound of the error of norm(v) when v itself is off by ev."""
    if kind == "none":
        return ev
    m = v.mean(-1, keepdims=True) if kind == "layer" else 0.0
    rstd = 1 / np.sqrt(((v - m) ** 2).mean(-1, keepdims=True) + EPS)
    n = np.abs((v - m) * rstd)
    return (C * (n + rstd * np.abs(v).mean(-1, keepdims=True)) + rstd * (ev + ev.mean(-1, keepdims=True))
            + n * rstd * np.sqrt((ev ** 2).mean(-1, keepdims=True)))


def _bounds(x, branch, gate, shift, scale, r, post, post_w, pre, pre_w):
    """Error bounds of x' and y before they are stored."""
    xo, y = O.residual_norm(x, branch, EPS, gate, shift, scale, r, post, post_w, pre, pre_w)
    e = np.zeros_like(xo)
    if branch is not None:
        u = O.norm(branch, post, EPS)
        f = np.abs(r) * (1.0 if post_w is None else np.abs(post_w)) * (1.0 if gate is None else np.abs(gate)[:, None])
        e = f * (_norm_err(np.asarray(branch, np.float64), post, np.zeros_like(xo)) + 4 * U * np.abs(u)) + U * np.abs(xo)
    n = O.norm(xo, pre, EPS)
    f = (1.0 if pre_w is None else np.abs(pre_w)) * (1.0 if scale is None else np.abs(1 + scale)[:, None])
    ey = f * (_norm_err(xo, pre, e) + 4 * U * np.abs(n)) + 2 * U * (np.abs(y) + np.abs(f * n))
    return xo, y, e, ey


def _inputs(B, N, D, dtype, seed, branch=True):
    d = "bf16" if dtype == BF else "f32"
    x = (synth.normal(seed, f"x{D}", (B, N, D), 2.0, d) + np.float32(0.5)).astype(np.float32)
    x = synth.bf16_round(x) if dtype == BF else x
    b = synth.normal(seed, f"b{D}", (B, N, D), 1.0, d) if branch else None
    table = synth.normal(seed, f"t{D}", (B, 3 * D), 0.5, "f32")
    pw = synth.normal(seed, f"p{D}", (D,), 0.2, "f32") + 1
    qw = synth.normal(seed, f"q{D}", (D,), 0.2, "f32") + 1
    return x, b, table, pw, qw


def _f64(a):
    return None if a is None else a.astype(np.float64)


SHAPES = [(1, 1, 1), (1, 1, 3072), (2, 5, 32), (3, 7, 1001), (2, 37, 3072), (1, 9, 256), (2, 3, 4104), (1, 2, 16384),
          (1, 3, 9999), (2, 300, 3072), (4, 33, 8), (1, 600, 512), (2, 150, 2048), (1, 260, 4096), (1, 40, 8192)]
KINDS = [("none", "layer", True, True, False, False, 1.0), ("rms", "rms", False, False, True, True, 0.5),
         ("layer", "rms", True, True, True, True, 0.7), ("rms", "none", True, False, False, False, 1.0),
         ("none", "none", False, True, False, True, -2.0), ("layer", "layer", True, False, True, False, 0.125)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,N,D", SHAPES)
@pytest.mark.parametrize("post,pre,gate,mod,pw,qw,r", KINDS)
def test_matches_oracle(af, B, N, D, dtype, post, pre, gate, mod, pw, qw, r):
    x, b, table, pwv, qwv = _inputs(B, N, D, dtype, 901)
    g, sh, sc = table[:, :D], table[:, D:2 * D], table[:, 2 * D:]
    t = to_f32(table)
    xo = torch.empty(B, N, D, dtype=dtype, device="cuda")
    y = torch.empty_like(xo)
    kw = dict(gate=t[:, :D] if gate else None, shift=t[:, D:2 * D] if mod else None,
              scale=t[:, 2 * D:] if mod else None, mod_stride=3 * D, residual_scale=r, post=post,
              post_weight=to_f32(pwv) if pw else None, pre=pre, pre_weight=to_f32(qwv) if qw else None)
    af.residual_norm(_dev(x, dtype), _dev(b, dtype), xo, y, EPS, **kw)
    rx, ry, ex, ey = _bounds(_f64(x), _f64(b), g if gate else None, sh if mod else None, sc if mod else None,
                             float(np.float32(r)), post, pwv if pw else None, pre, qwv if qw else None)
    gx, gy = xo.double().cpu().numpy(), y.double().cpu().numpy()
    assert np.all(np.abs(gx - rx) <= ex + (np.abs(rx) + ex) * STEP[dtype] + 1e-38)
    assert np.all(np.abs(gy - ry) <= ey + (np.abs(ry) + ey) * STEP[dtype] + 1e-38)
    # 8-bit output of the same y
    x2 = torch.empty_like(xo)
    y8 = torch.empty(B, N, D, dtype=torch.uint8, device="cuda")
    ys = torch.empty(B * N, device="cuda")
    af.residual_norm_e4m3(_dev(x, dtype), _dev(b, dtype), x2, y8, ys, EPS, **kw)
    assert torch.equal(x2, xo)
    s = ys.double().cpu().numpy().reshape(B, N, 1)
    amax = np.abs(ry).max(-1, keepdims=True)
    # the scale is amax / 448; 1 for a row of zeros
    assert np.all((np.abs(s * 448 - amax) <= ey.max(-1, keepdims=True) + 4 * U * amax) | ((amax == 0) & (s == 1)))
    v = LUT[y8.cpu().numpy().astype(np.int64)] * s
    assert np.all(np.abs(v - ry) <= ey + (np.abs(ry) + ey) * 2.0 ** -4 * (1 + 1e-5) + s * 2.0 ** -10)


@pytest.mark.parametrize("dtype,y8", [(BF, False), (BF, True), (F32, False)])
@pytest.mark.parametrize("B,N,D", [(2, 4360, 3072), (1, 3001, 1024), (3, 1100, 2048), (1, 2500, 4104), (1, 2100, 8192),
                                   (1, 20001, 256), (1, 60007, 32), (5, 1000, 520), (1, 1300, 16384), (1, 9001, 40),
                                   (3, 5001, 7), (1, 3000, 513), (2, 900, 1023), (1, 1200, 3001), (1, 40000, 13),
                                   (2, 7000, 101), (1, 70001, 1), (1, 5000, 250), (1, 2400, 3999), (1, 700, 16001),
                                   (1, 299, 3072), (1, 601, 3072), (2, 493, 3072), (2, 494, 3072), (1, 2401, 1024),
                                   (1, 370, 8192), (1, 371, 8192), (3, 247, 12288)])
@pytest.mark.parametrize("post,pre,branch", [("none", "layer", True), ("layer", "rms", True), ("none", "rms", False)])
def test_many_rows(af, B, N, D, dtype, y8, post, pre, branch):
    """Row counts at which a CTA takes several rounds of rows (more than twice
    what 148 SMs hold at once, or about as many as they hold of the widest
    row groups), against the formula in fp64 on the device."""
    g = torch.Generator(device="cuda").manual_seed(981)
    x = (torch.randn(B, N, D, device="cuda", generator=g) * 2 + 0.5).to(dtype)
    b = torch.randn(B, N, D, device="cuda", generator=g).to(dtype) if branch else None
    t = torch.randn(B, 3 * D, device="cuda", generator=g) * 0.5
    pw = torch.randn(D, device="cuda", generator=g) * 0.2 + 1
    full = torch.full((B * N + 1, D), 3.0, dtype=torch.uint8 if y8 else dtype, device="cuda")
    y, xo = full[:-1].view(B, N, D), torch.empty_like(x)
    kw = dict(shift=t[:, D:], scale=t[:, 2 * D:], mod_stride=3 * D, pre=pre, residual_scale=0.7)
    if branch:
        kw.update(gate=t, post=post, post_weight=pw)
    ys = torch.empty(B * N, device="cuda")
    if y8:
        af.residual_norm_e4m3(x, b, xo, y, ys, EPS, **kw)
    else:
        af.residual_norm(x, b, xo, y, EPS, **kw)

    def norm(v, kind):
        if kind == "layer":
            v = v - v.mean(-1, keepdim=True)
        return v if kind == "none" else v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)

    rx = x.double()
    if branch:
        rx = rx + float(np.float32(0.7)) * t[:, None, :D].double() * norm(b.double(), post) * pw.double()
    n = norm(rx, pre)
    f = 1 + t[:, None, 2 * D:].double()
    ry = n * f + t[:, None, D:2 * D].double()
    # the bounds of _norm_err with the row's largest values in the place of each value's own
    big = rx.abs().amax(-1, keepdim=True)
    nb = n.abs().amax(-1, keepdim=True)
    ex = (3 * C if branch else 0.0) * (big + 1)
    ey = f.abs() * (2 * C * (nb + 1) + 3 * ex * nb) + 4 * U * ry.abs()
    assert torch.all((xo.double() - rx).abs() <= ex + (rx.abs() + ex) * STEP[dtype])
    if y8:
        v = y.view(torch.float8_e4m3fn).double() * ys.double().view(B, N, 1)
        assert torch.all((v - ry).abs() <= ey + (ry.abs() + ey) * 2.0 ** -4 * (1 + 1e-5) + ys.view(B, N, 1) * 2.0 ** -10)
    else:
        assert torch.all((y.double() - ry).abs() <= ey + (ry.abs() + ey) * STEP[dtype])
    assert torch.all(full[-1].float() == 3.0)


@pytest.mark.parametrize("D", [3072, 77, 2048])
def test_without_branch_or_outputs(af, D):
    x, b, table, pw, qw = _inputs(2, 6, D, BF, 911)
    t = to_f32(table)
    xd, bd = to_bf16(x), to_bf16(b)
    y, xo, y2, xo2 = (torch.empty(2, 6, D, dtype=BF, device="cuda") for _ in range(4))
    # only the norm; with x' stored it is x
    af.residual_norm(xd, None, None, y, EPS, shift=t[:, D:], scale=t[:, 2 * D:], mod_stride=3 * D, pre="layer")
    af.residual_norm(xd, None, xo, y2, EPS, shift=t[:, D:], scale=t[:, 2 * D:], mod_stride=3 * D, pre="layer")
    assert torch.equal(xo, xd) and torch.equal(y, y2)
    rx, ry, ex, ey = _bounds(_f64(x), None, None, table[:, D:2 * D], table[:, 2 * D:], 1.0, "none", None, "layer", None)
    assert np.all(np.abs(y.double().cpu().numpy() - ry) <= ey + (np.abs(ry) + ey) * 2.0 ** -8)
    # only the residual
    af.residual_norm(xd, bd, xo, None, EPS, gate=t, mod_stride=3 * D, post="rms")
    af.residual_norm(xd, bd, xo2, y2, EPS, gate=t, mod_stride=3 * D, post="rms")
    assert torch.equal(xo, xo2)
    # the norm alone of the sum
    af.residual_norm(xd, bd, None, y, EPS, gate=t, mod_stride=3 * D, post="rms")
    assert torch.equal(y, y2)


@pytest.mark.parametrize("D,dtype", [(3072, BF), (1001, F32), (512, F32), (30, BF)])
def test_in_place(af, D, dtype):
    x, b, table, pw, _ = _inputs(2, 40, D, dtype, 921)
    t = to_f32(table)
    kw = dict(gate=t, shift=t[:, D:], scale=t[:, 2 * D:], mod_stride=3 * D, post="layer", post_weight=to_f32(pw))
    xd, bd = _dev(x, dtype), _dev(b, dtype)
    xo, y = torch.empty_like(xd), torch.empty_like(xd)
    af.residual_norm(xd, bd, xo, y, EPS, **kw)
    xi, bi = xd.clone(), bd.clone()
    af.residual_norm(xi, bi, xi, bi, EPS, **kw)
    assert torch.equal(xi, xo) and torch.equal(bi, y)
    xi = xd.clone()
    af.residual_norm(xi, bd, None, xi, EPS, **kw)
    assert torch.equal(xi, y)


@pytest.mark.parametrize("N,D,dtype", [(4400, 3072, BF), (6000, 1001, BF), (5000, 1014, F32), (30000, 45, BF),
                                       (9000, 1024, BF)])
def test_in_place_many_rows(af, N, D, dtype):
    """Rows are read ahead of the ones being written, and odd widths share
    vectors with their neighbours: in place must not change a bit."""
    g = torch.Generator(device="cuda").manual_seed(922)
    x = torch.randn(2, N, D, device="cuda", generator=g).to(dtype)
    b = torch.randn(2, N, D, device="cuda", generator=g).to(dtype)
    t = torch.randn(2, 3 * D, device="cuda", generator=g)
    kw = dict(gate=t, shift=t[:, D:], scale=t[:, 2 * D:], mod_stride=3 * D, post="rms", pre="layer")
    xo, y = torch.empty_like(x), torch.empty_like(x)
    af.residual_norm(x, b, xo, y, EPS, **kw)
    xi, bi = x.clone(), b.clone()
    af.residual_norm(xi, bi, xi, bi, EPS, **kw)
    assert torch.equal(xi, xo) and torch.equal(bi, y)
    xi = x.clone()
    af.residual_norm(xi, b, None, xi, EPS, **kw)
    assert torch.equal(xi, y)


@pytest.mark.parametrize("D,dtype", [(3072, BF), (512, BF), (256, F32)])
def test_odd_addresses_and_one_vector_for_all(af, D, dtype):
    """Tensors off 16-byte boundaries, an odd mod_stride, and mod_stride 0."""
    B, N = 3, 11
    x, b, table, _, _ = _inputs(B, N, D, dtype, 931)

    def shifted(a, dt):
        flat = torch.empty(a.size + 1, dtype=dt, device="cuda")
        flat[1:] = _dev(a, dt).view(-1)
        return flat[1:].view(*a.shape)

    stride = 3 * D + 1
    t = torch.zeros(B * stride + 1, device="cuda")
    tv = t[1:].view(B, stride)
    tv[:, :3 * D] = to_f32(table)
    for off in (False, True):
        xd, bd = (shifted(x, dtype), shifted(b, dtype)) if off else (_dev(x, dtype), _dev(b, dtype))
        xo = shifted(x, dtype) if off else torch.empty_like(xd)
        y = shifted(x, dtype) if off else torch.empty_like(xd)
        for ms, tab in ((stride, table), (0, np.repeat(table[:1], B, 0))):
            af.residual_norm(xd, bd, xo, y, EPS, gate=tv, shift=tv[:, D:], scale=tv[:, 2 * D:], mod_stride=ms, post="rms")
            rx, ry, ex, ey = _bounds(_f64(x), _f64(b), tab[:, :D], tab[:, D:2 * D], tab[:, 2 * D:], 1.0, "rms", None,
                                     "layer", None)
            assert np.all(np.abs(xo.double().cpu().numpy() - rx) <= ex + (np.abs(rx) + ex) * STEP[dtype])
            assert np.all(np.abs(y.double().cpu().numpy() - ry) <= ey + (np.abs(ry) + ey) * STEP[dtype])


@pytest.mark.parametrize("D", [3072, 640, 100])
def test_special_rows(af, D):
    """Zero and constant rows; NaN and infinities stay in their row; rows behind the tensor untouched."""
    x, b, table, _, _ = _inputs(1, 12, D, BF, 941)
    x[0, 0] = 0.0
    b[0, 0] = 0.0
    x[0, 1] = 3.0
    b[0, 1] = -1.0
    xd, bd = to_bf16(x), to_bf16(b)
    out = torch.full((2, 13, D), 5.0, dtype=BF, device="cuda")
    xo, y = out[0, :12].unsqueeze(0), out[1, :12].unsqueeze(0)
    af.residual_norm(xd, bd, xo, y, EPS, post="layer", pre="layer")
    assert torch.all(out[:, 12] == 5.0)
    assert torch.all(y[0, 0] == 0) and torch.all(xo[0, 0] == 0)
    assert torch.all(xo[0, 1] == 3.0) and torch.all(y[0, 1] == 0)
    xb, bb = xd.clone(), bd.clone()
    xb[0, 2, 3] = float("nan")
    bb[0, 3, 4] = float("inf")
    xo2, y2 = torch.empty_like(xd), torch.empty_like(xd)
    af.residual_norm(xb, bb, xo2, y2, EPS, post="layer", pre="layer")
    keep = [i for i in range(12) if i not in (2, 3)]
    assert torch.equal(xo2[:, keep], xo[:, keep]) and torch.equal(y2[:, keep], y[:, keep])
    assert torch.all(torch.isnan(y2[0, 2])) and torch.all(torch.isnan(y2[0, 3]))
    y8, ys = torch.empty(1, 12, D, dtype=torch.uint8, device="cuda"), torch.empty(12, device="cuda")
    af.residual_norm_e4m3(xd, bd, None, y8, ys, EPS, post="layer", pre="layer")
    assert torch.all(y8[0, 0] == 0) and ys[0] == 1.0


def test_close_to_the_two_calls_it_fuses(af):
    """With no post norm, x' equals the residual in torch fp32 and y is
    af_ln_modulate of it up to the rounding of x' (half a bf16 step of x',
    times rstd (1 + scale), with mean and root moving by less)."""
    x, b, table, _, _ = _inputs(2, 50, 3072, BF, 951)
    t = to_f32(table)
    xd, bd = to_bf16(x), to_bf16(b)
    xo, y, y2 = (torch.empty_like(xd) for _ in range(3))
    af.residual_norm(xd, bd, xo, y, EPS, gate=t, shift=t[:, 3072:], scale=t[:, 6144:], mod_stride=9216)
    af.ln_modulate(xo, t[:, 3072:], t[:, 6144:], 9216, y2, EPS)
    want = torch.addcmul(xd.float(), t[:, None, :3072], bd.float()).to(BF)
    assert (xo != want).float().mean() < 1e-3        # fused or separate rounding of the product, at a border
    rstd = 1 / xo.float().std(-1, keepdim=True)
    tol = 2 * 2.0 ** -8 * (xo.float().abs() + xo.float().abs().amax(-1, keepdim=True) / 8) * rstd * \
        (1 + t[:, None, 6144:]).abs() + 2 * 2.0 ** -8 * y.float().abs()
    assert torch.all((y.float() - y2.float()).abs() <= tol)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_adaln_unit_with_4_bit_modulations(af, dtype):
    """The two operators as a block uses them: six modulation vectors from
    4-bit weights and silu(temb), then norm, sub-block (a fixed branch here),
    gated residual and norm, then the second gate; one captured graph."""
    B, N, D, G = 2, 21, 256, 64
    w = synth.normal(961, "ada", (6 * D, D), 0.05)
    temb = synth.conditioning(962, (B, D))
    x, b1, _, _, _ = _inputs(B, N, D, dtype, 963)
    b2 = synth.normal(964, "b2", (B, N, D), 1.0, "bf16" if dtype == BF else "f32")
    (cs, ss) = af.w4_shapes(6 * D, D, G)
    codes, scales = torch.empty(cs, dtype=torch.uint8, device="cuda"), torch.empty(ss, dtype=BF, device="cuda")
    af.quantize_rows_w4(to_bf16(w), G, codes, scales)
    t, m = to_f32(temb), torch.empty(B, 6 * D, device="cuda")
    xd, b1d, b2d = _dev(x, dtype), _dev(b1, dtype), _dev(b2, dtype)
    y0, x1, y1, x2 = (torch.empty_like(xd) for _ in range(4))

    def unit():
        af.linear_w4(t, codes, scales, G, m, silu=True)
        c = [m[:, i * D:] for i in range(6)]
        af.residual_norm(xd, None, None, y0, EPS, shift=c[0], scale=c[1], mod_stride=6 * D)
        af.residual_norm(xd, b1d, x1, y1, EPS, gate=c[2], shift=c[3], scale=c[4], mod_stride=6 * D)
        af.residual_norm(x1, b2d, x2, None, EPS, gate=c[5], mod_stride=6 * D)

    unit()
    eager = [v.clone() for v in (m, y0, x1, y1, x2)]
    rc, rs = O.quantize_rows_w4(w, G)
    rm = O.linear_w4(temb, rc, rs, G, True)
    a = np.abs(O.silu(temb)) @ np.abs(O.dequantize_rows_w4(rc, rs, G, D)).T
    em = (D / 16 + D / 32 + 59) * 2.0 ** -23 * a  # as in test_gpu_w4.py
    gm = m.double().cpu().numpy()
    assert np.all(np.abs(gm - rm) <= em)
    # the rest from the modulations as computed
    c = [gm[:, i * D:(i + 1) * D] for i in range(6)]
    _, ry0, _, ey0 = _bounds(_f64(x), None, None, c[0], c[1], 1.0, "none", None, "layer", None)
    rx1, ry1, ex1, ey1 = _bounds(_f64(x), _f64(b1), c[2], c[3], c[4], 1.0, "none", None, "layer", None)
    gx1 = x1.double().cpu().numpy()
    rx2, _, ex2, _ = _bounds(gx1, _f64(b2), c[5], None, None, 1.0, "none", None, "none", None)
    for got, ref, e in ((y0, ry0, ey0), (x1, rx1, ex1), (y1, ry1, ey1), (x2, rx2, ex2)):
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= e + (np.abs(ref) + e) * STEP[dtype])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        unit()
    for v in (m, y0, x1, y1, x2):
        v.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((m, y0, x1, y1, x2), eager))


def test_two_streams(af):
    x, b, table, _, _ = _inputs(2, 400, 3072, BF, 971)
    t = to_f32(table)
    xd, bd = to_bf16(x), to_bf16(b)
    outs = [torch.empty_like(xd) for _ in range(4)]
    want = torch.empty_like(xd), torch.empty_like(xd)
    kw = dict(gate=t, shift=t[:, 3072:], scale=t[:, 6144:], mod_stride=9216, post="rms")
    af.residual_norm(xd, bd, want[0], want[1], EPS, **kw)
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for i, st in enumerate(ss):
            af.residual_norm(xd, bd, outs[2 * i], outs[2 * i + 1], EPS, stream=st, **kw)
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[2 * i], want[0]) and torch.equal(outs[2 * i + 1], want[1])
            outs[2 * i].zero_()
            outs[2 * i + 1].zero_()
        torch.cuda.synchronize()
