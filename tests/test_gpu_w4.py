"""GPU parity of 4-bit weights (quantiser, values, product) with the oracle.

The quantiser is a set of whole decisions: scales and codes are compared bit
for bit.  The product's tolerance is elementwise, from the sums themselves:
an fp32 sum of terms t_i whose longest chain has d additions is off by at
most d u sum |t_i|, with u = 2^-23 (a tensor-core addition may truncate
instead of rounding to half a step).  A chain passes at most K / 16 steps of
16 columns, K / 32 groups, 32 partial sums and a few last additions:
d = K / 16 + K / 32 + 48.  x enters as 24-bit fixed point, off by at most half
an fp32 step (2^-24) of the largest magnitude among its 256 columns.  SiLU of
|x| <= 5 adds the errors of exp (2 + 1.2 |x| steps), the sum (1/2) and the
division (2): at most 11 u of a term.  bf16 output adds half a step, 2^-8
relative.
"""
import numpy as np
import pytest
import torch

import oracle as O
import synth
from helpers import to_bf16, to_f32

pytestmark = pytest.mark.gpu
U = 2.0 ** -23
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def af():
    import diffusion_transformer_denoising_auraflow_b200 as m
    return m


def _dev(a, dtype):
    return to_bf16(a) if dtype == BF else to_f32(a)


def _draw(seed, name, shape, std, dtype):
    return synth.normal(seed, name, shape, std, "bf16" if dtype == BF else "f32")


def _pack(codes):
    """Oracle codes [N, padded K] to bytes, low nibble first."""
    return torch.from_numpy((codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)).cuda()


def _scales(s, n):
    out = torch.full((s.shape[0], (n + 7) // 8 * 8), float("nan"), dtype=BF, device="cuda")
    out[:, :n] = to_bf16(s)
    return out


def _tol(x, w, K, silu, out_dtype, ref):
    ax = np.abs(x)
    top = np.pad(ax, ((0, 0), (0, -K % 256))).reshape(len(x), -1, 256).max(-1).repeat(256, 1)[:, :K]
    t = ((K / 16 + K / 32 + 48 + (11 if silu else 0)) * U * ax + 2.0 ** -24 * top) @ np.abs(w).T + 1e-30
    return t + (np.abs(ref) * 2.0 ** -8 if out_dtype == BF else np.abs(ref) * U)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,K,group", [(1, 1, 32), (9, 33, 32), (17, 64, 64), (130, 1003, 128), (37, 3072, 64),
                                       (8, 130, 64), (5, 513, 32), (64, 4096, 128), (3, 200, 128)])
def test_quantize_bit_exact(af, N, K, group, dtype):
    w = _draw(801, f"qw{N}_{K}", (N, K), 0.02, dtype)
    w[N // 2, : min(K, group)] = 0.0            # a group without a value
    if K > 8:
        w[0, :8] = np.array([3.5, -3.5, .25, .75, -.25, 1.25, -1.75, 0.0]) * 2.0 ** -3   # ties
    (cs, ss) = af.w4_shapes(N, K, group)
    codes = torch.full(cs, 255, dtype=torch.uint8, device="cuda")
    scales = torch.full(ss, -1.0, dtype=BF, device="cuda")
    af.quantize_rows_w4(_dev(w, dtype), group, codes, scales)
    rc, rs = O.quantize_rows_w4(w, group)
    assert np.array_equal(scales[:, :N].float().cpu().numpy(), rs)
    assert torch.all(scales[:, N:] == -1.0)      # behind the last row: left as they were
    assert torch.equal(codes, _pack(rc))
    for out_dtype in (F32, BF):
        out = torch.empty(N, K, dtype=out_dtype, device="cuda")
        af.dequantize_rows_w4(codes, scales, group, out)
        v = O.dequantize_rows_w4(rc, rs, group, K)
        v = O.round_bf16(v) if out_dtype == BF else v.astype(np.float32)
        assert np.array_equal(out.float().cpu().numpy(), v)


def test_quantize_borders(af):
    """Values on, just below and just above every border between two codes."""
    rng = np.random.default_rng(802)
    rows = []
    for _ in range(64):
        s = float(O.round_bf16(np.array([abs(rng.normal()) + 0.01]))[0])
        border = np.float32(s) * np.arange(0.5, 7, 1.0, dtype=np.float32)
        r = np.concatenate([border, np.nextafter(border, np.float32(0)), np.nextafter(border, np.float32(99))])
        rows.append(np.concatenate([r, -r[:10], [7 * np.float32(s)]]).astype(np.float32))
    w = np.stack(rows)
    w = np.pad(w, ((0, 0), (0, 32 - w.shape[1]))) if w.shape[1] <= 32 else w[:, -32:]
    cs, ss = af.w4_shapes(64, 32, 32)
    codes, scales = torch.empty(cs, dtype=torch.uint8, device="cuda"), torch.empty(ss, dtype=BF, device="cuda")
    af.quantize_rows_w4(to_f32(w), 32, codes, scales)
    rc, rs = O.quantize_rows_w4(w, 32)
    assert np.array_equal(scales.float().cpu().numpy(), rs)
    assert torch.equal(codes, _pack(rc))


def test_quantize_every_bf16_quotient(af):
    """All 128 bf16 significands as the group's maximum, each with every bf16
    value down to 1/128 of it, both signs: ties and borders bit for bit."""
    top = (1 + np.arange(128) / 128.0)
    vals = np.concatenate([top * 2.0 ** -e for e in range(8)])       # 1024 values in [2^-7, 2)
    rows = []
    for i, a in enumerate(top):
        v = vals[vals <= a] * np.where(np.arange(np.sum(vals <= a)) % 2, -1.0, 1.0)
        v = np.pad(v, (0, -len(v) % 31)).reshape(-1, 31)
        rows.append(np.concatenate([np.full((len(v), 1), a), v], axis=1) * 2.0 ** (i % 40 - 20))
    w = np.concatenate(rows).astype(np.float32)
    N = len(w)
    cs, ss = af.w4_shapes(N, 32, 32)
    codes, scales = torch.empty(cs, dtype=torch.uint8, device="cuda"), torch.empty(ss, dtype=BF, device="cuda")
    rc, rs = O.quantize_rows_w4(w, 32)
    for dtype in (BF, F32):
        af.quantize_rows_w4(_dev(w, dtype), 32, codes, scales)
        assert np.array_equal(scales[:, :N].float().cpu().numpy(), rs)
        assert torch.equal(codes, _pack(rc))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_extreme_scales(af, dtype):
    """Groups from the smallest numbers (no scale, or one of few bits) to the largest."""
    base = synth.normal(803, "ex", (40, 64), 1.0, "bf16" if dtype == BF else "f32")
    w = (base.astype(np.float64) * 2.0 ** np.linspace(-149, 125, 40)[:, None]).astype(np.float32)
    w = synth.bf16_round(w) if dtype == BF else w
    cs, ss = af.w4_shapes(40, 64, 32)
    codes, scales = torch.empty(cs, dtype=torch.uint8, device="cuda"), torch.empty(ss, dtype=BF, device="cuda")
    af.quantize_rows_w4(_dev(w, dtype), 32, codes, scales)
    rc, rs = O.quantize_rows_w4(w, 32)
    assert np.array_equal(scales.double().cpu().numpy(), rs)
    assert torch.equal(codes, _pack(rc))


CASES = [  # M, N, K, group, x, out, silu, bias
    (1, 1, 1, 32, F32, F32, False, False), (1, 192, 32, 32, F32, F32, True, False),
    (2, 192, 32, 64, BF, BF, True, True), (3, 17, 31, 32, BF, F32, False, True),
    (7, 259, 2051, 32, BF, BF, False, True), (8, 100, 257, 64, F32, F32, False, False),
    (9, 1025, 256, 128, BF, F32, False, False), (1, 3000, 3072, 128, BF, BF, False, False),
    (2, 18432, 3072, 64, F32, F32, True, False), (25, 515, 3072, 128, F32, F32, True, True),
    (33, 130, 700, 32, BF, BF, True, False), (64, 96, 1024, 64, F32, BF, False, True),
    (130, 40, 320, 64, BF, F32, False, False), (5, 24, 16384, 32, F32, F32, False, False),
    (2, 16, 65536, 128, BF, F32, False, False), (70, 33, 9000, 32, F32, F32, True, True),
]


@pytest.mark.parametrize("M,N,K,group,xd,od,silu,bias", CASES)
def test_linear_matches_oracle(af, M, N, K, group, xd, od, silu, bias):
    w = synth.normal(811, f"lw{N}_{K}", (N, K), 0.02)
    x = _draw(812, f"lx{M}_{K}", (M, K), 1.0, xd)
    b = synth.normal(813, f"lb{N}", (N,), 0.1, "f32") if bias else None
    c, s = O.quantize_rows_w4(w, group)
    out = torch.full((M + 1, N), 77.0, dtype=od, device="cuda")
    af.linear_w4(_dev(x, xd), _pack(c), _scales(s, N), group, out[:M], silu=silu,
                 bias=None if b is None else to_f32(b))
    ref = O.linear_w4(x, c, s, group, silu, b)
    fx = O.silu(x) if silu else x.astype(np.float64)
    got = out[:M].double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= _tol(fx, O.dequantize_rows_w4(c, s, group, K), K, silu, od, ref))
    assert torch.all(out[M:] == 77.0)


def _small(af, M, N, K, group, seed, xd=F32):
    w = synth.normal(seed, "w", (N, K), 0.02)
    x = _draw(seed + 1, "x", (M, K), 1.0, xd)
    c, s = O.quantize_rows_w4(w, group)
    return x, c, s


def test_linear_on_a_range_of_rows(af):
    """Rows 24..83 of a larger matrix as a matrix of their own; x at an odd address."""
    x, c, s = _small(af, 3, 112, 200, 32, 821)
    codes, scales = _pack(c), _scales(s, 112)
    whole = torch.empty(3, 112, device="cuda")
    part = torch.empty(3, 60, device="cuda")
    xs = torch.empty(3 * 200 + 1, device="cuda")
    xs[1:] = to_f32(x).view(-1)
    af.linear_w4(xs[1:].view(3, 200), codes, scales, 32, whole)
    af.linear_w4(to_f32(x), codes[24:84], scales[:, 24:], 32, part)
    ref = O.linear_w4(x, c, s, 32)
    tol = _tol(x, O.dequantize_rows_w4(c, s, 32, 200), 200, False, F32, ref)
    assert np.all(np.abs(whole.double().cpu().numpy() - ref) <= tol)
    assert np.all(np.abs(part.double().cpu().numpy() - ref[:, 24:84]) <= tol[:, 24:84])


def test_linear_extreme_values(af):
    """Large and tiny x keep their relative error; infinities and NaN stay in their own row of x."""
    x, c, s = _small(af, 4, 40, 96, 32, 831)
    x[1] *= 1e30
    x[2] *= 1e-30
    c[:, 5] = np.maximum(c[:, 5], 9)                    # a positive weight everywhere
    xd = to_f32(x)
    out = torch.empty(4, 40, device="cuda")
    af.linear_w4(xd, _pack(c), _scales(s, 40), 32, out)
    ref = O.linear_w4(x, c, s, 32)
    assert np.all(np.abs(out.double().cpu().numpy() - ref)
                  <= _tol(x, O.dequantize_rows_w4(c, s, 32, 96), 96, False, F32, ref) + 1e-36)
    bad = xd.clone()
    bad[0, 5] = float("inf")
    bad[3, 7] = float("nan")
    out2 = torch.empty(4, 40, device="cuda")
    af.linear_w4(bad, _pack(c), _scales(s, 40), 32, out2)
    assert torch.all(torch.isinf(out2[0]) & (out2[0] > 0)) and torch.all(torch.isnan(out2[3]))
    assert torch.equal(out2[1:3], out[1:3])
    # SiLU of -inf is 0 * inf: NaN as in the formula; of a large negative number: 0
    bad[0, 5] = -1e30
    af.linear_w4(bad, _pack(c), _scales(s, 40), 32, out2, silu=True)
    assert torch.all(torch.isfinite(out2[0]))


@pytest.mark.parametrize("M,N,K", [(2, 700, 3072), (30, 64, 640), (1, 5000, 256)])
def test_linear_repeats_bit_for_bit(af, M, N, K):
    x, c, s = _small(af, M, N, K, 64, 841)
    args = (to_f32(x), _pack(c), _scales(s, N), 64)
    a, b = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    af.linear_w4(*args, a, silu=True)
    for _ in range(3):
        af.linear_w4(*args, b, silu=True)
        assert torch.equal(a, b)


def test_two_streams_and_graphs(af):
    """Two calls at once on two streams; two captured graphs replayed side by
    side with new inputs in the same buffers."""
    x, c, s = _small(af, 2, 2000, 3072, 64, 851)
    codes, scales = _pack(c), _scales(s, 2000)
    xs = [to_f32(x), to_f32(-2 * x)]
    outs = [torch.empty(2, 2000, device="cuda") for _ in range(2)]
    want = []
    for xi in xs:
        o = torch.empty(2, 2000, device="cuda")
        af.linear_w4(xi, codes, scales, 64, o)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for st, xi, o in zip(streams, xs, outs):
            o.zero_()
        torch.cuda.synchronize()
        for st, xi, o in zip(streams, xs, outs):
            af.linear_w4(xi, codes, scales, 64, o, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graphs = []
    for xi, o in zip(xs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            af.linear_w4(xi, codes, scales, 64, o)
        graphs.append(g)
    xs[0].copy_(to_f32(3 * x))
    torch.cuda.synchronize()
    for st, g in zip(streams, graphs):
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    o = torch.empty(2, 2000, device="cuda")
    af.linear_w4(xs[0], codes, scales, 64, o)
    assert torch.equal(outs[0], o) and torch.equal(outs[1], want[1])
