"""The 4-bit product on values that leave no room for a tolerance to hide a
lost digit: whole numbers whose result is exact, and rows of x whose largest
value meets a zero weight.

x enters as whole multiples of a power of two per row and 256 columns, at most
2^-30 (1 + 2^-7) of the largest magnitude a there (off by at most half of it),
cut into four signed bytes.  Sums of a group are whole numbers.  In fp32 are
added: the groups of 256 columns (256 / group), two products per byte pair and
256 columns (2 K / 256 at most), the two pairs, the sums of up to 16 warps and the
bias: d = 256 / group + 2 K / 256 + min(16, K / 256) + 3 additions, each off by at
most u = 2^-24 of what is added up.  A byte's value is at most 2.01 |x|
where it is the leading one (a signed byte of |x| below half a unit is 0), 1.01
|x| the next, 2^-8 of that the next: together 3.04 |x|.  So a result is off by
at most
  3.04 d u sum |x w| + (1 + 2^-7) 2^-31 sum a |w|
and half an fp32 step of itself.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def af():
    import diffusion_transformer_denoising_auraflow_b200 as m
    return m


def _pack(c, group):
    """Codes [N, K] as bytes, 8 behind column K."""
    N, K = c.shape
    c = torch.nn.functional.pad(c, (0, -K % group), value=8).to(torch.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def _values(c, scales, group):
    s = scales[:, :c.shape[0]].double().t().repeat_interleave(group, 1)[:, :c.shape[1]]
    return (c.double() - 8) * s


def _plain(x, w):
    return torch.matmul(x.double(), w.t())


def _bound(x, w, K, group, ref):
    ax = x.double().abs()
    top = torch.nn.functional.pad(ax, (0, -K % 256)).view(len(x), -1, 256).amax(-1).repeat_interleave(256, 1)[:, :K]
    chunks = -(-K // 256)
    d = 256 / group + 2 * chunks + min(16, chunks) + 3
    return (3.04 * d * U * ax + (1 + 2.0 ** -7) * 2.0 ** -31 * top) @ w.abs().t() + U * ref.abs()


# rows and columns with the rounds of row blocks and the warps that share a
# row's columns (148 SMs; KW, rounds): one row block and many ways, one way and
# one or several rounds, x too wide for shared memory with one and two rounds
EXACT = [(1, 192, 32, 32), (2, 517, 3072, 64), (2, 18432, 3072, 64), (7, 99, 16384, 32), (3, 33, 2052, 32),
         (2, 160000, 64, 64), (2, 160000, 520, 64), (1, 243000, 768, 128), (8, 60011, 512, 32), (8, 80000, 4096, 64),
         (4, 30007, 8200, 128), (25, 36864, 256, 128), (9, 70, 3072, 64), (16, 20000, 300, 64)]


@pytest.mark.parametrize("M,N,K,group", EXACT)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_whole_numbers_are_exact(af, M, N, K, group, dtype):
    """Pairs of columns with weights w and -w and values q and q + d of 24
    bits (bf16: 8): what is left is -w d summed up, small whole numbers that
    every sum on the way holds exactly."""
    g = torch.Generator(device="cuda").manual_seed(871)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, device="cuda", generator=g)

    half = K // 2
    bits = 24 if dtype == F32 else 8
    # half of the pairs large and equal, the others smaller and d apart
    e = whole(0, 6, M, half)
    q = whole(1 << (bits - 1), (1 << bits) - 4, M, half) * torch.where(whole(0, 2, M, half) > 0, 1, -1)
    d = whole(0, 4, M, half)
    d = torch.where(e > 0, 0, d)
    q = q * 2 ** e
    x = torch.stack([q, q + d], -1).view(M, 2 * half).to(dtype)
    assert torch.equal(x.double().view(M, half, 2)[..., 1].long(), q + d)
    x = torch.nn.functional.pad(x, (0, K - 2 * half))
    w = whole(1, 8, N, half)
    c = torch.stack([8 + w, 8 - w], -1).view(N, 2 * half)
    c = torch.nn.functional.pad(c, (0, K - 2 * half), value=8)
    groups = -(-K // group)
    scales = torch.full((groups, (N + 7) // 8 * 8), float("nan"), dtype=BF, device="cuda")
    scales[:, :N] = (2.0 ** whole(0, 2, groups, N)).to(BF)
    out = torch.full((M + 1, N), 3.0, device="cuda")
    af.linear_w4(x, _pack(c, group), scales, group, out[:M])
    # the pairs' own sum, whole numbers below 2^53
    s = scales[:, :N].double().t().repeat_interleave(group, 1)[:, :2 * half:2]
    want = -(d.double() @ (w.double() * s).t())
    assert want.abs().max() < 2 ** 24
    assert torch.equal(out[:M].double(), want)
    assert torch.all(out[M] == 3.0)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("M,N,K,group,ratio", [(1, 300, 256, 128, 300), (2, 300, 256, 128, 1000), (3, 1000, 256, 64, 1000),
                                               (2, 257, 1024, 128, 1000), (8, 64, 300, 32, 300)])
def test_largest_value_at_a_zero_weight(af, M, N, K, group, ratio, dtype):
    """One value of each 256 columns `ratio` times the rest, with a zero weight in every row."""
    g = torch.Generator(device="cuda").manual_seed(872)
    x = torch.randn(M, K, device="cuda", generator=g)
    c = torch.randint(1, 16, (N, K), device="cuda", generator=g)
    for k in range(0, K, 256):
        at = k + 17 + (k // 256) * 5
        x[:, min(at, K - 1)] = ratio
        c[:, min(at, K - 1)] = 8
    x = x.to(dtype)
    scales = (torch.rand(-(-K // group), (N + 7) // 8 * 8, device="cuda", generator=g) * 0.01 + 0.001).to(BF)
    out = torch.empty(M, N, device="cuda")
    af.linear_w4(x, _pack(c, group), scales, group, out)
    w = _values(c, scales, group)
    ref = _plain(x, w)
    assert torch.all((out.double() - ref).abs() <= _bound(x, w, K, group, ref))


@pytest.mark.parametrize("scale", [2.0 ** -149, 2.0 ** -140, 1e-38, 1e-30, 1.0, 1e30, 1e38])
def test_magnitudes_of_fp32(af, scale):
    """The smallest to the largest x: the bound is relative at any magnitude."""
    g = torch.Generator(device="cuda").manual_seed(873)
    x = (torch.rand(3, 700, device="cuda", generator=g).double() * 3 * scale).float()
    c = torch.randint(1, 16, (40, 700), device="cuda", generator=g)
    # weights that bring the results of the largest and smallest x into range
    up = 2.0 ** (-10 if scale > 1e20 else 60 if scale < 1e-20 else 0)
    scales = torch.full((11, 40), up, dtype=BF, device="cuda")
    out = torch.empty(3, 40, device="cuda")
    af.linear_w4(x, _pack(c, 64), scales, 64, out)
    w = _values(c, scales, 64)
    ref = _plain(x, w)
    # what is added up is at least 2^-149 2^60: no sum is rounded off the fp32 grid
    assert torch.all((out.double() - ref).abs() <= _bound(x, w, 700, 64, ref))


def test_the_bound_shows_a_lost_byte():
    """On the CPU's arithmetic: the same check refuses x held to 24 bits of the largest value."""
    g = torch.Generator().manual_seed(874)
    for K, ratio in ((256, 1000), (1024, 1000)):
        x = torch.randn(2, K, generator=g, dtype=torch.float64)
        w = torch.randint(-7, 8, (300, K), generator=g).double() * 0.005
        x[:, 17::256] = ratio
        w[:, 17::256] = 0.0
        step = ratio * 2.0 ** -23
        ref = _plain(x, w)
        err = (_plain(torch.round(x / step) * step, w) - ref).abs()
        assert torch.any(err > _bound(x, w, K, 128, ref))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_more_rows_than_one_launch_takes(af, dtype):
    """65535 CTAs of eight rows of x, and some rows behind them."""
    g = torch.Generator(device="cuda").manual_seed(875)
    M, N, K = 8 * 65535 + 13, 3, 33
    x = torch.randint(-100, 101, (M, K), device="cuda", generator=g).to(dtype)
    c = torch.randint(0, 16, (N, K), device="cuda", generator=g)
    scales = torch.ones(2, 8, dtype=BF, device="cuda")
    out = torch.full((M + 1, N), 3.0, device="cuda")
    af.linear_w4(x, _pack(c, 32), scales, 32, out[:M])
    assert torch.equal(out[:M].double(), _plain(x, _values(c, scales, 32)))   # whole numbers below 2^24
    assert torch.all(out[M] == 3.0)
