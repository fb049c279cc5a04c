"""The 4-bit product with rows of x that no single step fits.  Where fewer than
four, or than one in 16, of the values other than zero among 256 columns reach
2^-10 of the largest there, these are added as fp32 terms of their own, up to 32
a row, and the rest enters as whole multiples of a step of at most
2^-30 (1 + 2^-7) of the rest's largest magnitude a; a row with more of them is
summed term by term.  The first adds up to 32 terms to the additions of
test_gpu_w4_exact.py,
  (3.04 (256 / group + 2 K / 256 + min(16, K / 256) + 3) + 64) u sum |x w|
   + (1 + 2^-7) 2^-31 sum a |w|,   u = 2^-24,
the second has 32 additions per 16 bytes of codes and one for each of these, with
a product's rounding each: (K / 32 + 40) u sum |x w|.  Either is allowed, and half an
fp32 step of the result.  SiLU adds two functions good to a few steps, 2^-20 of a
term in all at |x| below 8.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def af():
    import diffusion_transformer_denoising_auraflow_b200 as m
    return m


def _case(M, N, K, group, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, device="cuda", generator=g).to(dtype)
    c = torch.randint(1, 16, (N, K), device="cuda", generator=g)
    scales = (torch.rand(-(-K // group), (N + 7) // 8 * 8, device="cuda", generator=g) * 0.01 + 0.001).to(BF)
    return x, c, scales


def _pack(c, group):
    c = torch.nn.functional.pad(c, (0, -c.shape[1] % group), value=8).to(torch.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def _check(af, x, c, scales, group, silu=False, rest=1e5):
    """The values at `rest` and above are those that are set aside or meet zero weights only."""
    (M, K), N = x.shape, c.shape[0]
    out = torch.full((M + 1, N), 5.0, device="cuda")
    af.linear_w4(x, _pack(c, group), scales, group, out[:M], silu=silu)
    s = scales[:, :N].double().t().repeat_interleave(group, 1)[:, :K]
    w = (c.double() - 8) * s
    fx = x.double() * torch.sigmoid(x.double()) if silu else x.double()
    ref = fx @ w.t()
    ax = fx.abs()
    a = torch.nn.functional.pad(torch.where(ax < rest, ax, 0.0), (0, -K % 256)).view(M, -1, 256).amax(-1)
    a = a.repeat_interleave(256, 1)[:, :K]
    chunks = -(-K // 256)
    d = max(3.04 * (256 / group + 2 * chunks + min(16, chunks) + 3) + 64, K / 32 + 40) * U + (2.0 ** -20 if silu else 0)
    tol = (d * ax + (1 + 2.0 ** -7) * 2.0 ** -31 * a) @ w.abs().t() + U * ref.abs()
    assert torch.all((out[:M].double() - ref).abs() <= tol)
    assert torch.all(out[M] == 5.0)
    return out[:M]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("ratio", [1e6, 1e9, 1e30])
@pytest.mark.parametrize("M,N,K,group", [(1, 1, 256, 128), (2, 300, 256, 64), (5, 257, 300, 32), (3, 1000, 3072, 64),
                                         (9, 64, 2051, 128)])
def test_one_value_far_above_the_rest(af, M, N, K, group, ratio, dtype):
    """... in the first row of x only, at a zero weight in every row of weights."""
    x, c, scales = _case(M, N, K, group, 881, dtype)
    x[0, 7] = -ratio
    c[:, 7] = 8
    _check(af, x, c, scales, group)


@pytest.mark.parametrize("K,step", [(1000, 40), (2051, 65), (2051, 64), (3072, 20), (16384, 600), (40000, 1300)])
@pytest.mark.parametrize("M", [1, 8])
def test_several_values_far_above_the_rest(af, M, K, step):
    """Up to 32 of them in a row and more, of two magnitudes, some in the same 256 columns, at weights other than zero too."""
    x, c, scales = _case(M, 300, K, 64, 882, F32)
    c[:, ::step] = 8
    x[:, ::step] = 1e8
    x[:, 2 * step::4 * step] = -3e12
    a = _check(af, x, c, scales, 64)
    x[:, ::step] = x[:, ::step] * 1e-3
    c[:150, ::step] = 9
    _check(af, x, c, scales, 64, rest=1e4)
    b = torch.empty_like(a)
    for _ in range(3):                # the same bits each time, whatever warp finds them first
        x[:, ::step] = 1e8
        x[:, 2 * step::4 * step] = -3e12
        c[:, ::step] = 8
        af.linear_w4(x, _pack(c, 64), scales, 64, b)
        assert torch.equal(a, b)


def test_repeats_bit_for_bit(af):
    """Terms of their own with weights other than zero: the order of the sum is that of the columns."""
    x, c, scales = _case(8, 2000, 3072, 64, 887, F32)
    at = torch.randperm(3072, device="cuda")[:30]
    x[:, at] = torch.randn(8, 30, device="cuda") * 1e6
    codes = _pack(c, 64)
    a, b = torch.empty(8, 2000, device="cuda"), torch.empty(8, 2000, device="cuda")
    af.linear_w4(x, codes, scales, 64, a)
    for _ in range(20):
        af.linear_w4(x, codes, scales, 64, b)
        assert torch.equal(a, b)


def test_the_other_rows_are_as_without_it(af):
    """A row summed term by term changes no bit of the others."""
    x, c, scales = _case(4, 500, 3072, 64, 883, F32)
    c[:, 5] = 8
    a = _check(af, x, c, scales, 64)
    y = x.clone()
    y[2, 5] = 1e7
    b = _check(af, y, c, scales, 64)
    assert torch.equal(a[[0, 1, 3]], b[[0, 1, 3]])


@pytest.mark.parametrize("M,rows,K", [(2, 160000, 300), (8, 60000, 4200)])
def test_over_several_rounds_of_row_blocks(af, M, rows, K):
    """... with x whole in shared memory, and in parts that are staged again each round."""
    x, c, scales = _case(M, rows, K, 64, 884, F32)
    x[1, 256] = 1e9
    c[:, 256] = 8
    _check(af, x, c, scales, 64)


def test_few_values_and_zeros(af):
    """Rows that are zero but for one or two values, and a row of zeros, are within the bound too."""
    x, c, scales = _case(5, 200, 520, 32, 885, F32)
    x[0] = 0
    x[1] = 0
    x[1, 77] = 3.25
    x[2] = 0
    x[2, 77], x[2, 300] = 1e9, 2.5
    x[3] = 0
    x[3, 77], x[3, 78] = 1e9, 2.3
    c[:, 77] = 8
    out = _check(af, x, c, scales, 32)
    assert torch.all(out[:2] == 0)


def test_silu_of_far_apart_values(af):
    """SiLU of -30 to 8: magnitudes from 1e-12 to 8 in the same columns."""
    g = torch.Generator(device="cuda").manual_seed(886)
    x, c, scales = _case(2, 300, 512, 64, 886, F32)
    x[0] = -5 - 2 * torch.rand(512, device="cuda", generator=g)
    x[0, ::256] = 7.5
    x[1] = 8 * torch.rand(512, device="cuda", generator=g)
    _check(af, x, c, scales, 64, silu=True)
