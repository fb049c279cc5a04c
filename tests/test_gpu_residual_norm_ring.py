"""Rows that stream through shared memory with one warp per row: the copy of a
later row goes to a place that all lanes have read.  Many rows of one width,
called several times over, give the same bits each time, and what the formula
says in fp64."""
import pytest
import torch

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def af():
    import diffusion_transformer_denoising_auraflow_b200 as m
    return m


@pytest.mark.parametrize("N,D", [(40000, 264), (33001, 512), (30011, 776), (26000, 1024)])
@pytest.mark.parametrize("post,pre", [("rms", "layer"), ("layer", "rms")])
def test_one_warp_per_row(af, N, D, post, pre):
    g = torch.Generator(device="cuda").manual_seed(991)
    x = torch.randn(1, N, D, device="cuda", generator=g).bfloat16()
    b = torch.randn(1, N, D, device="cuda", generator=g).bfloat16()
    t = torch.randn(1, 3 * D, device="cuda", generator=g)
    kw = dict(gate=t, shift=t[:, D:], scale=t[:, 2 * D:], mod_stride=3 * D, post=post, pre=pre)
    outs = [(torch.empty_like(x), torch.empty_like(x)) for _ in range(4)]
    for xo, y in outs:
        af.residual_norm(x, b, xo, y, EPS, **kw)
    for xo, y in outs[1:]:
        assert torch.equal(xo, outs[0][0]) and torch.equal(y, outs[0][1])
    # against the formula in fp64; each value within a bf16 half step (2^-8) of
    # it, and what a sum of D fp32 terms (32 lanes: D / 32 + 10 additions, twice
    # per norm) can move, in units of the row's largest value
    xr, br = x.double(), b.double()

    def norm(v, kind):
        if kind == "layer":
            v = v - v.mean(-1, keepdim=True)
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)

    c = 2 * (D / 32 + 24) * 2.0 ** -24
    tt = t.double()
    rx = xr + tt[:, :D] * norm(br, post)
    n = norm(rx, pre)
    f = 1 + tt[:, 2 * D:]
    ry = n * f + tt[:, D:2 * D]
    big = rx.abs().amax(-1, keepdim=True) + 1
    ex = 4 * c * big
    ey = f.abs() * 4 * c * (1 + big) * (n.abs().amax(-1, keepdim=True) + 1)
    assert torch.all((outs[0][0].double() - rx).abs() <= ex + rx.abs() * 2.0 ** -8)
    assert torch.all((outs[0][1].double() - ry).abs() <= ey + ry.abs() * 2.0 ** -8)
