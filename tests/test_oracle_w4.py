"""Pins of the oracle's 4-bit weights and of the residual between two norms:
hand-made rows, invariants and second ways of writing the same formula."""
import numpy as np
import pytest

import oracle as O


def test_quantize_hand_example():
    # a = 7 * 0.5: scale 0.5 exactly; halves go to the even whole number
    w = np.zeros((1, 33))
    w[0, :8] = [3.5, -3.5, 0.25, 0.75, -0.25, 1.0, 0.0, -1.26]
    w[0, 32] = -14.0                                   # a group of one column
    c, s = O.quantize_rows_w4(w, 32)
    assert c.shape == (1, 64) and s.shape == (2, 1)
    assert list(s[:, 0]) == [0.5, 2.0]
    assert list(c[0, :8]) == [15, 1, 8, 10, 8, 10, 8, 5]   # 0.5 -> 0, 1.5 -> 2, -0.5 -> 0, -2.52 -> -3
    assert c[0, 32] == 1 and np.all(c[0, 33:] == 8)
    v = O.dequantize_rows_w4(c, s, 32, 33)
    assert v.shape == (1, 33) and v[0, 0] == 3.5 and v[0, 32] == -14.0


def test_quantize_zero_rows_and_bound():
    rng = np.random.default_rng(5)
    w = rng.normal(size=(9, 200)) * 0.02
    w[3] = 0.0
    w[4, 64:128] = 0.0
    c, s = O.quantize_rows_w4(w, 64)
    assert np.all(c[3] == 8) and np.all(s[:, 3] == 0) and s[1, 4] == 0
    v = O.dequantize_rows_w4(c, s, 64, 200)
    step = np.repeat(s.T, 64, axis=1)[:, :200]
    # half a step, and at the group's maximum what bf16 took from the scale (7 steps x 2^-8)
    assert np.all(np.abs(v - w) <= step * (0.5 + 7 * 2.0 ** -8))
    assert c.min() >= 1 and c.max() <= 15


def test_linear_is_the_product_with_the_values():
    rng = np.random.default_rng(6)
    w, x, b = rng.normal(size=(5, 70)), rng.normal(size=(3, 70)), rng.normal(size=5)
    c, s = O.quantize_rows_w4(w, 32)
    v = O.dequantize_rows_w4(c, s, 32, 70)
    got = O.linear_w4(x, c, s, 32, True, b)
    want = [[b[n] + sum(x[m, k] / (1 + np.exp(-x[m, k])) * v[n, k] for k in range(70)) for n in range(5)]
            for m in range(3)]
    assert np.allclose(got, want, rtol=1e-12)


@pytest.mark.parametrize("post", ["none", "layer", "rms"])
def test_residual_norm_is_modulate_of_the_residual(post):
    rng = np.random.default_rng(7)
    x, b = rng.normal(size=(2, 3, 16)), rng.normal(size=(2, 3, 16)) + 1
    g, sh, sc = rng.normal(size=(3, 2, 16))
    xo, y = O.residual_norm(x, b, 1e-6, gate=g, shift=sh, scale=sc, residual_scale=0.5, post=post)
    assert np.allclose(y, O.modulate(xo, sh, sc, 1e-6))
    for i in range(2):
        for n in range(3):
            u = b[i, n]
            if post != "none":
                m = u.mean() if post == "layer" else 0.0
                u = (u - m) / np.sqrt(((u - m) ** 2).mean() + 1e-6)
            assert np.allclose(xo[i, n], x[i, n] + 0.5 * g[i] * u)


def test_residual_norm_invariants():
    rng = np.random.default_rng(8)
    x, b = rng.normal(size=(1, 4, 32)), rng.normal(size=(1, 4, 32))
    # zero gate: the residual stays; no branch: the same
    xo, y = O.residual_norm(x, b, 0.0, gate=np.zeros((1, 32)))
    x2, y2 = O.residual_norm(x, None, 0.0)
    assert np.array_equal(xo, x) and np.array_equal(x2, x) and np.array_equal(y, y2)
    # RMS norm: unit mean square; a post norm does not see the branch's scale
    _, y = O.residual_norm(x, b, 0.0, pre="rms")
    assert np.allclose((y * y).mean(-1), 1.0)
    a = O.residual_norm(x, b, 0.0, post="rms")[0]
    assert np.allclose(O.residual_norm(x, 10 * b, 0.0, post="rms")[0], a)
    assert np.allclose(O.residual_norm(x, b, 0.0, pre="none")[1], x + b)
