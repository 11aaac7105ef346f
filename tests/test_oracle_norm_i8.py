"""The oracle of the RMS norm and of the 8-bit linear: gradients against
differences, the codec's rules on crafted rows, and the error that the int8
rows leave in a product."""

import numpy as np
import pytest

from oracle import i8, rmsnorm


@pytest.mark.parametrize("M,K", [(3, 5), (2, 33), (1, 1)])
def test_rmsnorm_gradients_match_differences(M, K):
    g = np.random.default_rng(7)
    h, w, dy = g.standard_normal((M, K)), 1 + 0.1 * g.standard_normal(K), g.standard_normal((M, K))
    eps, d = 1e-5, 1e-6
    f = lambda hh, ww: (rmsnorm.fwd(hh, ww, eps) * dy).sum()
    dh, dw = rmsnorm.bwd(dy, h, w, eps)
    # A central difference is off by d^2 / 6 of the third derivative. With u = mean h^2 + eps, u' = 2 h_i / K and
    # h_i^2 <= K u: the second derivative of u^-1/2 is at most 4 u^-3/2 / K, and |h_k| times its third at most
    # 24 u^-3/2 / K, so the third derivative of h_k u^-1/2 is below 36 u^-3/2 (the row of one small element comes
    # near it: its u is eps); and the values it subtracts are rounded.
    u = (h * h).mean(axis=1).min() + eps
    tol = 1.1 * 6 * d * d * u ** -1.5 * np.abs(w * dy).sum() + 2.0 ** -48 * np.abs(rmsnorm.fwd(h, w, eps) * dy).sum() / d
    for i in np.ndindex(h.shape):
        e = np.zeros_like(h)
        e[i] = d
        assert abs((f(h + e, w) - f(h - e, w)) / (2 * d) - dh[i]) < tol
    for k in range(K):
        e = np.zeros(K)
        e[k] = d
        assert abs((f(h, w + e) - f(h, w - e)) / (2 * d) - dw[k]) < tol


def test_codec_rules_on_crafted_rows():
    x = np.array([[127, -127, 0.5, 1.5, 2.5, -2.5, 0.0, 63.49],   # scale 1: ties to even
                  [0, 0, 0, 0, 0, 0, 0, 0],
                  [1, np.nan, 0, 0, 0, 0, 0, 0],
                  [1, -np.inf, 0, 0, 0, 0, 0, 0],
                  [1e-45, -1e-45, 0, 0, 0, 0, 0, 0],              # max / 127 rounds to zero
                  [3e38, -1e38, 0, 0, 0, 0, 0, 1e-30]], np.float32)
    q, s = i8.quantize(x)
    assert q[0].tolist() == [127, -127, 0, 2, 2, -2, 0, 63] and s[0] == 1
    assert not q[1].any() and s[1] == 0
    assert not q[2].any() and np.isnan(s[2]) and not q[3].any() and np.isnan(s[3])
    assert not q[4].any() and s[4] == 0
    assert q[5].tolist() == [127, -42, 0, 0, 0, 0, 0, 0]
    over = np.full(8, 1e10, np.float32)   # the column scale overflows one row's maximum
    q, s = i8.quantize(x[5:], over)
    assert not q.any() and np.isnan(s[0])


def test_codec_error_is_half_a_step():
    g = np.random.default_rng(8)
    x = (g.standard_normal((50, 300)) * 10.0 ** g.integers(-20, 20, (50, 1))).astype(np.float32)
    q, s = i8.quantize(x)
    assert np.abs(q).max() == 127
    err = np.abs(q.astype(np.float64) * s[:, None] - x)
    # half a step, and the roundings of the scale and the quotient (127.5 steps, 2^-24 each)
    assert np.all(err <= s[:, None].astype(np.float64) * (0.5 + 3 * 127.5 * 2.0 ** -24))


def test_input_gradient_is_that_of_the_dequantised_layer():
    """The int8 gradient against dY W^ of the dequantised weight: off by the
    rounding of the rows of dY sw alone, half a step of each row an element."""
    g = np.random.default_rng(9)
    M, N, K = 6, 64, 48
    wq, sw = i8.quantize((g.standard_normal((N, K)) * 0.02).astype(np.float32))
    dY = g.standard_normal((M, N)).astype(np.float32)
    got = i8.linear_dx(dY, wq, sw)
    exact = (dY * sw.astype(np.float64)) @ wq.astype(np.float64)
    _, sg = i8.quantize(dY, sw)
    bound = 0.5001 * sg.astype(np.float64)[:, None] * np.abs(wq.astype(np.float64)).sum(axis=0)
    assert np.all(np.abs(got - exact) <= bound)
