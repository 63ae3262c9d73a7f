"""Pins of the oracle of the operators around the token mixer: gradients against central differences of the forward,
forwards against closed forms and brute-force sums."""
import math

import numpy as np
import pytest

from oracle import block_oracle as O


def differences(f, args, k, step=1e-6):
    """Gradient of the scalar f for args[k] by central differences."""
    a = args[k]
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + step
        hi = f(*args)
        a[i] = keep - step
        g[i] = (hi - f(*args)) / (2 * step)
        a[i] = keep
    return g


# central differences with step 1e-6 in fp64: rounding 2^-53 / 1e-6 (1e-10) times the value, truncation 1e-12
def close(a, b):
    assert np.abs(a - b).max() <= 1e-8 * max(1.0, np.abs(b).max())


@pytest.mark.parametrize("residual", [False, True])
def test_layer_norm_gradients_are_its_differences(residual):
    rng = np.random.default_rng(1)
    x, res = rng.standard_normal((3, 7)), rng.standard_normal((3, 7)) if residual else None
    gamma, beta, dy, dr = (rng.standard_normal(s) for s in ((7,), (7,), (3, 7), (3, 7)))

    def loss(x, gamma, beta):
        y, r = O.layer_norm(x, res, gamma, beta, 1e-5)
        return (y * dy).sum() + (r * dr).sum()

    dx, dgamma, dbeta = O.layer_norm_bwd(O.layer_norm(x, res, gamma, beta, 1e-5)[1], gamma, dy, dr, 1e-5)
    for k, g in enumerate((dx, dgamma, dbeta)):
        close(g, differences(loss, [x, gamma, beta], k))


def test_layer_norm_closed_forms():
    y, r = O.layer_norm(np.array([[1.0, 3.0]]), np.array([[1.0, 1.0]]), None, None, 0.0)
    assert np.array_equal(r, [[2.0, 4.0]]) and np.allclose(y, [[-1.0, 1.0]], atol=1e-15)
    y, _ = O.layer_norm(np.full((2, 5), 3.25), None, np.full(5, 2.0), np.arange(5.0), 1e-5)
    assert np.array_equal(y, np.tile(np.arange(5.0), (2, 1)))         # a constant row: beta alone
    dx, _, _ = O.layer_norm_bwd(np.array([[1.0, 2.0, 4.0]]), None, np.ones((1, 3)), None, 1e-5)
    assert np.abs(dx).max() < 1e-15                                    # y's sum does not depend on r


@pytest.mark.parametrize("state", [False, True])
def test_gated_scan_gradients_are_its_differences(state):
    rng = np.random.default_rng(2)
    x, gate, dh = (rng.standard_normal((2, 5, 3)) for _ in range(3))
    init, dfinal = (rng.standard_normal((2, 3)) if state else None for _ in range(2))

    def loss(x, gate, init):
        h, last = O.gated_scan(x, gate, init)
        return (h * dh).sum() + (0.0 if dfinal is None else (last * dfinal).sum())

    grads = O.gated_scan_bwd(x, gate, O.gated_scan(x, gate, init)[0], init, dh, dfinal)
    for k in range(3 if state else 2):
        close(grads[k], differences(loss, [x, gate, init], k))


def test_gated_scan_is_its_weighted_sum():
    """h_t = (prod f) init + sum_s (prod of f after s) (1 - f_s) x_s; a constant gate decays geometrically."""
    rng = np.random.default_rng(3)
    x, gate, init = rng.standard_normal((2, 6, 4)), rng.standard_normal((2, 6, 4)), rng.standard_normal((2, 4))
    f = 1 / (1 + np.exp(-gate))
    h, last = O.gated_scan(x, gate, init)
    for t in range(6):
        want = f[:, :t + 1].prod(axis=1) * init
        for s in range(t + 1):
            want = want + f[:, s + 1:t + 1].prod(axis=1) * (1 - f[:, s]) * x[:, s]
        assert np.allclose(h[:, t], want, rtol=0, atol=1e-14)
    assert np.array_equal(last, h[:, -1])
    h, _ = O.gated_scan(np.zeros((1, 9, 1)), np.zeros((1, 9, 1)), np.ones((1, 1)))
    assert np.allclose(h[0, :, 0], 0.5 ** np.arange(1, 10), rtol=1e-15)
    h, _ = O.gated_scan(np.ones((1, 3, 1)), np.full((1, 3, 1), -800.0), np.full((1, 1), 7.0))
    assert np.array_equal(h[0, :, 0], np.ones(3))                      # a closed gate copies x


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_ffn_gradients_are_its_differences(kind):
    rng = np.random.default_rng(4)
    M, D, F = 3, 4, 5
    x, wg, wu, wd = (rng.standard_normal(s) for s in ((M, D), (F, D), (F, D), (D, F)))
    dout = rng.standard_normal((M, D))
    gate, up, h, _ = O.gated_ffn(x, wg, wu, wd, kind)
    loss = lambda *a: (O.gated_ffn(*a, kind)[3] * dout).sum()
    for k, g in enumerate(O.gated_ffn_bwd(x, gate, up, h, wg, wu, wd, dout, kind)):
        close(g, differences(loss, [x, wg, wu, wd], k))


def test_activations():
    g = np.array([-30.0, -1.0, 0.0, 2.0, 40.0])
    silu = O.activation(g, "silu")[0]
    assert np.allclose(silu, [v / (1 + math.exp(-v)) for v in g], rtol=1e-14)
    gelu = O.activation(g, "gelu")[0]
    assert np.allclose(gelu, [v * 0.5 * math.erfc(-v / math.sqrt(2)) for v in g], rtol=1e-12, atol=1e-15)
