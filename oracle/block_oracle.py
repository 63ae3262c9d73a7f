"""Oracle of the operators around the token mixer: layer norm, the per-channel gated recurrence and the gated
feed-forward block, with their gradients, as plain fp64 numpy.

TEST INFRASTRUCTURE ONLY: nothing in the library imports this module and it imports nothing from the library.
"""
import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def layer_norm(x, residual, gamma, beta, eps):
    """y and r of rows x (+ residual): r = x + residual, y = (r - mean) / sqrt(var + eps) gamma + beta."""
    r = x if residual is None else x + residual
    mu = r.mean(axis=1, keepdims=True)
    var = ((r - mu) ** 2).mean(axis=1, keepdims=True)
    y = (r - mu) / np.sqrt(var + eps)
    return y * (1.0 if gamma is None else gamma) + (0.0 if beta is None else beta), r


def layer_norm_bwd(r, gamma, dy, dr, eps):
    """Gradients of sum <dy, y> + <dr, r> for r, gamma and beta."""
    mu = r.mean(axis=1, keepdims=True)
    rstd = 1.0 / np.sqrt(((r - mu) ** 2).mean(axis=1, keepdims=True) + eps)
    xhat = (r - mu) * rstd
    g = dy * (1.0 if gamma is None else gamma)
    dx = rstd * (g - g.mean(axis=1, keepdims=True) - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return dx + (0.0 if dr is None else dr), (dy * xhat).sum(axis=0), dy.sum(axis=0)


def gates(gate):
    """sigmoid(gate) and its complement, each without overflow and at full relative accuracy."""
    e = np.exp(-np.abs(gate))
    small = e / (1.0 + e)
    return np.where(gate >= 0, 1.0 / (1.0 + e), small), np.where(gate >= 0, small, 1.0 / (1.0 + e))


def gated_scan(x, gate, init):
    """All h_t = f_t h_{t-1} + (1 - f_t) x_t of x, gate [B, T, W], token by token, and the last state."""
    f, q = gates(gate)
    h = np.zeros(x.shape[::2]) if init is None else init.copy()
    out = np.empty_like(x)
    for t in range(x.shape[1]):
        h = f[:, t] * h + q[:, t] * x[:, t]
        out[:, t] = h
    return out, h


def gated_scan_bwd(x, gate, h, init, dh, dfinal):
    """Gradients of sum <dh, h> + <dfinal, h_last> for x, gate and init, with h as the forward stored it."""
    f, q = gates(gate)
    lam = np.zeros(x.shape[::2]) if dfinal is None else dfinal.copy()
    dx, dgate = np.empty_like(x), np.empty_like(x)
    for t in range(x.shape[1] - 1, -1, -1):
        lam = lam + dh[:, t]
        before = h[:, t - 1] if t else (0.0 if init is None else init)
        dx[:, t] = q[:, t] * lam
        dgate[:, t] = lam * (before - x[:, t]) * f[:, t] * q[:, t]
        lam = f[:, t] * lam
    return dx, dgate, lam


def activation(g, kind):
    """act(g) and act'(g) of "silu" or "gelu"."""
    if kind == "silu":
        s, q = gates(g)
        return g * s, s * (1.0 + g * q)
    c = 0.5 * (1.0 + _erf(g / math.sqrt(2.0)))
    return g * c, c + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)


def gated_ffn(x, w_gate, w_up, w_down, kind):
    """gate, up, h and out of the block."""
    gate, up = x @ w_gate.T, x @ w_up.T
    h = activation(gate, kind)[0] * up
    return gate, up, h, h @ w_down.T


def gated_ffn_bwd(x, gate, up, h, w_gate, w_up, w_down, dout, kind):
    """Gradients of sum <dout, out> for x, w_gate, w_up and w_down, at the stored gate, up and h."""
    act, slope = activation(gate, kind)
    dh = dout @ w_down
    dgate, dup = dh * up * slope, dh * act
    return dgate @ w_gate + dup @ w_up, dgate.T @ x, dup.T @ x, dout.T @ h
