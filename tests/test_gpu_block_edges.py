"""The operators around the token mixer where values are small, far from zero or not finite, over many rows, and beside
the layer itself: on the GPU through the C ABI, against 64-bit results, with bounds derived in each test.

u = 2^-24 is fp32's rounding; a tensor stored in type t is rounded once, by at most finfo(t).eps / 2 of its value.
"""
import math

import numpy as np
import pytest
import torch

from parameter_space_moe_b200 import swimba
from tests.test_gpu_block import TYPES, U, Out, ok, within

pytestmark = pytest.mark.gpu

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


# ------------------------------------------------------------------------------------------------ feed-forward
def gelu_tail(g, dt):
    """gelu(g) and its slope without cancellation, and the relative error of the kernel's tail, which its complement for
    positive g keeps in absolute terms (at most as large relative to it, and one rounding)."""
    z = -g / math.sqrt(2.0)
    c = 0.5 * _erfc(z)
    n = np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if dt != "f32":
        # the exponent g^2 / 2 and its change of base carry four roundings; ex2, the quotient 2 ulp; the fit 2^-19.9;
        # two products
        return g * c, c + g * n, c, n, U * (4 * 0.5 * g * g + 4 + 4 + 2) + 2.0 ** -19.9
    # z carries two roundings (the constant's and the product's), which erfc passes on by |z erfc'(z) / erfc(z)|;
    # erfc itself is good to 4 ulp, 8 u
    rel = U * (2 * np.abs(z) * 2 * np.exp(-z * z) / (math.sqrt(math.pi) * _erfc(z)) + 8)
    return g * c, c + g * n, c, n, rel


@pytest.mark.parametrize("dt", TYPES)
def test_gelu_keeps_its_negative_tail(dt):
    """h = gelu(g) up and its two factors' gradients for g in [-8, 8], element by element and relative to the value: the
    products around them are exact (one non-zero term of 1 each)."""
    code, t = TYPES[dt]
    D = F = 264
    g = torch.linspace(-8, 8, 256).to(t)
    gn = g.double().numpy()
    value, slope, c, n, rel = gelu_tail(gn, dt)
    # forward: x = (g, 1, 0 ..), gate = x and up = x[256] = 1 by weights of zeros and ones
    x = torch.zeros(1, D, dtype=t)
    x[0, :256], x[0, 256] = g, 1
    wg, wu = torch.zeros(F, D, dtype=t), torch.zeros(F, D, dtype=t)
    wg[range(256), range(256)], wu[:, 256] = 1, 1
    d = swimba.ffn_dims(1, D, F, code, swimba.GELU)
    ws = torch.empty(max(swimba.gated_ffn_workspace_size(d), swimba.gated_ffn_bwd_workspace_size(d)), dtype=torch.uint8,
                     device="cuda")
    gate, up, h, out = (Out((1, k), t) for k in (F, F, F, D))
    swimba.gated_ffn(d, x.cuda(), wg.cuda(), wu.cuda(), torch.zeros(D, F, dtype=t).cuda(), gate.t, up.t, h.t, out.t, ws)
    ok()
    assert np.array_equal(gate.np()[0, :256], gn) and (up.np() == 1).all()
    # the cumulative term's error, then its half, times g, times up
    within(h.np()[0, :256], value, np.abs(value) * (rel + 3 * U), t, f"gelu {dt}")
    # backward: dh = 1, up = 1, x = (1, 0 ..), so that the first columns of dw_gate and dw_up are dgate and dup, rounded once
    one = torch.zeros(1, D, dtype=t)
    one[0, 0] = 1
    wd = torch.zeros(D, F, dtype=t)
    wd[0] = 1
    stored = torch.zeros(1, F, dtype=t)
    stored[0, :256] = g
    dx, dwg, dwu, dwd = Out((1, D), t), Out((F, D), t), Out((F, D), t), Out((D, F), t)
    swimba.gated_ffn_bwd(d, one.cuda(), stored.cuda(), torch.ones(1, F, dtype=t).cuda(), h.t, wg.cuda(), wu.cuda(), wd.cuda(),
                         one.cuda(), dx.t, dwg.t, dwu.t, dwd.t, ws)
    ok()
    within(dwu.np()[:256, 0], value, np.abs(value) * (rel + 3 * U), t, "dup")
    # the density: the exponent -g^2 / 2 and its change of base carry four roundings, ex2 2 ulp, the constant and two
    # products one rounding each; then the sum's
    e = c * rel + np.abs(gn) * n * U * (4 * 0.5 * gn * gn + 4 + 4) + U * np.abs(slope)
    within(dwg.np()[:256, 0], slope, e + 2 * U * np.abs(slope), t, "dgate")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("M,D,F", [(1 << 20, 64, 72), ((1 << 18) + 40, 264, 136)])
def test_gradients_of_the_weights_over_many_rows(M, D, F, dt):
    """Sums over a million rows of one sign: the tensor cores cut, they do not round, so an unbroken chain drifts."""
    code, t = TYPES[dt]
    gen = torch.Generator(device="cuda").manual_seed(M + D)
    draw = lambda *s: (torch.rand(*s, generator=gen, device="cuda") + 0.5).to(t)
    x, gate, up, h, dout = draw(M, D), draw(M, F), draw(M, F), draw(M, F), (draw(M, D) * 2.0 ** -10).to(t)
    wd = draw(D, F) / 64
    d = swimba.ffn_dims(M, D, F, code)
    ws = torch.empty(swimba.gated_ffn_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    w = draw(F, D) / 64
    dx, dwg, dwu, dwd = torch.empty_like(x), Out((F, D), t), Out((F, D), t), Out((D, F), t)
    swimba.gated_ffn_bwd(d, x, gate, up, h, w, w, wd, dout, dx, dwg.t, dwu.t, dwd.t, ws)
    ok()
    want_d, want_u = torch.zeros(D, F, dtype=torch.float64, device="cuda"), torch.zeros(F, D, dtype=torch.float64, device="cuda")
    rough = torch.zeros_like(want_u)
    for i in range(0, M, 1 << 16):
        j = slice(i, min(M, i + (1 << 16)))
        want_d += dout[j].double().T @ h[j].double()
        g = gate[j].double()
        dup = (dout[j].double() @ wd.double()) * g * torch.sigmoid(g)
        want_u += dup.T @ x[j].double()
        rough += dup.abs().T @ x[j].double().abs()
    # every term is positive, so a chain's running sum never passes its end: a step of 16 cuts less than 2^-23 of it, and
    # a chain is 65536 of K (bf16) or 16384 (fp16) long; the split sums, 64 at most, add a rounding each
    cut = (4096 if dt == "bf16" else 1024) * 2.0 ** -23 + 64 * U
    want = want_d.cpu().numpy()
    within(dwd.np(), want, cut * np.abs(want), t, f"dw_down {M}x{D}x{F} {dt}")
    # dup is rounded to the type on its way, and its own product cuts K / 16 steps
    want, rough = want_u.cpu().numpy(), rough.cpu().numpy()
    within(dwu.np(), want, cut * np.abs(want) + (torch.finfo(t).eps / 2 + (D / 16 + 32) * 2.0 ** -23) * rough, t, "dw_up")
