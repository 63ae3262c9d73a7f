"""The operators around the token mixer where values are small, far from zero or not finite, over many rows, and beside
the layer itself: on the GPU through the C ABI, against 64-bit results, with bounds derived in each test.

u = 2^-24 is fp32's rounding; a tensor stored in type t is rounded once, by at most finfo(t).eps / 2 of its value.
"""
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from oracle import swimba_oracle as S
from parameter_space_moe_b200 import configs, inputs, swimba

from .parity import check_topk, device_weights, f64, out_dtype, tol_of
from .test_gpu_block import ROW_ADDS, TYPES, U, Out, ok, within

pytestmark = pytest.mark.gpu

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


# ------------------------------------------------------------------------------------------------ layer norm
# Every layout of a row (columns a thread, one or several warps, single columns or vectors) over at least four rows a
# team and a last turn that some teams sit out: the loads a row ahead, the steps of the pointers, the sums' two copies, the
# room of the asynchronous copies.  The last entry is the layout of few rows, two a team.
MANY_ROWS = [(14401, 29), (14401, 61), (14401, 93), (14401, 125), (14401, 189), (14401, 221), (14401, 253), (1801, 219),
             (1801, 411), (1801, 659), (1801, 823), (1801, 1319), (1801, 1567), (1801, 2047), (1801, 2049), (1801, 5001),
             (601, 8191), (601, 16383), (19001, 96), (19001, 132), (19001, 256), (14401, 264), (14401, 260), (14401, 384),
             (14401, 500), (14401, 512), (7201, 768), (7201, 776), (2401, 876), (7201, 1000), (3601, 2048), (1801, 2052),
             (1801, 2636), (1801, 3000), (1801, 4096), (1801, 4100), (1801, 4104), (1801, 5000), (601, 6148), (601, 6152),
             (601, 8200), (601, 16384), (591, 1024)]


def drawn(gen, shape, t, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale + shift).to(t)


def near(got, ref, bound, t, what):
    """within() on the GPU: |got - ref| <= bound + the one rounding to t."""
    eps, low = torch.finfo(t).eps / 2, torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2
    tol = 1.01 * (bound + eps * (ref.abs() + bound)) + low
    worst = ((got.double() - ref).abs() / tol).max()
    assert bool(torch.isfinite(got).all()) and float(worst) <= 1.0, f"{what}: {float(worst):.3f} of its bound"


def row_stats(r, eps):
    """xhat, rstd, and the errors of xhat and (relative) of rstd in fp32: the row's mean is off by ROW_ADDS u mean|r|, a
    centred value by that, its own rounding and the difference's; the variance by twice that over its terms and its sum."""
    mu = r.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((r - mu) ** 2).mean(1, keepdim=True) + eps)
    xhat = (r - mu) * rstd
    dev = U * (ROW_ADDS * r.abs().mean(1, keepdim=True) + r.abs()) * rstd + U * xhat.abs()
    rel = (dev * xhat.abs()).mean(1, keepdim=True) + U * (ROW_ADDS + 8)
    return xhat, rstd, dev + rel * xhat.abs(), rel


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,D", MANY_ROWS)
def test_layer_norm_over_many_rows(M, D, dt):
    """Rows of a wider tensor, the residual stream updated in place."""
    code, t = TYPES[dt]
    eps = float(np.float32(1e-5))
    gen = torch.Generator(device="cuda").manual_seed(M + D)
    x, res = drawn(gen, (M, D + 8), t, 1.5, 0.7)[:, :D], Out((M, D), t)
    res.t.copy_(drawn(gen, (M, D), t, 3.0, -0.4))
    gamma, beta = drawn(gen, (D,), torch.float32, 0.3, 1.0), drawn(gen, (D,), torch.float32, 0.3)
    r = x.double() + res.t.double()
    y = Out((M, D), t)
    swimba.layer_norm(swimba.norm_dims(M, D, code, x_stride=D + 8, eps=eps), x, res.t, gamma, beta, y.t, res.t)
    ok()
    xhat, _, dx, _ = row_stats(r, eps)
    near(y.t, xhat * gamma.double() + beta.double(), dx * gamma.double().abs()
         + 3 * U * (xhat.abs() * gamma.double().abs() + beta.double().abs()), t, f"y {M}x{D} {dt}")
    near(res.t, r, U * r.abs(), t, "r")
    y.np(), res.np()  # nothing is written behind them


@pytest.mark.parametrize("dt,gt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("M,D", MANY_ROWS)
def test_layer_norm_gradients_over_many_rows(M, D, dt, gt):
    """With gamma and the gradient that reaches r past the norm (dx over it), and without either."""
    (code, t), (gcode, g_t) = TYPES[dt], TYPES[gt]
    eps = float(np.float32(1e-5))
    gen = torch.Generator(device="cuda").manual_seed(M * 3 + D)
    r, gamma = drawn(gen, (M, D), t, 2.0, 0.5), drawn(gen, (D,), torch.float32, 0.3, 1.0)
    dy, dr = drawn(gen, (M, D), g_t, 0.5), drawn(gen, (M, D), g_t, 0.5)
    d = swimba.norm_dims(M, D, code, gcode, eps=eps)
    ws = torch.empty(swimba.layer_norm_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    mean = lambda v: v.mean(1, keepdim=True)
    rd, dyd = r.double(), dy.double()
    xhat, rstd, dxhat, rel = row_stats(rd, eps)
    for gm, past in ((gamma, dr), (None, None)):
        dx, dg, db = Out((M, D), g_t), Out((D,), torch.float32), Out((D,), torch.float32)
        if past is not None:
            dx.t.copy_(past)
        swimba.layer_norm_bwd(d, r, gm, dy, dx.t if past is not None else None, dx.t, dg.t, db.t, ws)
        ok()
        ga = torch.ones(D, dtype=torch.float64, device="cuda") if gm is None else gm.double()
        g = dyd * ga
        want = rstd * (g - mean(g) - xhat * mean(g * xhat))
        mg, mgx = mean(g.abs()), mean(g.abs() * xhat.abs())
        inner = g.abs() + mg + xhat.abs() * mgx
        bound = rstd * (U * (ROW_ADDS + 2) * mg + dxhat * mgx + xhat.abs() * (mean(g.abs() * dxhat) + U * (ROW_ADDS + 4) * mgx)
                        + (4 * U + rel) * inner)
        if past is not None:
            want = want + past.double()
            bound = bound + U * (past.double().abs() + rstd * inner)
        near(dx.t, want, bound, g_t, f"dx {M}x{D} {dt}/{gt}")
        # a column's sum: a team's rows, then the block's teams, at most 19 partial rows in a thread and 32 threads
        adds = M / 148 + 1 + 16 + 19 + 32
        near(dg.t, (dyd * xhat).sum(0), (dyd.abs() * (dxhat + (adds + 1) * U * xhat.abs())).sum(0), torch.float32, "dgamma")
        near(db.t, dyd.sum(0), adds * U * dyd.abs().sum(0), torch.float32, "dbeta")
        dx.np(), dg.np(), db.np()


# ------------------------------------------------------------------------------------------------ gated scan
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,W", [(400, 64), (2100, 33)])
def test_what_is_not_finite_stays_in_its_channel_for_good(T, W, dt):
    """A state that is not finite stays so: f = 0 times it is NaN.  The other channels keep their bits."""
    code, t = TYPES[dt]
    gen = torch.Generator(device="cuda").manual_seed(T)
    x, gate = drawn(gen, (1, T, W), t), drawn(gen, (1, T, W), t)
    gate[:, 250] = -float("inf")
    want, h = torch.empty_like(x), torch.empty_like(x)
    fin = torch.empty(1, W, device="cuda")
    d = swimba.gated_dims(1, T, W, code)
    swimba.gated_scan(d, x, gate, None, want, None)
    x[0, 41, 7], x[0, 137, 20] = float("inf"), float("nan")
    swimba.gated_scan(d, x, gate, None, h, fin)
    ok()
    assert torch.equal(want[0, 250], x[0, 250])
    for c, first in ((7, 41), (20, 137)):
        assert not bool(torch.isfinite(h[0, first:, c]).any()) and not bool(torch.isfinite(fin[0, c]))
        assert torch.equal(h[0, :first, c], want[0, :first, c])
    rest = [c for c in range(W) if c not in (7, 20)]
    assert torch.equal(h[..., rest], want[..., rest]) and bool(torch.isfinite(fin[0, rest]).all())


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
    # a chain is 65536 of K (bf16) or 16384 (fp16) long; the sums of the chains, 64 at most, add a rounding each
    cut = (4096 if dt == "bf16" else 1024) * 2.0 ** -23 + 64 * U
    want = want_d.cpu().numpy()
    within(dwd.np(), want, cut * np.abs(want), t, f"dw_down {M}x{D}x{F} {dt}")
    # dup is rounded to the type on its way, and its own product cuts K / 16 steps
    want, rough = want_u.cpu().numpy(), rough.cpu().numpy()
    within(dwu.np(), want, cut * np.abs(want) + (torch.finfo(t).eps / 2 + (D / 16 + 32) * 2.0 ** -23) * rough, t, "dw_up")


def chained(K, planes=6):
    """Norm-wise error of an fp32 product over K on three bf16 planes a tensor, random signs.  A chain is 256 of K: 16
    steps that each cut less than 2^-23 of the running sum, which is at most the chain's end; the chains' cuts have their
    chains' signs and add up like them.  The chains, 6 K / 256 of them, are added with a rounding of u each, independent
    ones; the plane products left out are 2^-24 of the whole, the result is rounded once."""
    return 16 * 2.0 ** -23 + U * (math.sqrt(planes * K / 256 + planes) + 2)


def normwise(got, ref, bar, what):
    e = float((got.double() - ref).norm() / ref.norm())
    print(f"{what}: {e:.2e} of {bar:.2e}")
    assert e <= bar, what


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("M,D,F", [(300, 768, 2816), (2900, 264, 1032), (130, 2816, 264), (5000, 520, 3000)])
def test_fp32_products_keep_their_accuracy(M, D, F, kind):
    """Norm-wise, each product from the operands that the GPU holds: an unbroken chain (2e-5 at 12 x 2816) or a plane
    product left out (2^-16) is many times the bar."""
    gen = torch.Generator(device="cuda").manual_seed(M + F)
    draw = lambda *s, std=1.0: drawn(gen, s, torch.float32, std)
    x, dout = draw(M, D), draw(M, D)
    wg, wu, wd = draw(F, D, std=D ** -0.5), draw(F, D, std=D ** -0.5), draw(D, F, std=F ** -0.5)
    d = swimba.ffn_dims(M, D, F, swimba.F32, swimba.SILU if kind == "silu" else swimba.GELU)
    ws = torch.empty(max(swimba.gated_ffn_workspace_size(d), swimba.gated_ffn_bwd_workspace_size(d)), dtype=torch.uint8,
                     device="cuda")
    gate, up, h, out = (torch.empty(M, k, device="cuda") for k in (F, F, F, D))
    swimba.gated_ffn(d, x, wg, wu, wd, gate, up, h, out, ws)
    dx, dwg, dwu, dwd = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu), torch.empty_like(wd)
    swimba.gated_ffn_bwd(d, x, gate, up, h, wg, wu, wd, dout, dx, dwg, dwu, dwd, ws)
    ok()
    x, dout, wg, wu, wd, G, P, H = (v.double() for v in (x, dout, wg, wu, wd, gate, up, h))
    normwise(gate, x @ wg.T, chained(D), "gate")
    normwise(up, x @ wu.T, chained(D), "up")
    if kind == "silu":
        s = torch.sigmoid(G)
        act, slope = G * s, s * (1 + G * (1 - s))
    else:
        c = 0.5 * torch.special.erfc(-G / math.sqrt(2.0))
        act, slope = G * c, c + G * torch.exp(-0.5 * G * G) / math.sqrt(2 * math.pi)
    # h is formed from the sums that gate and up are stored from: the same values in fp32
    normwise(h, act * P, 16 * U, "h")
    normwise(out, H @ wd.T, chained(F), "out")
    dh = dout @ wd
    dg, du = dh * P * slope, dh * act
    # the products behind dgate and dup carry dh's error and the activation's 32 u, which random signs pass on as they are
    normwise(dx, dg @ wg + du @ wu, chained(2 * F) + chained(D) + 32 * U, "dx")
    normwise(dwg, dg.T @ x, chained(M) + chained(D) + 32 * U, "dw_gate")
    normwise(dwu, du.T @ x, chained(M) + chained(D) + 32 * U, "dw_up")
    normwise(dwd, dout.T @ H, chained(M), "dw_down")


@pytest.mark.parametrize("exponent", [-100, -114, -126])
def test_fp32_small_values(exponent):
    """A value's third plane ends at bf16's smallest subnormal, 2^-133: below 2^-108 it is off by up to half of that."""
    M, D, F = 256, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    h, w, wd = drawn(gen, (M, F), torch.float32), drawn(gen, (F, D), torch.float32), drawn(gen, (D, F), torch.float32)
    dout = torch.ldexp(drawn(gen, (M, D), torch.float32), torch.tensor(float(exponent), device="cuda"))
    d = swimba.ffn_dims(M, D, F, swimba.F32)
    ws = torch.empty(swimba.gated_ffn_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    dx, dwg, dwu, dwd = torch.empty(M, D, device="cuda"), torch.empty_like(w), torch.empty_like(w), torch.empty_like(wd)
    swimba.gated_ffn_bwd(d, torch.ones(M, D, device="cuda"), h, h, h, w, w, wd, dout, dx, dwg, dwu, dwd, ws)
    ok()
    want, size = dout.double().T @ h.double(), dout.double().abs().T @ h.double().abs()
    # one chain of 256 a plane product; the results are stored down to fp32's own subnormals
    tol = (16 * 2.0 ** -23 + 8 * U) * size + 2.0 ** -134 * h.double().abs().sum(0) + 2.0 ** -149
    assert bool(((dwd.double() - want).abs() <= tol).all())


def test_fp32_infinities_stay_in_their_rows():
    """An infinite input makes what depends on it not finite (infinite, or NaN where plane products of both signs meet or a
    plane is 0) and leaves the other rows their bits."""
    M, D, F = 140, 72, 136
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = drawn(gen, (M, D), torch.float32)
    wg, wu, wd = drawn(gen, (F, D), torch.float32), drawn(gen, (F, D), torch.float32), drawn(gen, (D, F), torch.float32)
    d = swimba.ffn_dims(M, D, F, swimba.F32)
    ws = torch.empty(swimba.gated_ffn_workspace_size(d), dtype=torch.uint8, device="cuda")
    outs = []
    for bad in (False, True):
        if bad:
            x[3, 5], x[77, 70] = float("inf"), -float("inf")
        gate, up, h, out = (torch.empty(M, k, device="cuda") for k in (F, F, F, D))
        swimba.gated_ffn(d, x, wg, wu, wd, gate, up, h, out, ws)
        ok()
        outs.append((gate, up, h, out))
    rest = [m for m in range(M) if m not in (3, 77)]
    for a, b in zip(*outs):
        assert bool(torch.isfinite(a).all()) and torch.equal(a[rest], b[rest])
    for v in outs[1][:2]:
        assert not bool(torch.isfinite(v[[3, 77]]).any())
    assert bool(torch.isnan(outs[1][3][[3, 77]]).all())   # both signs, or NaN, among the hidden features


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("exponent", [-14, -7, 5])
def test_gradients_of_small_and_large_losses(exponent, dt):
    """Upstream gradients from fp16's subnormals to 2^7: dgate and dup are rounded to the type, subnormal spacing
    included, which is why the caller scales an fp16 loss."""
    code, t = TYPES[dt]
    M, D, F = 300, 264, 520
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, gate, up, h = (drawn(gen, s, t) for s in ((M, D), (M, F), (M, F), (M, F)))
    wg, wu, wd = (drawn(gen, s, t, s[1] ** -0.5) for s in ((F, D), (F, D), (D, F)))
    dout = drawn(gen, (M, D), t, 2.0 ** exponent)
    d = swimba.ffn_dims(M, D, F, code)
    ws = torch.empty(swimba.gated_ffn_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    dx, dwg, dwu, dwd = Out((M, D), t), Out((F, D), t), Out((F, D), t), Out((D, F), t)
    swimba.gated_ffn_bwd(d, x, gate, up, h, wg, wu, wd, dout, dx.t, dwg.t, dwu.t, dwd.t, ws)
    ok()
    x, dout, wg, wu, wd, g, u, h = (v.double() for v in (x, dout, wg, wu, wd, gate, up, h))
    s = torch.sigmoid(g)
    act, slope = g * s, s * (1 + g * (1 - s))
    dot = lambda a, b: 2 * U * a.shape[1] * (a.abs() @ b.abs())
    eps, low = torch.finfo(t).eps / 2, torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2
    dh, e = dout @ wd, dot(dout, wd)
    dg, du = dh * u * slope, dh * act
    bg = e * (u * slope).abs() + 32 * U * (dh * u).abs() * (1 + g.abs())
    bu = e * act.abs() + 16 * U * (dh * g).abs()
    rg, ru = (b + eps * (v.abs() + b) + low for v, b in ((dg, bg), (du, bu)))
    near(dx.t, dg @ wg + du @ wu, 2 * (dot(dg, wg) + dot(du, wu)) + rg @ wg.abs() + ru @ wu.abs(), t, "dx")
    near(dwg.t, dg.T @ x, dot(dg.T, x) + rg.T @ x.abs(), t, "dw_gate")
    near(dwu.t, du.T @ x, dot(du.T, x) + ru.T @ x.abs(), t, "dw_up")
    near(dwd.t, dout.T @ h, dot(dout.T, h), t, "dw_down")
    dx.np(), dwg.np(), dwu.np(), dwd.np()


# ------------------------------------------------------------------------------------------------ beside the layer
@pytest.mark.parametrize("w", [configs.TINY_F32.with_(name="row_f32", seqlen=200, seed=151),
                               configs.BASE.with_(name="row_bf16", batch=2, seqlen=300, d_model=128, nheads=2, n_experts=4,
                                                  chunk=128, seed=152)], ids=lambda w: w.name)
def test_a_row_with_the_layer(w):
    """Norm, the Swimba layer, output projection, norm over the residual sum, feed-forward block, then the gradients of
    the block, the second norm, the layer (fp32, for a seeded dy) and the first norm (fp32 gradients beside its type), all
    in a row on one stream without a pause.  Every call's result is held to its operator's 64-bit result on what the GPU
    gave it; the row with a pause behind every call gives the same bits
    up to the layer's gradients."""
    B, T, D, F, M, HP = w.batch, w.seqlen, w.d_model, 256, w.M, w.nheads * w.headdim
    t = out_dtype(w)
    code = swimba.F32 if t is torch.float32 else swimba.BF16
    inp = inputs.make_inputs(w)
    d, W = swimba.dims_of(w), device_weights(inp)
    gen = torch.Generator(device="cuda").manual_seed(w.seed)
    f32 = torch.float32
    x, dout, dy = drawn(gen, (M, D), t), drawn(gen, (M, D), t, 0.3), drawn(gen, (M, HP), f32)
    g1, b1, g2, b2 = (drawn(gen, (D,), f32, 0.2, m) for m in (1.0, 0.0, 1.0, 0.0))
    wg, wu, wd = (drawn(gen, s, t, s[1] ** -0.5) for s in ((F, D), (F, D), (D, F)))
    w_out = inp["W_out"].cuda()
    nd, n32, fd = swimba.norm_dims(M, D, code), swimba.norm_dims(M, D, code, swimba.F32), swimba.ffn_dims(M, D, F, code)
    ws = torch.empty(max(swimba.layer_bwd_workspace_size(d), swimba.gated_ffn_workspace_size(fd),
                         swimba.gated_ffn_bwd_workspace_size(fd), swimba.layer_norm_bwd_workspace_size(n32)),
                     dtype=torch.uint8, device="cuda")

    def row(pause):
        new = lambda *s, ty=t: torch.full(s, float("nan"), dtype=ty, device="cuda")
        v = dict(n1=new(M, D), y=new(M, HP), p=new(M, D), n2=new(M, D), r=new(M, D), gate=new(M, F), up=new(M, F),
                 h=new(M, F), out=new(M, D), dn2=new(M, D), dr=new(M, D), dg2=new(D, ty=f32), db2=new(D, ty=f32),
                 dn1=new(M, D, ty=f32), dx=new(M, D, ty=f32), dg1=new(D, ty=f32), db1=new(D, ty=f32))
        idx = torch.empty(M, w.top_k, dtype=torch.int32, device="cuda")
        lw = [new(*s, ty=f32) for s in ((w.n_experts, D), (w.nheads, D), (w.nheads,), (w.nheads,), (w.n_experts, w.W_e, D))]
        dwg, dwu, dwd = new(F, D), new(F, D), new(D, F)
        torch.cuda.synchronize()
        for call in (lambda: swimba.layer_norm(nd, x, None, g1, b1, v["n1"], None),
                     lambda: swimba.layer_fwd(d, v["n1"], W, None, v["y"], None, idx, None, ws),
                     lambda: swimba.out_proj(d, v["y"], w_out, v["p"]),
                     lambda: swimba.layer_norm(nd, v["p"], x, g2, b2, v["n2"], v["r"]),
                     lambda: swimba.gated_ffn(fd, v["n2"], wg, wu, wd, v["gate"], v["up"], v["h"], v["out"], ws),
                     lambda: swimba.gated_ffn_bwd(fd, v["n2"], v["gate"], v["up"], v["h"], wg, wu, wd, dout, v["dn2"], dwg, dwu,
                                                  dwd, ws),
                     lambda: swimba.layer_norm_bwd(nd, v["r"], g2, v["dn2"], dout, v["dr"], v["dg2"], v["db2"], ws),
                     lambda: swimba.layer_bwd(d, v["n1"], W, None, dy, v["dn1"], *lw, None, ws),
                     lambda: swimba.layer_norm_bwd(n32, x, g1, v["dn1"], None, v["dx"], v["dg1"], v["db1"], ws)):
            call()
            if pause:
                torch.cuda.synchronize()
        ok()
        return v, idx

    row(False)
    (v, idx), (slow, _) = row(False), row(True)
    for k in v:
        assert bool(torch.isfinite(v[k]).all()), k
        if k not in ("dn1", "dx", "dg1", "db1"):    # the layer's gradients are summed by atomics, in any order
            assert torch.equal(v[k], slow[k]), k
    n = {k: a.double().cpu().numpy() for k, a in v.items()}
    num = lambda a: a.double().cpu().numpy()
    eps = float(np.float32(1e-5))
    own = 1e-5 if code == swimba.F32 else 2.0 ** -8    # one rounding, beside which the fp32 sums' are nothing
    layer = tol_of(w)
    held = lambda got, ref, bar, what: normwise(torch.from_numpy(got), torch.from_numpy(ref.reshape(got.shape)), bar, what)
    held(n["n1"], O.layer_norm(num(x), None, num(g1), num(b1), eps)[0], own, "n1")
    X = n["n1"].reshape(B, T, D)
    weights = [f64(inp[k]) for k in ("W_r", "W_dt", "b_dt", "A", "W_exp")]
    fl, forced = check_topk(idx.cpu().numpy(), S.router_logits(n["n1"], weights[0]), w.top_k)
    forced = forced.reshape(B, T, w.top_k) if fl.any() else None
    shape = (w.nheads, w.headdim, w.dstate, w.G, w.top_k)
    held(n["y"], S.layer_fwd(X, *weights, *shape, forced_idx=forced)["y"], layer, "y")
    held(n["p"], S.out_proj(n["y"], f64(inp["W_out"])), layer, "projection")
    n2, r = O.layer_norm(n["p"], num(x), num(g2), num(b2), eps)
    held(n["n2"], n2, own, "n2")
    held(n["r"], r, own, "r")
    gate, up, h, out = O.gated_ffn(n["n2"], num(wg), num(wu), num(wd), "silu")
    for k, ref in (("gate", gate), ("up", up), ("h", h), ("out", out)):
        held(n[k], ref, (2 if k == "out" else 1) * own, k)
    dn2 = O.gated_ffn_bwd(n["n2"], n["gate"], n["up"], n["h"], num(wg), num(wu), num(wd), num(dout), "silu")[0]
    held(n["dn2"], dn2, 2 * own, "dn2")
    dr, dg2, db2 = O.layer_norm_bwd(n["r"], num(g2), n["dn2"], num(dout), eps)
    held(n["dr"], dr, own, "dr")
    held(n["dg2"], dg2, 1e-5, "dg2")
    held(n["db2"], db2, 1e-5, "db2")
    held(n["dn1"], S.layer_bwd(X, *weights, *shape, num(dy).reshape(B, T, w.nheads, w.headdim), None, forced)["dX"], layer,
         "dn1")
    dx, dg1, db1 = O.layer_norm_bwd(num(x), num(g1), n["dn1"], None, eps)
    for k, ref in (("dx", dx), ("dg1", dg1), ("db1", db1)):
        held(n[k], ref, 1e-5, k)
