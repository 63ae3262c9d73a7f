"""The operators around the token mixer (layer norm, per-channel gated recurrence, gated feed-forward block) and
their gradients on the GPU, through the C ABI, against the fp64 oracle, element by element.

Tolerances are bounds, not fits.  u = 2^-24 is fp32's rounding; a tensor stored in type t is rounded once, by at
most half(t) = finfo(t).eps / 2 of its value.  A sum of n fp32 terms is off by at most (adds on its longest chain)
x u x (sum of magnitudes).  The functions named *_bound carry these through each formula.  A trailing factor 1.01
covers the second-order terms.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from parameter_space_moe_b200 import swimba

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": (swimba.F32, torch.float32), "bf16": (swimba.BF16, torch.bfloat16), "f16": (swimba.F16, torch.float16)}
SENTINEL = 1024.0


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the spacing of the type's subnormals."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def rand(rng, shape, dtype, scale=1.0, shift=0.0):
    """Values of the type on the GPU and the same values in fp64."""
    t = torch.from_numpy((rng.standard_normal(shape) * scale + shift).astype(np.float32)).to(dtype)
    return t.cuda(), t.double().numpy()


class Out:
    """An output tensor with 64 sentinels behind it."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape))
        self.all = torch.full((n + 64,), SENTINEL, dtype=dtype, device="cuda")
        self.all[:n] = float("nan")
        self.n, self.t = n, self.all[:n].view(*shape)

    def np(self):
        assert (self.all[self.n:].double() == SENTINEL).all(), "written past the end"
        return self.t.double().cpu().numpy()


def within(got, ref, bound, dtype, what):
    """|got - ref| <= bound + the one rounding to dtype, everywhere."""
    tol = 1.01 * (bound + half(dtype) * (np.abs(ref) + bound)) + tiny(dtype)
    off = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    worst = float((off / np.maximum(tol, 1e-300)).max())
    print(f"{what}: worst {worst:.3f} of its bound, norm-wise {np.linalg.norm(off) / max(np.linalg.norm(ref), 1e-300):.2e}")
    assert worst <= 1.0, what


def ok():
    assert swimba.check_device_status() == 0


# ------------------------------------------------------------------------------------------------ layer norm
# A row's sum has at most 32 adds in a thread, 5 in a warp and 15 over the block's warps (53 with the residual's one).
ROW_ADDS = 56


def norm_stats(r, eps):
    mu = r.mean(1, keepdims=True)
    rstd = 1 / np.sqrt(((r - mu) ** 2).mean(1, keepdims=True) + eps)
    xhat = (r - mu) * rstd
    # the mean is off by ROW_ADDS u mean|r|, an element's r by u |r|, and the difference is rounded once more
    dev = U * (ROW_ADDS * np.abs(r).mean(1, keepdims=True) + np.abs(r)) * rstd + U * np.abs(xhat)
    # rstd's relative error: half of the variance's (2 dev |xhat| in the mean, its sum, its square), rsqrt's 2 ulp
    rel = (dev * np.abs(xhat)).mean(1, keepdims=True) + U * (ROW_ADDS + 8)
    return xhat, rstd, dev + rel * np.abs(xhat), rel


def norm_bound(r, gamma, beta, eps):
    xhat, _, dxhat, _ = norm_stats(r, eps)
    g = 1.0 if gamma is None else np.abs(gamma)
    return dxhat * g + 3 * U * (np.abs(xhat) * g + (0 if beta is None else np.abs(beta)))


NORM_SHAPES = [(1, 1), (3, 8), (5, 33), (2, 64), (7, 255), (4, 768), (300, 768), (3, 1000), (2, 1001), (9, 2048), (2, 4096),
               (3, 5003), (2, 8192), (2, 8200), (2, 16384), (1, 16383),
               # enough rows for the layouts with more columns a thread, and columns that fill no layout
               (700, 2048), (600, 1001), (3, 5000), (601, 520)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,D", NORM_SHAPES)
def test_layer_norm(M, D, dt):
    code, t = TYPES[dt]
    rng = np.random.default_rng(M * D)
    x, xn = rand(rng, (M, D), t, 1.5, 0.7)
    res, rn = rand(rng, (M, D), t, 3.0, -0.4)
    gamma, gn = rand(rng, (D,), torch.float32, 0.3, 1.0)
    beta, bn = rand(rng, (D,), torch.float32, 0.3)
    d = swimba.norm_dims(M, D, code, eps=1e-5)
    y, r = Out((M, D), t), Out((M, D), t)
    swimba.layer_norm(d, x, res, gamma, beta, y.t, r.t)
    ok()
    ry, rr = O.layer_norm(xn, rn, gn, bn, float(np.float32(1e-5)))
    within(y.np(), ry, norm_bound(rr, gn, bn, 1e-5), t, f"y {M}x{D} {dt}")
    within(r.np(), rr, U * np.abs(rr), t, "r")
    # no residual, no parameters, no stored sum
    y = Out((M, D), t)
    swimba.layer_norm(d, x, None, None, None, y.t, None)
    ok()
    within(y.np(), O.layer_norm(xn, None, None, None, float(np.float32(1e-5)))[0], norm_bound(xn, None, None, 1e-5), t,
           "bare y")


@pytest.mark.parametrize("dt", TYPES)
def test_layer_norm_strided_rows_and_the_stream_in_place(dt):
    code, t = TYPES[dt]
    rng = np.random.default_rng(5)
    for M, D, stride in ((6, 96, 96 + 8), (5, 40, 41), (4, 33, 80)):
        wide, wn = rand(rng, (M, stride), t)
        x, xn = wide[:, :D], wn[:, :D]
        res, rn = rand(rng, (M, D), t, 2.0)
        y = Out((M, D), t)
        swimba.layer_norm(swimba.norm_dims(M, D, code, x_stride=stride), x, res, None, None, y.t, res)
        ok()
        ry, rr = O.layer_norm(xn, rn, None, None, float(np.float32(1e-5)))
        within(y.np(), ry, norm_bound(rr, None, None, 1e-5), t, "strided y")
        within(res.double().cpu().numpy(), rr, U * np.abs(rr), t, "stream in place")


def test_layer_norm_hard_rows():
    """A constant row gives beta; a row far from zero keeps its small deviations; NaN and infinity stay in their row."""
    D = 768
    x = torch.randn(6, D, device="cuda")
    x[1] = 7.25
    x[2] = 4096 + torch.randn(D, device="cuda") * 2
    x[3, 5] = float("nan")
    x[4, 9] = float("inf")
    y = Out((6, D), torch.float32)
    beta = torch.randn(D, device="cuda")
    swimba.layer_norm(swimba.norm_dims(6, D, swimba.F32), x, None, None, beta, y.t, None)
    ok()
    assert (y.all[6 * D:] == SENTINEL).all()
    got = y.t.double().cpu().numpy()
    rows = [0, 1, 2, 5]
    xn, bn = x[rows].double().cpu().numpy(), beta.double().cpu().numpy()
    # the constant row's sum is exact up to ROW_ADDS u 7.25, and rstd = eps^-1/2: the general bound covers it
    within(got[rows], O.layer_norm(xn, None, None, bn, float(np.float32(1e-5)))[0], norm_bound(xn, None, bn, 1e-5),
           torch.float32, "hard rows")
    assert np.isnan(got[3]).all() and np.isnan(got[4]).all()


def norm_bwd_bounds(r, gamma, dy, dr, eps):
    xhat, rstd, dxhat, rel = norm_stats(r, eps)
    ga = np.ones(r.shape[1]) if gamma is None else np.abs(gamma)
    g = np.abs(dy) * ga
    mean = lambda v: v.mean(1, keepdims=True)
    mg, mgx = mean(g), mean(g * np.abs(xhat))
    dmg, dmgx = U * (ROW_ADDS + 2) * mg, mean(g * dxhat) + U * (ROW_ADDS + 4) * mgx
    inner = g + mg + np.abs(xhat) * mgx
    bdx = rstd * (dmg + dxhat * mgx + np.abs(xhat) * dmgx + (4 * U + rel) * inner)
    if dr is not None:
        bdx = bdx + U * (np.abs(dr) + rstd * inner)
    # a column's sum: the rows of a block, then at most 37 partial sums in a thread and 32 threads
    adds = r.shape[0] / 148 + 1 + 37 + 32
    bdg = (np.abs(dy) * (dxhat + (adds + 1) * U * np.abs(xhat))).sum(0)
    return bdx, bdg, adds * U * np.abs(dy).sum(0)


@pytest.mark.parametrize("dt,gt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("M,D", NORM_SHAPES + [(2500, 96), (700, 768), (640, 760), (300, 223)])
def test_layer_norm_bwd(M, D, dt, gt):
    code, t = TYPES[dt]
    gcode, gty = TYPES[gt]
    rng = np.random.default_rng(M + D)
    r, rn = rand(rng, (M, D), t, 2.0, 0.5)
    gamma, gn = rand(rng, (D,), torch.float32, 0.3, 1.0)
    dy, dyn = rand(rng, (M, D), gty, 0.5)
    dr, drn = rand(rng, (M, D), gty, 0.5)
    d = swimba.norm_dims(M, D, code, gcode)
    ws = torch.empty(swimba.layer_norm_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    for use, use_n, gm, gm_n in ((dr, drn, gamma, gn), (None, None, None, None)):
        dx, dg, db = Out((M, D), gty), Out((D,), torch.float32), Out((D,), torch.float32)
        swimba.layer_norm_bwd(d, r, gm, dy, use, dx.t, dg.t, db.t, ws)
        ok()
        want = O.layer_norm_bwd(rn, gm_n, dyn, use_n, float(np.float32(1e-5)))
        bounds = norm_bwd_bounds(rn, gm_n, dyn, use_n, 1e-5)
        for o, w, b, ty, what in zip((dx, dg, db), want, bounds, (gty, torch.float32, torch.float32),
                                     ("dx", "dgamma", "dbeta")):
            within(o.np(), w, b, ty, f"{what} {M}x{D} {dt}/{gt}")
    # parameters' gradients left out, one of them left out, and the gradient in place
    db2 = Out((D,), torch.float32)
    swimba.layer_norm_bwd(d, r, None, dy, None, dy, None, db2.t, ws)
    ok()
    assert torch.equal(dy, dx.t) and torch.equal(db2.t, db.t)


# ------------------------------------------------------------------------------------------------ gated scan
def gate_error(gate):
    """Relative error of the smaller of f and 1 - f: the argument of exp2 (|g| u), exp2 and the quotient (2 ulp
    each), the sum; the larger one is the complement, off by as much in absolute terms and one rounding."""
    f, q = O.gates(gate)
    small = np.minimum(f, q)
    return U * (12 + np.abs(gate)) * small + U / 2


def scan_bound(a, values, da, b_err, scale):
    """Error of c_t = a_t c_{t-1} + b_t along axis 1 when a is off by da, b by b_err, and each step is rounded.  The
    composed maps add at most 8 roundings of the size `scale` a step."""
    e = np.zeros(a.shape[::2])
    out = np.empty_like(a)
    prev = np.zeros(a.shape[::2]) + scale
    for t in range(a.shape[1]):
        e = a[:, t] * e + da[:, t] * prev + b_err[:, t] + 8 * U * scale
        prev = np.maximum(np.abs(values[:, t]), scale)
        out[:, t] = e
    return out


SCAN_SHAPES = [(1, 1, 1), (2, 1, 64), (3, 5, 7), (1, 64, 32), (2, 65, 66), (1, 63, 33), (1, 700, 200), (4, 513, 96), (3, 1111, 333),
               (1, 2100, 2), (70, 3, 128), (1, 4097, 65), (2, 600, 1536),
               # few columns and many tokens: the largest clusters and the long rounds
               (1, 9001, 64), (3, 2500, 256), (1, 300, 4096)]


def scan_inputs(rng, B, T, W, t, cut):
    x, xn = rand(rng, (B, T, W), t)
    gate, gn = rand(rng, (B, T, W), t, 2.0, 1.5)
    if cut:  # halves of one projection's rows
        step = -(-W // 8) * 8
        both = torch.full((B, T, 2 * step), SENTINEL, dtype=t, device="cuda")
        both[..., :W], both[..., step:step + W] = x, gate
        x, gate = both[..., :W], both[..., step:step + W]
    return x, xn, gate, gn


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("B,T,W", SCAN_SHAPES)
@pytest.mark.parametrize("state,cut", [(True, False), (False, True)])
def test_gated_scan(B, T, W, dt, state, cut):
    code, t = TYPES[dt]
    rng = np.random.default_rng(B + T + W)
    x, xn, gate, gn = scan_inputs(rng, B, T, W, t, cut)
    init, inn = rand(rng, (B, W), torch.float32) if state else (None, None)
    h, fin = Out((B, T, W), t), Out((B, W), torch.float32)
    d = swimba.gated_dims(B, T, W, code, x_stride=x.stride(1) if cut else 0, gate_stride=gate.stride(1) if cut else 0)
    swimba.gated_scan(d, x, gate, init, h.t, fin.t)
    ok()
    want, last = O.gated_scan(xn, gn, inn)
    f, q = O.gates(gn)
    err, scale = gate_error(gn), max(1.0, np.abs(xn).max(), 0 if inn is None else np.abs(inn).max())
    bound = scan_bound(f, want, err, (err + 2 * U * q) * np.abs(xn), scale)
    within(h.np(), want, bound, t, f"h {B}x{T}x{W} {dt}")
    within(fin.np(), last, bound[:, -1], torch.float32, "final state")
    if state:  # the state continued in place gives the same
        keep = init.clone()
        swimba.gated_scan(d, x, gate, keep, h.t, keep)
        ok()
        assert torch.equal(keep, fin.t)


@pytest.mark.parametrize("dt,gt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("B,T,W", SCAN_SHAPES)
@pytest.mark.parametrize("state,cut", [(True, False), (False, True)])
def test_gated_scan_bwd(B, T, W, dt, gt, state, cut):
    code, t = TYPES[dt]
    gcode, gty = TYPES[gt]
    rng = np.random.default_rng(B * T + W)
    x, xn, gate, gn = scan_inputs(rng, B, T, W, t, cut)
    h, hn = rand(rng, (B, T, W), t, 0.5)
    dh, dhn = rand(rng, (B, T, W), gty, 0.5)
    init, inn = rand(rng, (B, W), torch.float32) if state else (None, None)
    dfin, dfn = rand(rng, (B, W), torch.float32) if state else (None, None)
    dx, dg, di = Out((B, T, W), gty), Out((B, T, W), gty), Out((B, W), torch.float32)
    d = swimba.gated_dims(B, T, W, code, gcode, x_stride=x.stride(1) if cut else 0,
                          gate_stride=gate.stride(1) if cut else 0)
    swimba.gated_scan_bwd(d, x, gate, h, init, dh, dfin, dx.t, dg.t, di.t)
    ok()
    wx, wg, wi = O.gated_scan_bwd(xn, gn, hn, inn, dhn, dfn)
    f, q = O.gates(gn)
    err = gate_error(gn)
    # the adjoint in reversed time, lam_t = dh_t + c, c <- f lam: memories of 1/(1-f) tokens sum up to
    # max|dh| / min(1 - f), bounded through the recurrence itself
    lam, e = (np.zeros((B, W)) if dfn is None else np.abs(dfn)), np.zeros((B, W))
    bx, bg = np.empty_like(xn), np.empty_like(xn)
    for s in range(T - 1, -1, -1):
        lam = lam + np.abs(dhn[:, s])
        e = e + 8 * U * lam
        before = (0 if inn is None else inn) if s == 0 else hn[:, s - 1]
        diff = np.abs(before - xn[:, s])
        rest = U * (np.abs(before) + np.abs(xn[:, s]))
        bx[:, s] = q[:, s] * e + (err[:, s] + 2 * U * q[:, s]) * lam
        bg[:, s] = f[:, s] * q[:, s] * (diff * e + lam * rest) + lam * diff * (err[:, s] * (f[:, s] + q[:, s])
                                                                               + 6 * U * f[:, s] * q[:, s])
        e = f[:, s] * e + err[:, s] * lam + U * lam
        lam = f[:, s] * lam
    within(dx.np(), wx, bx, gty, f"dx {B}x{T}x{W} {dt}/{gt}")
    within(dg.np(), wg, bg, gty, "dgate")
    within(di.np(), wi, e, torch.float32, "dinit")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("B,W", [(1, 1), (3, 7), (256, 128), (5, 1001), (2, 4096)])
def test_gated_step_is_a_scan_of_one_token(B, W, dt):
    code, t = TYPES[dt]
    rng = np.random.default_rng(W)
    init, _ = rand(rng, (B, W), torch.float32)
    x, _, gate, _ = scan_inputs(rng, B, 6, W, t, False)
    state = Out((B, W), torch.float32)
    state.t.copy_(init)
    hs = []
    for s in range(6):
        h = Out((B, 1, W), t)
        xs, gs = x[:, s:s + 1], gate[:, s:s + 1]       # rows 6 W apart
        if W % 8:
            xs, gs = xs.clone(), gs.clone()
        swimba.gated_step(swimba.gated_dims(B, 1, W, code, x_stride=xs.stride(0), gate_stride=gs.stride(0)), xs, gs, state.t,
                          h.t)
        h.np()
        hs.append(h.t)
    want, fin = torch.empty_like(x), torch.empty_like(init)
    swimba.gated_scan(swimba.gated_dims(B, 6, W, code), x, gate, init, want, fin)
    ok()
    state.np()
    # the same fp32 steps in the same order, but for one fused rounding of q x against f h + q x, and the maps'
    # composition: 8 u of the largest value a step
    scale = max(1.0, float(x.float().abs().max()), float(init.abs().max()))
    assert float((state.t - fin).abs().max()) <= 6 * 8 * U * scale
    got = torch.cat(hs, 1).double()
    assert bool(((got - want.double()).abs() <= 48 * U * scale + 2 * half(t) * want.double().abs() + tiny(t)).all())


def test_gated_scan_extreme_gates():
    """Gates of plus and minus infinity hold and replace the state; NaN stays in its channel.  A held state is the same
    bits within a warp's tokens; a later warp starts from the composed maps, (a2 a1) c + (a2 b1 + b2), where the one
    before applied them in turn, a2 (a1 c + b1) + b2: the two differ by their roundings, each within scan_bound of the
    exact value."""
    T, W = 300, 64
    x = torch.randn(1, T, W, device="cuda")
    gate = torch.randn(1, T, W, device="cuda")
    gate[:, 100:200, :8] = float("inf")
    gate[:, 150, 8:16] = -float("inf")
    gate[:, 40, 20] = float("nan")
    gate[:, :, 30], gate[:, :, 31] = 3.4e38, -3.4e38
    h = Out((1, T, W), torch.float32)
    init = torch.randn(1, W, device="cuda")
    swimba.gated_scan(swimba.gated_dims(1, T, W, swimba.F32), x, gate, init, h.t, None)
    ok()
    g = h.t[0]
    gn, xn, inn = (v[..., :8].double().cpu().numpy() for v in (gate, x, init))
    f, q = O.gates(gn)
    err = np.where(np.isinf(gn), 0.0, gate_error(np.where(np.isinf(gn), 0.0, gn)))
    e = scan_bound(f, O.gated_scan(xn, gn, inn)[0], err, (err + 2 * U * q) * np.abs(xn), np.abs(xn).max())
    held = (g[100:200, :8] - g[99, :8]).abs().double().cpu().numpy()
    assert (held <= e[0, 100:200] + e[0, 99]).all()
    assert torch.equal(g[150, 8:16], x[0, 150, 8:16])
    assert bool(torch.isnan(g[40:, 20]).all()) and bool(torch.isfinite(g[:40, 20]).all())
    others = [c for c in range(W) if c != 20]
    assert bool(torch.isfinite(g[:, others]).all())
    assert bool((g[:, 30] == init[0, 30]).all()) and torch.equal(g[:, 31], x[0, :, 31])


# ------------------------------------------------------------------------------------------------ feed-forward
FFN_SHAPES = [(1, 64, 128), (1, 8, 8), (3, 72, 40), (16, 256, 512), (17, 128, 264), (100, 320, 200), (128, 64, 64), (129, 200, 136),
              (300, 768, 2048), (257, 520, 1032),
              # tiles enough for CTA pairs in every product of one of the two, ragged in all three sizes
              (1500, 264, 2056), (5000, 520, 264)]
# longest chain of fp32 adds of a product over K: each of the K terms may be added one after the other, and the
# tensor cores may cut an addend's last bits instead of rounding them, 2 u a term
def dot_bound(a, b):
    return 2 * U * a.shape[1] * (np.abs(a) @ np.abs(b))


def ffn_inputs(M, D, F, t):
    rng = np.random.default_rng(M + D + F)
    x, xn = rand(rng, (M, D), t)
    wg, wgn = rand(rng, (F, D), t, D ** -0.5)
    wu, wun = rand(rng, (F, D), t, D ** -0.5)
    wd, wdn = rand(rng, (D, F), t, F ** -0.5)
    return rng, (x, wg, wu, wd), (xn, wgn, wun, wdn)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("M,D,F", FFN_SHAPES)
def test_gated_ffn(M, D, F, kind, dt):
    code, t = TYPES[dt]
    _, (x, wg, wu, wd), (xn, wgn, wun, wdn) = ffn_inputs(M, D, F, t)
    d = swimba.ffn_dims(M, D, F, code, swimba.SILU if kind == "silu" else swimba.GELU)
    ws = torch.empty(swimba.gated_ffn_workspace_size(d), dtype=torch.uint8, device="cuda")
    g, u, h, o = Out((M, F), t), Out((M, F), t), Out((M, F), t), Out((M, D), t)
    swimba.gated_ffn(d, x, wg, wu, wd, g.t, u.t, h.t, o.t, ws)
    ok()
    gate, up, hid, out = O.gated_ffn(xn, wgn, wun, wdn, kind)
    bg, bu = dot_bound(xn, wgn.T), dot_bound(xn, wun.T)
    act, slope = O.activation(gate, kind)
    # the activation's slope is at most 1.13; its own error 16 u of |gate| (exp, quotient, erf: 2 ulp each and
    # the argument's)
    bh = (1.13 * bg + 16 * U * np.abs(gate)) * (np.abs(up) + bu) + np.abs(act) * bu
    within(g.np(), gate, bg, t, f"gate {M}x{D}x{F} {dt}")
    within(u.np(), up, bu, t, "up")
    within(h.np(), hid, bh, t, "h")
    # the last product reads the rounded h
    bo = dot_bound(hid, wdn.T) + (bh + half(t) * (np.abs(hid) + bh) + tiny(t)) @ np.abs(wdn.T)
    within(o.np(), out, bo, t, "out")
    h2, o2 = Out((M, F), t), Out((M, D), t)          # gate and up not kept: the same values
    swimba.gated_ffn(d, x, wg, wu, wd, None, None, h2.t, o2.t, ws)
    ok()
    assert torch.equal(h2.t, h.t) and torch.equal(o2.t, o.t)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("M,D,F", FFN_SHAPES)
def test_gated_ffn_bwd(M, D, F, kind, dt):
    code, t = TYPES[dt]
    rng, (x, wg, wu, wd), (xn, wgn, wun, wdn) = ffn_inputs(M, D, F, t)
    gate, gn = rand(rng, (M, F), t)
    up, un = rand(rng, (M, F), t)
    h, hn = rand(rng, (M, F), t)
    dout, don = rand(rng, (M, D), t, 0.5)
    d = swimba.ffn_dims(M, D, F, code, swimba.SILU if kind == "silu" else swimba.GELU)
    ws = torch.empty(swimba.gated_ffn_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    dx, dwg, dwu, dwd = Out((M, D), t), Out((F, D), t), Out((F, D), t), Out((D, F), t)
    swimba.gated_ffn_bwd(d, x, gate, up, h, wg, wu, wd, dout, dx.t, dwg.t, dwu.t, dwd.t, ws)
    ok()
    want = O.gated_ffn_bwd(xn, gn, un, hn, wgn, wun, wdn, don, kind)
    act, slope = O.activation(gn, kind)
    dh, bdh = don @ wdn, dot_bound(don, wdn)
    dg, du = dh * un * slope, dh * act
    # dgate and dup: from dh's error, the activation's (16 u, its slope's terms 32 u), rounded once to the type
    bdg = bdh * np.abs(un * slope) + 32 * U * np.abs(dh * un) * (1 + np.abs(gn))
    bdu = bdh * np.abs(act) + 16 * U * np.abs(dh * gn)
    rdg, rdu = (b + half(t) * (np.abs(v) + b) + tiny(t) for v, b in ((dg, bdg), (du, bdu)))
    bx = (dot_bound(dg, wgn) + dot_bound(du, wun)) * 2 + rdg @ np.abs(wgn) + rdu @ np.abs(wun)
    bwg = dot_bound(dg.T, xn) + rdg.T @ np.abs(xn)
    bwu = dot_bound(du.T, xn) + rdu.T @ np.abs(xn)
    bwd = dot_bound(don.T, hn)
    for o, w, b, what in zip((dx, dwg, dwu, dwd), want, (bx, bwg, bwu, bwd), ("dx", "dw_gate", "dw_up", "dw_down")):
        within(o.np(), w, b, t, f"{what} {M}x{D}x{F} {kind} {dt}")


# ------------------------------------------------------------------------------------------------ together
class Stack:
    """A residual block of a recurrent model on the GPU: norm, gated recurrence, norm over the residual sum, gated
    feed-forward block; forward, and backward for an upstream gradient of the block's output sum."""

    def __init__(self, B, T, D, F, dt, seed):
        self.B, self.T, self.D, self.F = B, T, D, F
        self.code, self.t = TYPES[dt]
        rng = np.random.default_rng(seed)
        M = B * T
        self.host, dev = {}, {}
        for name, shape, ty, scale, shift in (
                ("x", (M, D), self.t, 1.0, 0.2), ("gate", (M, D), self.t, 1.5, 1.0), ("g1", (D,), torch.float32, 0.2, 1.0),
                ("b1", (D,), torch.float32, 0.2, 0.0), ("g2", (D,), torch.float32, 0.2, 1.0),
                ("b2", (D,), torch.float32, 0.2, 0.0), ("wg", (F, D), self.t, D ** -0.5, 0.0),
                ("wu", (F, D), self.t, D ** -0.5, 0.0), ("wd", (D, F), self.t, F ** -0.5, 0.0),
                ("dout", (M, D), self.t, 0.3, 0.0)):
            dev[name], self.host[name] = rand(rng, shape, ty, scale, shift)
        self.v = dev
        f32 = torch.float32
        new = lambda *s, ty=self.t: torch.empty(*s, dtype=ty, device="cuda")
        for name, shape, ty in (("n1", (M, D), None), ("h", (M, D), None), ("r", (M, D), None), ("n2", (M, D), None),
                                ("gt", (M, F), None), ("up", (M, F), None), ("hid", (M, F), None), ("out", (M, D), None),
                                ("dn2", (M, D), None), ("dr", (M, D), None), ("dn1", (M, D), None), ("dgate", (M, D), None),
                                ("dx", (M, D), None), ("dg1", (D,), f32), ("db1", (D,), f32), ("dg2", (D,), f32),
                                ("db2", (D,), f32), ("dwg", (F, D), None), ("dwu", (F, D), None), ("dwd", (D, F), None)):
            dev[name] = new(*shape, ty=ty or self.t)
        self.nd = swimba.norm_dims(M, D, self.code)
        self.gd = swimba.gated_dims(B, T, D, self.code)
        self.fd = swimba.ffn_dims(M, D, F, self.code)
        size = max(swimba.layer_norm_bwd_workspace_size(self.nd), swimba.gated_ffn_workspace_size(self.fd),
                   swimba.gated_ffn_bwd_workspace_size(self.fd))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        v, ws = self.v, self.ws
        swimba.layer_norm(self.nd, v["x"], None, v["g1"], v["b1"], v["n1"], None, stream=stream)
        swimba.gated_scan(self.gd, v["n1"], v["gate"], None, v["h"], None, stream=stream)
        swimba.layer_norm(self.nd, v["h"], v["x"], v["g2"], v["b2"], v["n2"], v["r"], stream=stream)
        swimba.gated_ffn(self.fd, v["n2"], v["wg"], v["wu"], v["wd"], v["gt"], v["up"], v["hid"], v["out"], ws, stream=stream)
        swimba.gated_ffn_bwd(self.fd, v["n2"], v["gt"], v["up"], v["hid"], v["wg"], v["wu"], v["wd"], v["dout"], v["dn2"],
                             v["dwg"], v["dwu"], v["dwd"], ws, stream=stream)
        # the sum out + r is the block's output: dout reaches r past the feed-forward block
        swimba.layer_norm_bwd(self.nd, v["r"], v["g2"], v["dn2"], v["dout"], v["dr"], v["dg2"], v["db2"], ws, stream=stream)
        swimba.gated_scan_bwd(self.gd, v["n1"], v["gate"], v["h"], None, v["dr"], None, v["dn1"], v["dgate"], None,
                              stream=stream)
        swimba.layer_norm_bwd(self.nd, v["x"], v["g1"], v["dn1"], v["dr"], v["dx"], v["dg1"], v["db1"], ws, stream=stream)

    OUT = ("out", "r", "dx", "dgate", "dg1", "db1", "dg2", "db2", "dwg", "dwu", "dwd")

    def oracle(self):
        v, B, T, D = self.host, self.B, self.T, self.D
        eps = float(np.float32(1e-5))
        seq = lambda a: a.reshape(B, T, D)
        n1, _ = O.layer_norm(v["x"], None, v["g1"], v["b1"], eps)
        h, _ = O.gated_scan(seq(n1), seq(v["gate"]), None)
        n2, r = O.layer_norm(h.reshape(-1, D), v["x"], v["g2"], v["b2"], eps)
        gt, up, hid, out = O.gated_ffn(n2, v["wg"], v["wu"], v["wd"], "silu")
        dn2, dwg, dwu, dwd = O.gated_ffn_bwd(n2, gt, up, hid, v["wg"], v["wu"], v["wd"], v["dout"], "silu")
        dr, dg2, db2 = O.layer_norm_bwd(r, v["g2"], dn2, v["dout"], eps)
        dn1, dgate, _ = O.gated_scan_bwd(seq(n1), seq(v["gate"]), h, None, seq(dr), None)
        dx, dg1, db1 = O.layer_norm_bwd(v["x"], v["g1"], dn1.reshape(-1, D), dr, eps)
        return dict(out=out, r=r, dx=dx, dgate=dgate.reshape(-1, D), dg1=dg1, db1=db1, dg2=dg2, db2=db2, dwg=dwg, dwu=dwu,
                    dwd=dwd)


@pytest.mark.parametrize("dt", TYPES)
def test_the_operators_together(dt):
    """Norm, recurrence, norm, feed-forward and all their gradients in a row against the oracle's row.  A value passes at
    most eight tensors of the type on its way (n1, h, r, n2, gate or h, dgate, dn2, dr, dn1), each rounding independent and
    at most half(t), and the norms and products keep relative sizes: eight half(t) norm-wise in 16 bits.  In fp32 the sums'
    roundings count besides: the layer's own bar of 1e-5."""
    s = Stack(2, 150, 96, 264, dt, 11)
    s.run()
    ok()
    want = s.oracle()
    for k in Stack.OUT:
        got = s.v[k].double().cpu().numpy()
        e = np.linalg.norm(got - want[k]) / np.linalg.norm(want[k])
        print(f"{k} {dt}: {e:.2e}")
        assert np.isfinite(got).all() and e <= (1e-5 if dt == "f32" else 8 * half(s.t)), k


def test_gradients_are_differences_of_the_gpu_forward():
    """The whole row in fp32: the change of sum <dout, out + r> along a direction of x, gate and the weights, taken from
    two forward runs on the GPU, against the gradients' product with that direction.  With step s the difference is off by
    the sums' fp32 errors (1e-6 of sum |dout out|, far above what they are) over 2 s and by the third derivative's s^2."""
    s = Stack(1, 40, 64, 128, "f32", 12)
    rng = np.random.default_rng(13)
    s.run()
    step, slope = 2.0 ** -7, 0.0
    grads = {"x": "dx", "gate": "dgate", "g1": "dg1", "g2": "dg2", "wg": "dwg", "wd": "dwd"}
    saved = {k: s.v[k].clone() for k in grads}
    got = {g: s.v[g].double().cpu().numpy() for g in grads.values()}
    for k in grads:
        direction = torch.from_numpy(rng.standard_normal(tuple(saved[k].shape)).astype(np.float32)).cuda()
        direction *= saved[k].double().square().mean().sqrt().float()
        vals = []
        for sign in (1, -1):
            s.v[k].copy_(saved[k] + sign * step * direction)
            s.run()
            vals.append(float((s.v["dout"].double() * (s.v["out"].double() + s.v["r"].double())).sum()))
        s.v[k].copy_(saved[k])
        moved = (saved[k] + step * direction).double() - (saved[k] - step * direction).double()   # as rounded
        slope = float((torch.from_numpy(got[grads[k]]).cuda().view_as(moved) * moved).sum())
        size = float((s.v["dout"].double() * s.v["out"].double()).abs().sum())
        print(k, vals[0] - vals[1], slope, size)
        # third derivative: each value moves by step of its size; s^2 = 6e-5 of the slope's own scale, taken as the root
        # of the number of terms times their size
        scale = float((torch.from_numpy(got[grads[k]]).cuda().view_as(moved) * moved).square().sum().sqrt())
        assert abs(vals[0] - vals[1] - slope) <= 1e-6 * size + 20 * step ** 2 * scale, k
    ok()


def test_streams_graphs_and_repeats():
    """The row on a stream of its own, captured and replayed on new inputs, and twice in a row: the same bits."""
    s = Stack(2, 200, 128, 256, "bf16", 14)
    s.run()
    ok()
    first = {k: s.v[k].clone() for k in Stack.OUT}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.run(stream=side)
    side.synchronize()
    for k in Stack.OUT:
        assert torch.equal(first[k], s.v[k]), k
    other = Stack(2, 200, 128, 256, "bf16", 15)
    other.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for k in ("x", "gate", "g1", "b1", "g2", "b2", "wg", "wu", "wd", "dout"):
        s.v[k].copy_(other.v[k])
    for _ in range(2):
        for k in Stack.OUT:
            s.v[k].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for k in Stack.OUT:
            assert torch.equal(other.v[k], s.v[k]), k
    ok()


def test_two_rows_at_once():
    """Two stacks with workspaces of their own on two streams at once give what each gives alone."""
    stacks = [Stack(2, 300, 128, 256, "bf16", 16 + i) for i in range(2)]
    want = []
    for s in stacks:
        s.run()
        torch.cuda.synchronize()
        want.append({k: s.v[k].clone() for k in Stack.OUT})
    streams = [torch.cuda.Stream() for _ in stacks]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, st in zip(stacks, streams):
            s.run(stream=st)
    torch.cuda.synchronize()
    ok()
    for s, w in zip(stacks, want):
        for k in Stack.OUT:
            assert torch.equal(w[k], s.v[k]), k


def test_the_binding_checks_its_tensors():
    """Wrong type, size, layout and a CPU tensor among GPU ones are refused before the library is called."""
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    d = swimba.norm_dims(8, 64, swimba.BF16)
    bad = [x.float(), x[:7], x.T, x.cpu(), torch.zeros(8, 128, dtype=torch.bfloat16, device="cuda")[:, :64]]
    f = swimba.ffn_dims(8, 64, 64, swimba.BF16)
    w = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    g = swimba.gated_dims(8, 1, 64, swimba.BF16)
    st = torch.zeros(8, 64, device="cuda")
    for b in bad:
        for go in (lambda: swimba.layer_norm(d, x, b, None, None, x, None),
                   lambda: swimba.layer_norm(d, b, None, None, None, x, None),
                   lambda: swimba.layer_norm_bwd(d, x, None, b, None, x, None, None, ws),
                   lambda: swimba.gated_step(g, x, x, b if b.dtype != torch.float32 else b[:7], x.clone()),
                   lambda: swimba.gated_step(g, x, b, st, x.clone()),
                   lambda: swimba.gated_scan(g, x, x, None, b, None),
                   lambda: swimba.gated_scan_bwd(g, x, x, x, None, b, None, x, x, None),
                   lambda: swimba.gated_ffn(f, b, w, w, w, None, None, x, x, ws),
                   lambda: swimba.gated_ffn(f, x, w, w, w, None, b, x, x, ws),
                   lambda: swimba.gated_ffn_bwd(f, x, x, x, x, w, w, w, b, x, w, w, w, ws)):
            with pytest.raises(swimba.SwimbaError) as e:
                go()
            assert e.value.code == 1
    for n in (0, 100):
        with pytest.raises(swimba.SwimbaError) as e:
            swimba.gated_ffn(f, x, w, w, w, None, None, x, x, ws[:n] if n else None)
        assert e.value.code == 4
    ok()


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last rows and tokens come out like a small call's on the same values."""
    D, M = 8192, 270000
    x = torch.zeros(M, D, dtype=torch.bfloat16, device="cuda")
    x[-4:] = torch.randn(4, D, device="cuda").bfloat16()
    y = torch.empty_like(x)
    swimba.layer_norm(swimba.norm_dims(M, D, swimba.BF16), x, None, None, None, y, None)
    ok()
    tail = x[-4:].double().cpu().numpy()
    within(y[-4:].double().cpu().numpy(), O.layer_norm(tail, None, None, None, float(np.float32(1e-5)))[0],
           norm_bound(tail, None, None, 1e-5), torch.bfloat16, "tail rows")
    assert float(y[:-4].float().abs().max()) == 0.0
    d = swimba.norm_dims(M, D, swimba.BF16)
    ws = torch.empty(swimba.layer_norm_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    dy = torch.zeros_like(x)
    dy[-4:] = torch.randn(4, D, device="cuda").bfloat16()
    dg = torch.empty(D, device="cuda")
    swimba.layer_norm_bwd(d, x, None, dy, None, y, dg, None, ws)
    ok()
    dyn = dy[-4:].double().cpu().numpy()
    dx, dgn, _ = O.layer_norm_bwd(tail, None, dyn, None, float(np.float32(1e-5)))
    bx, bg, _ = norm_bwd_bounds(tail, None, dyn, None, 1e-5)
    within(y[-4:].double().cpu().numpy(), dx, bx, torch.bfloat16, "tail gradients")
    within(dg.double().cpu().numpy(), dgn, bg, torch.float32, "dgamma")
    # one sequence of 2^31 + values as the recurrence: the last tokens, behind a closed gate, know nothing of the others
    B, T, W = 1, 540000, 4096
    gate = x.view(B, T, W)
    gate.zero_()
    gate[0, T - 40] = -float("inf")
    src = dy.view(B, T, W)
    src[0, -41:] = torch.randn(41, W, device="cuda").bfloat16()
    src[0, :-41] = 3.0
    out, fin = y.view(B, T, W), torch.empty(B, W, device="cuda")
    swimba.gated_scan(swimba.gated_dims(B, T, W, swimba.BF16), src, gate, None, out, fin)
    ok()
    want = torch.empty(B, 40, W, dtype=torch.bfloat16, device="cuda")
    last = torch.empty(B, W, device="cuda")
    swimba.gated_scan(swimba.gated_dims(B, 40, W, swimba.BF16), src[:, -40:].contiguous(), gate[:, -40:].contiguous(), None,
                      want, last)
    ok()
    # gates of 1/2 forget within 40 tokens; both sides' fp32 values are off by 8 u of the largest x a step, summed by the
    # gates to twice that, and h is rounded once on either side
    big = float(src[0, -40:].float().abs().max())
    assert float((fin - last).abs().max()) <= 2 * 2 * 8 * U * big
    a, b = out[:, -40:].double(), want.double()
    assert bool(((a - b).abs() <= 2 * half(torch.bfloat16) * b.abs() + 32 * U * big).all())
    assert bool((out[0, 1000:2000].float() == 3.0).all())
