"""Measured cases of the operators that stand around the token mixer in a recurrent language model: layer norm
(with the residual sum fused in), the per-channel gated linear recurrence (scan over a sequence, its gradients,
the single-token step) and the gated feed-forward block, each forward and backward.

listed() names the cases, draw() gives further ones of the same ranges, prepare() makes what a program holds
before the call, run() makes one pass, work() counts what a pass cannot do without, exact() computes the same
outputs in 64 bits.  With `own` false, run() uses elementary torch operations in 32 bits, rounded once at the
end; with `own` true it calls the library.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


def listed():
    return [
        # the norm in front of a decode step: one token of 256 sequences, added to the residual stream
        {"name": "norm_decode", "op": "norm", "rows": 256, "width": 2048, "dtype": "bf16", "residual": True},
        # the norm of a long prompt, the residual sum kept for the next block
        {"name": "norm_long", "op": "norm", "rows": 32768, "width": 2048, "dtype": "bf16", "residual": True},
        # training at the base layer's size: the gradient arrives in fp32, as the token mixer's gradients leave it
        {"name": "norm_bwd_base", "op": "norm_bwd", "rows": 8192, "width": 768, "dtype": "bf16", "grad": "f32",
         "residual": True},
        # an odd width in fp32 with a ragged number of rows, no residual branch
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 4099, "width": 1001, "dtype": "f32", "grad": "f32",
         "residual": False},
        # a training batch at the base layer's width (24 heads of 64)
        {"name": "scan_base", "op": "scan", "batch": 4, "seqlen": 2048, "width": 1536, "dtype": "bf16",
         "sliced": False, "state": False},
        # one long sequence continued from a state; x and gate are halves of one projection's output
        {"name": "scan_long", "op": "scan", "batch": 1, "seqlen": 32768, "width": 2048, "dtype": "bf16",
         "sliced": True, "state": True},
        {"name": "scan_bwd_base", "op": "scan_bwd", "batch": 4, "seqlen": 2048, "width": 1536, "dtype": "bf16",
         "grad": "bf16", "state": False},
        # odd sizes in fp32 with a state at both ends
        {"name": "scan_bwd_odd", "op": "scan_bwd", "batch": 3, "seqlen": 1111, "width": 333, "dtype": "f32",
         "grad": "f32", "state": True},
        # a decode step of 256 sequences
        {"name": "step_decode", "op": "step", "batch": 256, "width": 4096, "dtype": "bf16"},
        # the feed-forward block of a decode step: the weights' bytes bound it
        {"name": "ffn_decode", "op": "ffn", "rows": 256, "d_model": 2048, "d_ff": 5632, "dtype": "bf16",
         "act": "silu", "save": False},
        # a training forward at the base layer's tokens and width, gate and up kept for the gradients
        {"name": "ffn_base", "op": "ffn", "rows": 8192, "d_model": 768, "d_ff": 2048, "dtype": "bf16",
         "act": "silu", "save": True},
        # the gradients of a wide block
        {"name": "ffn_bwd_wide", "op": "ffn_bwd", "rows": 8192, "d_model": 2048, "d_ff": 5632, "dtype": "bf16",
         "act": "silu"},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "scan", "scan_bwd", "step", "ffn", "ffn_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    grad = rng.choice([dtype, "f32"])
    if op in ("norm", "norm_bwd"):
        width = _log_between(rng, 33, 8192)
        if rng.random() < 0.6:
            width = max(64, width // 8 * 8)
        rows = _log_between(rng, 1, min(32768, (1 << 26) // width // 2))
        case = {"op": op, "rows": rows, "width": width, "dtype": dtype, "residual": rng.random() < 0.5}
        return {**case, "grad": grad} if op == "norm_bwd" else case
    if op == "step":
        width = _log_between(rng, 33, 8192)
        return {"op": op, "batch": _log_between(rng, 1, (1 << 21) // width), "width": width, "dtype": dtype}
    if op in ("scan", "scan_bwd"):
        width = _log_between(rng, 33, 4096)
        if rng.random() < 0.6:
            width = max(64, width // 8 * 8)
        seqlen = _log_between(rng, 1, 32768)
        most = (1 << 26 if op == "scan" else 1 << 24) // 2
        seqlen = min(seqlen, most // width)
        batch = _log_between(rng, 1, max(1, min(64, most // (width * seqlen))))
        case = {"op": op, "batch": batch, "seqlen": seqlen, "width": width, "dtype": dtype,
                "state": rng.random() < 0.5}
        if op == "scan":
            return {**case, "sliced": width % 8 == 0 and rng.random() < 0.5}
        return {**case, "grad": grad}
    d_model, d_ff = _log_between(rng, 8, 256) * 8, _log_between(rng, 16, 704) * 8
    rows = _log_between(rng, 1, 8192 if dtype != "f32" else 2048)
    case = {"op": op, "rows": rows, "d_model": d_model, "d_ff": d_ff, "dtype": dtype,
            "act": rng.choice(["silu", "gelu"])}
    return {**case, "save": rng.random() < 0.5} if op == "ffn" else case


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    grad = TYPES[case.get("grad", case["dtype"])]
    op = case["op"]

    def normal(*shape, std=1.0, mean=0.0, to=dtype):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(to)

    def empty(*shape, to=dtype):
        return torch.empty(*shape, dtype=to, device="cuda")

    s = {"case": dict(case)}
    if op in ("norm", "norm_bwd"):
        M, D = case["rows"], case["width"]
        s["gamma"] = normal(D, std=0.2, mean=1.0, to=torch.float32)
        s["beta"] = normal(D, std=0.2, to=torch.float32)
        # the residual stream: channels of unequal scale around a mean that is not zero
        stream = normal(M, D, to=torch.float32) * (0.5 + 2 * torch.rand(D, generator=gen, device="cuda")) + 0.3
        if op == "norm":
            s["x"] = normal(M, D) if case["residual"] else stream.to(dtype)
            s["residual"] = stream.to(dtype) if case["residual"] else None
            s["y"], s["r"] = empty(M, D), empty(M, D) if case["residual"] else None
        else:
            s["r"] = stream.to(dtype)
            s["dy"] = normal(M, D, std=0.1, to=grad)
            s["dr"] = normal(M, D, std=0.1, to=grad) if case["residual"] else None
            s["dx"] = empty(M, D, to=grad)
            s["dgamma"], s["dbeta"] = empty(D, to=torch.float32), empty(D, to=torch.float32)
    elif op in ("scan", "scan_bwd", "step"):
        B, T, W = case["batch"], case.get("seqlen", 1), case["width"]
        # channels that remember for one token up to some hundreds
        bias = torch.rand(W, generator=gen, device="cuda") * 6 - 1
        if case.get("sliced"):
            both = empty(B, T, 2 * W)
            both[..., :W] = normal(B, T, W)
            both[..., W:] = normal(B, T, W, to=torch.float32) + bias
            s["x"], s["gate"] = both[..., :W], both[..., W:]
        else:
            s["x"] = normal(B, T, W)
            s["gate"] = (normal(B, T, W, to=torch.float32) + bias).to(dtype)
        f32 = torch.float32
        if op == "step":
            s["state"], s["h"] = normal(B, W, std=0.5, to=f32), empty(B, 1, W)
        else:
            s["init"] = normal(B, W, std=0.5, to=f32) if case["state"] else None
            if op == "scan":
                s["h"], s["final"] = empty(B, T, W), empty(B, W, to=f32) if case["state"] else None
            else:
                # the saved forward output: any values of its scale serve, the gradients are defined on them
                s["h"] = normal(B, T, W, std=0.4)
                s["dh"] = normal(B, T, W, std=0.1, to=grad)
                s["dfinal"] = normal(B, W, std=0.1, to=f32) if case["state"] else None
                s["dx"], s["dgate"] = empty(B, T, W, to=grad), empty(B, T, W, to=grad)
                s["dinit"] = empty(B, W, to=f32) if case["state"] else None
    else:
        M, D, F = case["rows"], case["d_model"], case["d_ff"]
        s["x"] = normal(M, D)
        s["w_gate"], s["w_up"] = normal(F, D, std=D ** -0.5), normal(F, D, std=D ** -0.5)
        s["w_down"] = normal(D, F, std=F ** -0.5)
        if op == "ffn":
            s["gate"] = empty(M, F) if case["save"] else None
            s["up"] = empty(M, F) if case["save"] else None
            s["h"], s["out"] = empty(M, F), empty(M, D)
        else:
            s["gate"], s["up"] = s["x"] @ s["w_gate"].T, s["x"] @ s["w_up"].T
            g = s["gate"].float()
            act = g * torch.sigmoid(g) if case["act"] == "silu" else 0.5 * g * (1 + torch.erf(g * 0.5 ** 0.5))
            s["h"] = (act * s["up"].float()).to(dtype)
            s["dout"] = normal(M, D, std=0.1)
            s["dx"] = empty(M, D)
            s["dw_gate"], s["dw_up"], s["dw_down"] = empty(F, D), empty(F, D), empty(D, F)
    return s


# ------------------------------------------------------------------------------------------ one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    """The calls of a user of the library; the dims and the workspace are made once and kept."""
    from parameter_space_moe_b200 import swimba
    c = s["case"]
    op = c["op"]
    code = {"f32": swimba.F32, "bf16": swimba.BF16, "f16": swimba.F16}
    if op in ("norm", "norm_bwd"):
        if "dims" not in s:
            s["dims"] = swimba.norm_dims(c["rows"], c["width"], code[c["dtype"]], code[c.get("grad", c["dtype"])],
                                         eps=EPS)
            if op == "norm_bwd":
                s["ws"] = torch.empty(swimba.layer_norm_bwd_workspace_size(s["dims"]), dtype=torch.uint8,
                                      device="cuda")
        if op == "norm":
            swimba.layer_norm(s["dims"], s["x"], s["residual"], s["gamma"], s["beta"], s["y"], s["r"])
            return {"y": s["y"], "r": s["r"]}
        swimba.layer_norm_bwd(s["dims"], s["r"], s["gamma"], s["dy"], s["dr"], s["dx"], s["dgamma"], s["dbeta"],
                              s["ws"])
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op in ("scan", "scan_bwd", "step"):
        if "dims" not in s:
            s["dims"] = swimba.gated_dims(c["batch"], c.get("seqlen", 1), c["width"], code[c["dtype"]],
                                          code[c.get("grad", c["dtype"])], x_stride=s["x"].stride(1),
                                          gate_stride=s["gate"].stride(1))
        if op == "step":
            swimba.gated_step(s["dims"], s["x"], s["gate"], s["state"], s["h"])
            return {"h": s["h"], "state": s["state"]}
        if op == "scan":
            swimba.gated_scan(s["dims"], s["x"], s["gate"], s["init"], s["h"], s["final"])
            return {"h": s["h"], "final": s["final"]}
        swimba.gated_scan_bwd(s["dims"], s["x"], s["gate"], s["h"], s["init"], s["dh"], s["dfinal"], s["dx"],
                              s["dgate"], s["dinit"])
        return {"dx": s["dx"], "dgate": s["dgate"], "dinit": s["dinit"]}
    if "dims" not in s:
        s["dims"] = swimba.ffn_dims(c["rows"], c["d_model"], c["d_ff"], code[c["dtype"]],
                                    {"silu": swimba.SILU, "gelu": swimba.GELU}[c["act"]])
        size = swimba.gated_ffn_workspace_size if op == "ffn" else swimba.gated_ffn_bwd_workspace_size
        s["ws"] = torch.empty(size(s["dims"]), dtype=torch.uint8, device="cuda")
    if op == "ffn":
        swimba.gated_ffn(s["dims"], s["x"], s["w_gate"], s["w_up"], s["w_down"], s["gate"], s["up"], s["h"],
                         s["out"], s["ws"])
        return {"out": s["out"], "h": s["h"], "gate": s["gate"], "up": s["up"]}
    swimba.gated_ffn_bwd(s["dims"], s["x"], s["gate"], s["up"], s["h"], s["w_gate"], s["w_up"], s["w_down"],
                         s["dout"], s["dx"], s["dw_gate"], s["dw_up"], s["dw_down"], s["ws"])
    return {"dx": s["dx"], "dw_gate": s["dw_gate"], "dw_up": s["dw_up"], "dw_down": s["dw_down"]}


def _scan(a, b):
    """All h_t = a_t h_{t-1} + b_t along dim 1 from h = 0, by doubling the reach of each pass."""
    reach = 1
    while reach < a.shape[1]:
        b = torch.cat((b[:, :reach], b[:, reach:] + a[:, reach:] * b[:, :-reach]), 1)
        if 2 * reach < a.shape[1]:
            a = torch.cat((a[:, :reach], a[:, reach:] * a[:, :-reach]), 1)
        reach *= 2
    return b


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        sg = torch.sigmoid(g)
        return g * sg, sg * (1 + g * (1 - sg))
    cdf = 0.5 * (1 + torch.erf(g * 0.5 ** 0.5))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5


def _plain(s):
    c = s["case"]
    op, dtype, grad = c["op"], TYPES[c["dtype"]], TYPES[c.get("grad", c["dtype"])]
    if op == "norm":
        r = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
        centred = r - r.mean(-1, keepdim=True)
        y = centred * torch.rsqrt((centred * centred).mean(-1, keepdim=True) + EPS) * s["gamma"] + s["beta"]
        return {"y": y.to(dtype), "r": None if s["residual"] is None else r.to(dtype)}
    if op == "norm_bwd":
        r, dy = s["r"].float(), s["dy"].float()
        centred = r - r.mean(-1, keepdim=True)
        rstd = torch.rsqrt((centred * centred).mean(-1, keepdim=True) + EPS)
        xhat, g = centred * rstd, dy * s["gamma"]
        dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
        if s["dr"] is not None:
            dx = dx + s["dr"].float()
        return {"dx": dx.to(grad), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}
    if op == "step":
        f = torch.sigmoid(s["gate"][:, 0].float())
        s["state"].copy_(f * s["state"] + torch.sigmoid(-s["gate"][:, 0].float()) * s["x"][:, 0].float())
        return {"h": s["state"].to(dtype)[:, None], "state": s["state"]}
    if op == "scan":
        gate = s["gate"].float()
        f, b = torch.sigmoid(gate), torch.sigmoid(-gate) * s["x"].float()
        if s["init"] is not None:
            b[:, 0] += f[:, 0] * s["init"]
        h = _scan(f, b)
        return {"h": h.to(dtype), "final": h[:, -1].clone() if s["init"] is not None else None}
    if op == "scan_bwd":
        gate, x, h = s["gate"].float(), s["x"].float(), s["h"].float()
        f, q, lam = torch.sigmoid(gate), torch.sigmoid(-gate), s["dh"].float().clone()
        first = torch.zeros_like(h[:, 0]) if s["init"] is None else s["init"]
        if s["dfinal"] is not None:
            lam[:, -1] += s["dfinal"]
        # the adjoint runs backwards and decays by the following token's gate
        lam = _scan(torch.cat((f[:, :1], f.flip(1)[:, :-1]), 1), lam.flip(1)).flip(1)
        before = torch.cat((first[:, None], h[:, :-1]), 1)
        return {"dx": (q * lam).to(grad), "dgate": (lam * (before - x) * f * q).to(grad),
                "dinit": f[:, 0] * lam[:, 0] if s["init"] is not None else None}
    wg, wu, wd = s["w_gate"].float(), s["w_up"].float(), s["w_down"].float()
    x = s["x"].float()
    if op == "ffn":
        gate, up = x @ wg.T, x @ wu.T
        h = _act(gate, c["act"])[0] * up
        out = h @ wd.T
        return {"out": out.to(dtype), "h": h.to(dtype), "gate": gate.to(dtype) if c["save"] else None,
                "up": up.to(dtype) if c["save"] else None}
    dout, up = s["dout"].float(), s["up"].float()
    act, slope = _act(s["gate"].float(), c["act"])
    dh = dout @ wd
    dgate, dup = dh * up * slope, dh * act
    return {"dx": (dgate @ wg + dup @ wu).to(dtype), "dw_gate": (dgate.T @ x).to(dtype),
            "dw_up": (dup.T @ x).to(dtype), "dw_down": (dout.T @ s["h"].float()).to(dtype)}


# ------------------------------------------------------------------------------------------ what it needs

def work(case):
    e = {"f32": 4, "bf16": 2, "f16": 2}[case["dtype"]]
    ge = {"f32": 4, "bf16": 2, "f16": 2}[case.get("grad", case["dtype"])]
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, D = case["rows"] * case["width"], case["width"]
        if op == "norm":
            return {"bytes": n * e * (4 if case["residual"] else 2) + 8 * D, "flops": 8 * n}
        return {"bytes": n * (e + (3 if case["residual"] else 2) * ge) + 12 * D, "flops": 16 * n}
    if op == "step":
        n = case["batch"] * case["width"]
        return {"bytes": n * (3 * e + 8), "flops": 8 * n}
    if op in ("scan", "scan_bwd"):
        n, ends = case["batch"] * case["seqlen"] * case["width"], 4 * case["batch"] * case["width"]
        if op == "scan":
            return {"bytes": n * 3 * e + (2 * ends if case["state"] else 0), "flops": 8 * n}
        return {"bytes": n * (3 * e + 3 * ge) + (3 * ends if case["state"] else 0), "flops": 14 * n}
    M, D, F = case["rows"], case["d_model"], case["d_ff"]
    if op == "ffn":
        # x and the weights in; h, out and, where they are kept, gate and up out
        return {"bytes": e * (2 * M * D + 3 * F * D + (3 if case["save"] else 1) * M * F), "flops": 6 * M * D * F}
    return {"bytes": e * (3 * M * D + 6 * F * D + 3 * M * F), "flops": 12 * M * D * F}


# ------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in prepare(case, seed).items()}
    op = case["op"]
    if op == "norm":
        r = s["x"] + (s["residual"] if case["residual"] else 0)
        var, mean = torch.var_mean(r, dim=1, correction=0)
        y = (r - mean[:, None]) / torch.sqrt(var + EPS)[:, None]
        return {"y": torch.addcmul(s["beta"], y, s["gamma"]), "r": r if case["residual"] else None}
    if op == "norm_bwd":
        r = s["r"]
        var, mean = torch.var_mean(r, dim=1, correction=0)
        sd = torch.sqrt(var + EPS)
        xhat = (r - mean[:, None]) / sd[:, None]
        g = s["dy"] * s["gamma"]
        D = case["width"]
        dot = torch.einsum("md,md->m", g, xhat)
        dx = (D * g - g.sum(1)[:, None] - xhat * dot[:, None]) / (D * sd)[:, None]
        return {"dx": dx + (s["dr"] if case["residual"] else 0),
                "dgamma": torch.einsum("md,md->d", s["dy"], xhat), "dbeta": s["dy"].sum(0)}
    if op in ("scan", "scan_bwd", "step"):
        f = 1 / (1 + torch.exp(-s["gate"]))
        q = 1 / (1 + torch.exp(s["gate"]))
        if op == "step":
            h = torch.lerp(s["x"][:, 0], s["state"], f[:, 0])
            return {"h": h[:, None], "state": h}
        T = case["seqlen"]
        if op == "scan":
            h = torch.zeros_like(f[:, 0]) if s["init"] is None else s["init"]
            out, b = torch.empty_like(f), q * s["x"]
            for t in range(T):
                h = torch.addcmul(b[:, t], f[:, t], h)
                out[:, t] = h
            return {"h": out, "final": h if case["state"] else None}
        lam = torch.zeros_like(f[:, 0]) if s["dfinal"] is None else s["dfinal"]
        adj = torch.empty_like(f)
        for t in range(T - 1, -1, -1):
            adj[:, t] = lam + s["dh"][:, t]
            lam = f[:, t] * adj[:, t]
        before = torch.roll(s["h"], 1, 1)
        before[:, 0] = 0 if s["init"] is None else s["init"]
        return {"dx": q * adj, "dgate": adj * f * q * (before - s["x"]), "dinit": lam if case["state"] else None}
    inner = torch.nn.functional
    if op == "ffn":
        gate, up = inner.linear(s["x"], s["w_gate"]), inner.linear(s["x"], s["w_up"])
        h = (inner.silu(gate) if case["act"] == "silu" else inner.gelu(gate)) * up
        return {"out": inner.linear(h, s["w_down"]), "h": h, "gate": gate if case["save"] else None,
                "up": up if case["save"] else None}
    gate, up = s["gate"].requires_grad_(), s["up"].requires_grad_()
    with torch.enable_grad():
        h = (inner.silu(gate) if case["act"] == "silu" else inner.gelu(gate)) * up
        dgate, dup = torch.autograd.grad(h, (gate, up), torch.matmul(s["dout"], s["w_down"]))
    return {"dx": torch.addmm(dgate @ s["w_gate"], dup, s["w_up"]), "dw_gate": torch.mm(dgate.t(), s["x"]),
            "dw_up": torch.mm(dup.t(), s["x"]), "dw_down": torch.mm(s["dout"].t(), s["h"])}
