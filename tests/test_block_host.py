"""Host-side checks of the operators around the token mixer (no GPU needed): workspaces are sized, and invalid or
unsupported arguments are refused by the C ABI before anything is launched and by the binding before it calls."""
import ctypes
import math

import pytest
import torch

from parameter_space_moe_b200 import swimba

FAKE = 1 << 20      # aligned, never dereferenced: validation fails first
ODD = FAKE + 4


@pytest.fixture(scope="module")
def L():
    try:
        return swimba.lib()
    except OSError:
        import __graft_entry__
        __graft_entry__.build()
        return swimba.lib()


def norm(**kw):
    d = swimba.norm_dims(8, 64, swimba.BF16)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def gated(**kw):
    d = swimba.gated_dims(2, 1, 64, swimba.BF16)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def ffn(**kw):
    d = swimba.ffn_dims(8, 64, 128, swimba.BF16)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


BIG = 1 << 40


def call(L, name, d, miss=None, at=FAKE, ws_bytes=BIG):
    """Calls entry point `name` with every pointer FAKE but argument `miss`, which is `at`."""
    n = {"layer_norm": 6, "layer_norm_bwd": 8, "gated_scan": 5, "gated_scan_bwd": 9, "gated_step": 4, "gated_ffn": 9,
         "gated_ffn_bwd": 13}[name]
    args = [FAKE] * n
    if miss is not None:
        args[miss] = at
    if name in ("layer_norm_bwd", "gated_ffn", "gated_ffn_bwd"):
        args.append(ws_bytes)
    return getattr(L, f"swimba_{name}")(d, *args, None)


OPS = {"layer_norm": norm, "layer_norm_bwd": norm, "gated_scan": gated, "gated_scan_bwd": gated, "gated_step": gated,
       "gated_ffn": ffn, "gated_ffn_bwd": ffn}
OPTIONAL = {"layer_norm": {1, 2, 3, 5}, "layer_norm_bwd": {1, 3, 5, 6}, "gated_scan": {2, 4},
            "gated_scan_bwd": {3, 5, 8}, "gated_step": set(), "gated_ffn": {4, 5}, "gated_ffn_bwd": set()}
WORKSPACE = {"layer_norm_bwd": 7, "gated_ffn": 8, "gated_ffn_bwd": 12}


@pytest.mark.parametrize("name", OPS)
def test_pointers(L, name):
    """Misaligned pointers are refused everywhere, null ones where they are not optional, the workspace with its
    own code; null dims too."""
    d = OPS[name]()
    n = {"layer_norm": 6, "layer_norm_bwd": 8, "gated_scan": 5, "gated_scan_bwd": 9, "gated_step": 4, "gated_ffn": 9,
         "gated_ffn_bwd": 13}[name]
    for i in range(n):
        if i == WORKSPACE.get(name):
            assert call(L, name, d, i, ODD) == 4 and call(L, name, d, i, None) == 4
            continue
        assert call(L, name, d, i, ODD) == 1, i
        if i not in OPTIONAL[name]:
            assert call(L, name, d, i, None) == 1, i
    if name in WORKSPACE:
        need = getattr(swimba, f"{name}_workspace_size")(d)
        assert need > 0 and call(L, name, d, ws_bytes=need - 1) == 4
    assert call(L, name, None) == 1


@pytest.mark.parametrize("name,kw,code", [
    *[("layer_norm", kw, 1) for kw in (dict(rows=0), dict(rows=-1), dict(width=0), dict(dtype=3), dict(dtype=-1),
                                       dict(grad_dtype=swimba.F16), dict(eps=0.0), dict(eps=-1.0),
                                       dict(eps=math.nan), dict(eps=math.inf), dict(x_stride=63),
                                       dict(x_stride=-64))],
    ("layer_norm", dict(width=16385), 2), ("layer_norm", dict(x_stride=1 << 31), 2),
    ("layer_norm", dict(rows=(1 << 30) + 1), 2),
    *[("gated_scan", kw, 1) for kw in (dict(batch=0), dict(seqlen=0), dict(seqlen=-5), dict(width=0), dict(dtype=7),
                                       dict(grad_dtype=swimba.F16), dict(x_stride=1), dict(gate_stride=63))],
    ("gated_scan", dict(batch=1 << 20, seqlen=1 << 20), 2), ("gated_scan", dict(batch=1 << 20, width=1 << 14), 2),
    ("gated_scan", dict(gate_stride=1 << 31), 2), ("gated_step", dict(seqlen=2), 1),
    *[("gated_ffn", kw, 1) for kw in (dict(rows=0), dict(d_model=0), dict(d_ff=-8), dict(dtype=5),
                                      dict(activation=2), dict(activation=-1))],
    *[("gated_ffn", kw, 2) for kw in (dict(d_model=60), dict(d_ff=132), dict(dtype=swimba.F32, d_ff=126),
                                      dict(d_ff=(1 << 20) + 8), dict(rows=(1 << 24) + 1),
                                      dict(dtype=swimba.F32, d_model=68), dict(rows=1 << 24, d_ff=1 << 20),
                                      dict(d_model=1 << 20, d_ff=1 << 20))],
])
def test_dims(L, name, kw, code):
    d = OPS[name](**kw)
    for n in (name, name + "_bwd"):
        if n in OPS:
            assert call(L, n, d) == code
            if n in WORKSPACE:
                assert getattr(swimba, f"{n}_workspace_size")(d) == 0


def test_workspace_sizes(L):
    """The norm's gradients keep partial sums of both parameters; the block's keep dgate and dup."""
    assert swimba.layer_norm_bwd_workspace_size(norm(rows=1, width=768)) >= 2 * 768 * 4
    small, large = (swimba.layer_norm_bwd_workspace_size(norm(rows=r, width=768)) for r in (100, 1 << 20))
    assert small <= large == swimba.layer_norm_bwd_workspace_size(norm(rows=1 << 21, width=768))
    assert swimba.gated_ffn_bwd_workspace_size(ffn()) >= 2 * 8 * 128 * 2
    assert swimba.gated_ffn_workspace_size(ffn()) > 0


def test_fp32_workspaces_hold_the_planes(L):
    """fp32 tensors of the block are split into three bf16 planes in the workspace: 6 bytes a value."""
    M, D, F = 100, 64, 128
    d = ffn(rows=M, dtype=swimba.F32)
    assert swimba.gated_ffn_workspace_size(d) >= 6 * (M * D + 3 * F * D + M * F)
    assert swimba.gated_ffn_bwd_workspace_size(d) >= 8 * M * F + 6 * (2 * M * D + 3 * F * D + 3 * M * F)


def test_the_binding_refuses_tensors_off_the_gpu():
    t = torch.zeros(8, 64, dtype=torch.bfloat16)
    for go in (lambda: swimba.layer_norm(norm(), t, None, None, None, t, None),
               lambda: swimba.layer_norm_bwd(norm(), t, None, t, None, t, None, None, None),
               lambda: swimba.gated_scan(gated(), t, t, None, t, None),
               lambda: swimba.gated_scan_bwd(gated(), t, t, t, None, t, None, t, t, None),
               lambda: swimba.gated_step(gated(), t, t, t, t),
               lambda: swimba.gated_ffn(ffn(), t, t, t, t, None, None, t, t, None),
               lambda: swimba.gated_ffn_bwd(ffn(), t, t, t, t, t, t, t, t, t, t, t, t, None),
               lambda: swimba.layer_norm(norm(), None, None, None, None, t, None)):
        with pytest.raises(swimba.SwimbaError) as e:
            go()
        assert e.value.code == 1


def test_row_strides():
    """The binding's check of strided rows, on CPU tensors standing for device ones (device -1 on both sides)."""
    both = torch.zeros(2, 5, 96)
    rows = lambda t, stride, m=10, w=48: swimba._rows("f", -1, m, w, stride, torch.float32, t)
    assert rows(both[..., :48], 96) == both.data_ptr()
    assert rows(both[..., 48:], 96) == both.data_ptr() + 48 * 4
    assert rows(torch.zeros(10, 48), 0) and rows(torch.zeros(2, 5, 48), 48)
    one = torch.zeros(1, 48)
    assert rows(one, 96, m=1)                                           # one row: no stride to check
    for t, stride in ((both[..., :48], 0), (both[..., :48], 48), (both[..., :48], 192), (both[..., ::2], 96),
                      (torch.zeros(10, 48), 96), (torch.zeros(2, 6, 96)[:, :5, :48], 96),
                      (torch.zeros(48, 10).T, 0), (torch.zeros(10, 47), 0), (torch.zeros(5, 96), 0)):
        with pytest.raises(swimba.SwimbaError):
            rows(t, stride)
