"""moe_residual_norm, its gradient and moe_combine_residual_norm against the 64-bit oracle.

Bounds: u = eps/2 of the stored type, v = 2^-24.  A row's sum of squares has at
most 64 addends in a lane, 6 steps over the lanes and 16 over the waves: its
relative error is below 90 v, that of 1/rms below half of it and 4 v more; two
products bring p to 52 v of itself.  The three sums of the backward have the
same shape, up to 100 v of the sum of their addends' absolute values, with up
to 8 roundings in an addend; c1, c2 and the last combination stay below 16
more: 128 v of everything that is added.  Sums over the tokens: at most
T / 256 + 1 rows in a lane, 192 blocks in a wave and 16 waves.
"""
import numpy as np
import pytest
import torch

from mixture_experts_layer_03_amd import abi
from oracle import around_block as O

pytestmark = pytest.mark.gpu
V = O.U32
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda:0"


def _u(dt):
    return torch.finfo(dt).eps / 2


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _rand(g, *shape, dt=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dt).to(DEV)


def _inputs(T, d, dt, post, pre, gate, seed):
    g = torch.Generator().manual_seed(seed)
    x, y = _rand(g, T, d, dt=dt), _rand(g, T, d, dt=dt, scale=3.0)
    wp = (1 + 0.3 * torch.randn(d, generator=g)).to(dt).to(DEV) if post else None
    wn = (1 + 0.3 * torch.randn(d, generator=g)).to(dt).to(DEV) if pre else None
    gt = {"none": None, "channel": _rand(g, d, dt=dt), "token": _rand(g, T, 1),
          "element": _rand(g, T, d, dt=dt)}[gate]
    return g, x, y, wp, wn, gt


def _close(name, got, ref, tol):
    got = _np(got)
    assert got.shape == ref.shape, name
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g over %.3g" % (
        name, bad.sum(), bad.size, np.abs(got - ref)[bad].max(), np.broadcast_to(tol, bad.shape)[bad].min())


# d: one piece, a part of a wave, several waves, past 512, 1024 and 2048 pieces, the largest
SHAPES = [(1, 8), (2055, 72), (2500, 776), (2049, 1544), (2048, 2056), (3, 64), (5, 520), (7, 2880), (2, 4104), (3, 8200), (2, 16384), (2051, 1032), (2049, 2880), (2050, 4096)]


def _check_forward(x, y, out, n, rp, rn, wp, wn, gt, scale, eps):
    dt = out.dtype
    ref, _, rrp, _, size = O.residual_norm(_np(x), _np(y), _np(wp), None, _np(gt), scale, eps, None)
    _close("out", out, ref, _u(dt) * abs(ref) * 1.01 + 56 * V * size)
    if wp is not None:
        _close("rstd_post", rp, rrp[:, 0], 50 * V * rrp[:, 0])
    if wn is not None:
        o = _np(out)
        r = O.rstd(o, eps)
        _close("rstd_pre", rn, r[:, 0], 50 * V * r[:, 0])
        ref = o * r * _np(wn)
        _close("n", n, ref, (_u(dt) * 1.01 + 52 * V) * abs(ref))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("post,pre,gate", [(True, True, "none"), (True, True, "channel"), (False, True, "token"),
                                           (True, False, "element"), (True, True, "token"), (False, False, "channel")])
def test_forward(T, d, dtype, post, pre, gate):
    dt = DT[dtype]
    _, x, y, wp, wn, gt = _inputs(T, d, dt, post, pre, gate, T + d)
    out, n = torch.empty_like(x), torch.empty_like(x) if pre else None
    rp = torch.empty(T, device=DEV) if post else None
    rn = torch.empty(T, device=DEV) if pre else None
    abi.moe_residual_norm(x, y, out, n, wp, wn, gt, 0.75, 1e-5, rp, rn)
    _check_forward(x, y, out, n, rp, rn, wp, wn, gt, 0.75, 1e-5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("post,pre,gate", [(True, True, "none"), (True, True, "channel"), (False, True, "token"),
                                           (True, False, "element"), (True, True, "token"), (False, True, "channel"),
                                           (True, True, "element")])
def test_backward(T, d, dtype, post, pre, gate):
    dt = DT[dtype]
    g, o, y, wp, wn, gt = _inputs(T, d, dt, post, pre, gate, T + d + 1)
    d_out, d_n = _rand(g, T, d, dt=dt), _rand(g, T, d, dt=dt) if pre else None
    rp = torch.tensor(O.rstd(_np(y), 1e-5)[:, 0]).float().to(DEV) if post else None
    rn = torch.tensor(O.rstd(_np(o), 1e-5)[:, 0]).float().to(DEV) if pre else None
    d_x, d_y = torch.empty_like(o), torch.empty_like(o)
    dwp = torch.empty(d, device=DEV) if post else None
    dwn = torch.empty(d, device=DEV) if pre else None
    dg = None if gt is None else torch.empty_like(gt, dtype=torch.float32 if gate == "channel" else gt.dtype)
    ws = torch.empty(abi.moe_residual_norm_bwd_workspace_size(T, d), dtype=torch.uint8, device=DEV)
    call = lambda: abi.moe_residual_norm_bwd(d_out, d_n, o, y, d_x, d_y, ws, wp, wn, gt, 0.75, rp, rn, dwp, dwn, dg)
    call()
    col = lambda t: None if t is None else _np(t)[:, None]
    ref = O.residual_norm_bwd(_np(d_out), _np(d_n), _np(o), _np(y), _np(wp), _np(wn), _np(gt), 0.75, col(rp), col(rn))
    got = {"d_x": d_x, "d_y": d_y, "d_w_post": dwp, "d_w_pre": dwn, "d_gate": dg}
    assert {n for n, t in got.items() if t is not None} == set(ref)
    over_t = T / 256 + 1 + 3072 / 16 + 16
    for name, (v, size) in ref.items():
        t = got[name]
        sums = over_t if name.startswith("d_w") or (name == "d_gate" and gate == "channel") else 0
        _close(name, t.view(v.shape), v, (_u(t.dtype) * 1.01 if t.dtype == torch.bfloat16 else V) * abs(v) + (128 + sums) * V * size)
    first = {n: t.clone() for n, t in got.items() if t is not None}
    call()
    for n, t in first.items():
        assert torch.equal(t, got[n]), n       # fixed order of sums


def test_gradients_against_differences():
    """The whole operator's gradients, fp32, by central differences of the 64-bit forward."""
    T, d, eps, scale = 3, 24, 1e-5, 0.5
    for gate in ("channel", "token", "element"):
        g, x, y, wp, wn, gt = _inputs(T, d, torch.float32, True, True, gate, 5)
        out, n = torch.empty_like(x), torch.empty_like(x)
        rp, rn = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        abi.moe_residual_norm(x, y, out, n, wp, wn, gt, scale, eps, rp, rn)
        go, gn = _rand(g, T, d), _rand(g, T, d)
        grads = {"x": torch.empty_like(x), "y": torch.empty_like(x), "wp": torch.empty_like(wp), "wn": torch.empty_like(wn),
                 "gt": torch.empty_like(gt)}
        ws = torch.empty(abi.moe_residual_norm_bwd_workspace_size(T, d), dtype=torch.uint8, device=DEV)
        abi.moe_residual_norm_bwd(go, gn, out, y, grads["x"], grads["y"], ws, wp, wn, gt, scale, rp, rn,
                                  grads["wp"], grads["wn"], grads["gt"])
        a = {"x": _np(x), "y": _np(y), "wp": _np(wp), "wn": _np(wn), "gt": _np(gt)}

        def loss(a):
            o, nn, *_ = O.residual_norm(a["x"], a["y"], a["wp"], a["wn"], a["gt"], scale, eps, lambda v: v)
            return (o * _np(go)).sum() + (nn * _np(gn)).sum()

        h = 1e-5   # the third derivative's share, h^2, and the sum's rounding, 1e-16 * 100 / h, are below 1e-8
        for name, t in grads.items():
            want = np.zeros_like(a[name])
            for i in np.ndindex(want.shape):
                keep = a[name][i]
                a[name][i] = keep + h
                up = loss(a)
                a[name][i] = keep - h
                want[i] = (up - loss(a)) / (2 * h)
                a[name][i] = keep
            # fp32 operands of size ~10, sums of up to 72 addends: 128 + 72 roundings of 2^-24 of ~100
            _close(name, t, want, 1.2e-3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d,k", [(1, 8, 1), (5, 2880, 4), (3, 4104, 9), (2049, 264, 6), (2053, 2048, 8), (2, 8200, 32)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_residual_norm_is_the_two_calls(T, d, k, dtype, weighted):
    dt = DT[dtype]
    g, x, _, wp, wn, gt = _inputs(T, d, dt, True, True, "channel", T + k)
    R = T * k                                   # rows that no slot names hold NaN
    y_perm = torch.full((R, d), float("nan"), dtype=dt, device=DEV)
    rows = torch.randperm(R, generator=g)[:T * k].to(torch.int32)
    rows[torch.rand(T * k, generator=g) < 0.15] = -1
    rows[:k] = -1                               # a token without a row
    rows = rows.to(DEV)
    live = rows[rows >= 0].long()
    y_perm[live] = _rand(g, len(live), d, dt=dt)
    w = torch.softmax(torch.randn(T, k, generator=g), 1).to(DEV) if weighted else None
    y, y1 = torch.empty_like(x), torch.empty_like(x)
    if weighted:
        abi.moe_combine_weighted(y_perm, rows, w, y)
    else:
        abi.moe_combine(y_perm, rows, T, k, y)
    outs = [[torch.empty_like(x), torch.empty_like(x), torch.empty(T, device=DEV), torch.empty(T, device=DEV)] for _ in range(3)]
    abi.moe_residual_norm(x, y, outs[0][0], outs[0][1], wp, wn, gt, 0.5, 1e-6, outs[0][2], outs[0][3])
    abi.moe_combine_residual_norm(y_perm, rows, w, k, x, outs[1][0], outs[1][1], y1, wp, wn, gt, 0.5, 1e-6, outs[1][2], outs[1][3])
    abi.moe_combine_residual_norm(y_perm, rows, w, k, x, outs[2][0], outs[2][1], None, wp, wn, gt, 0.5, 1e-6, outs[2][2], outs[2][3])
    assert torch.equal(y, y1)
    for a, b, c in zip(*outs):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert (y[0] == 0).all()                    # without a row: norm(0) = 0, out = scale x
    assert torch.equal(outs[0][0][0], (0.5 * x[0].float()).to(dt))


@pytest.mark.parametrize("T", [37, 2051])
def test_norm_alone_and_in_place(T):
    g, x, y, wp, wn, _ = _inputs(T, 2880, torch.bfloat16, True, True, "none", 9)
    n, rn = torch.empty_like(x), torch.empty(T, device=DEV)
    abi.moe_residual_norm(x, None, None, n, w_pre=wn, eps=1e-5, rstd_pre=rn)
    r = O.rstd(_np(x), 1e-5)
    ref = _np(x) * r * _np(wn)
    _close("n", n, ref, (_u(x.dtype) * 1.01 + 52 * V) * abs(ref))
    d_n, d_x, dw = _rand(g, T, 2880, dt=x.dtype), torch.empty_like(x), torch.empty(2880, device=DEV)
    ws = torch.empty(abi.moe_residual_norm_bwd_workspace_size(T, 2880), dtype=torch.uint8, device=DEV)
    for d_out in (None, _rand(g, T, 2880, dt=x.dtype)):
        abi.moe_residual_norm_bwd(d_out, d_n, x, None, d_x, None, ws, w_pre=wn, rstd_pre=rn, d_w_pre=dw)
        ref = O.residual_norm_bwd(_np(d_out), _np(d_n), _np(x), np.zeros((T, 2880)), None, _np(wn), None, 1.0, None, _np(rn)[:, None])
        _close("d_x", d_x, ref["d_x"][0], _u(x.dtype) * 1.01 * abs(ref["d_x"][0]) + 128 * V * ref["d_x"][1])
        _close("d_w_pre", dw, ref["d_w_pre"][0], (T / 256 + 209 + 128) * V * ref["d_w_pre"][1])
    # out over x, n over y, d_x over d_out
    out, n2 = torch.empty_like(x), torch.empty_like(x)
    abi.moe_residual_norm(x, y, out, n2, wp, wn)
    x2, y2 = x.clone(), y.clone()
    abi.moe_residual_norm(x2, y2, x2, y2, wp, wn)
    assert torch.equal(out, x2) and torch.equal(n2, y2)
    abi.moe_residual_norm_bwd(d_out, d_n, x, None, d_out, None, ws, w_pre=wn, rstd_pre=rn)
    assert torch.equal(d_out, d_x)


def test_gradient_of_zero_rows_with_a_tiny_eps():
    """1/rms is 1e15 there: d_x = scale (d_out + rn d_n w), and no product of three of it overflows against a zero."""
    T, d = 5, 264
    g, x, y, wp, wn, _ = _inputs(T, d, torch.float32, True, True, "none", 4)
    x[2], y[3] = 0.0, 0.0
    rp, rn = (torch.tensor(O.rstd(_np(t), 1e-30)[:, 0]).float().to(DEV) for t in (y, x))
    go, gn = _rand(g, T, d), _rand(g, T, d)
    d_x, d_y = torch.empty_like(x), torch.empty_like(x)
    abi.moe_residual_norm_bwd(go, gn, x, y, d_x, d_y, None, wp, wn, None, 1.0, rp, rn)
    ref = O.residual_norm_bwd(_np(go), _np(gn), _np(x), _np(y), _np(wp), _np(wn), None, 1.0, _np(rp)[:, None], _np(rn)[:, None])
    for name, t in (("d_x", d_x), ("d_y", d_y)):
        v, size = ref[name]
        _close(name, t, v, V * abs(v) + 128 * V * size)


@pytest.mark.parametrize("T", [6, 2050])
def test_without_a_stream(T):
    """x None: out = gate norm(y) w_post, and no d_x."""
    d = 776
    g, _, y, wp, wn, gt = _inputs(T, d, torch.bfloat16, True, True, "token", 8)
    out, n, z = (torch.empty_like(y) for _ in range(3))
    rp, rn = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    abi.moe_residual_norm(None, y, out, n, wp, wn, gt, 0.75, 1e-5, rp, rn)
    _check_forward(torch.zeros_like(y), y, out, n, rp, rn, wp, wn, gt, 0.75, 1e-5)
    abi.moe_residual_norm(torch.zeros_like(y), y, z, n, wp, wn, gt, 0.75, 1e-5)
    assert torch.equal(out, z)
    go, gn = _rand(g, T, d, dt=y.dtype), _rand(g, T, d, dt=y.dtype)
    a, b, dx = (torch.empty_like(y) for _ in range(3))
    abi.moe_residual_norm_bwd(go, gn, out, y, None, a, None, wp, wn, gt, 0.75, rp, rn)
    abi.moe_residual_norm_bwd(go, gn, out, y, dx, b, None, wp, wn, gt, 0.75, rp, rn)
    assert torch.equal(a, b)


def test_what_is_not_needed_is_not_read():
    T, d = 6, 520
    g, x, _, _, wn, gt = _inputs(T, d, torch.bfloat16, False, True, "channel", 4)
    nan = torch.full_like(x, float("nan"))
    rn = torch.tensor(O.rstd(_np(x), 1e-5)[:, 0]).float().to(DEV)
    go, gn = _rand(g, T, d, dt=x.dtype), _rand(g, T, d, dt=x.dtype)
    a, b = [torch.empty_like(x) for _ in range(2)], [torch.empty_like(x) for _ in range(2)]
    abi.moe_residual_norm_bwd(go, gn, x, nan, a[0], a[1], None, None, wn, gt, 1.0, None, rn)
    abi.moe_residual_norm_bwd(go, gn, x, None, b[0], b[1], None, None, wn, gt, 1.0, None, rn)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(a[1]).all()
    c = torch.empty_like(x)      # without the second norm, out is not read
    abi.moe_residual_norm_bwd(go, None, nan, None, c, None, None, None, None, gt, 0.5)
    assert torch.equal(c, (0.5 * go.float()).to(c.dtype))


def test_rows_that_are_zero_inf_or_nan_stay_alone():
    T, d = 9, 520
    _, x, y, wp, wn, _ = _inputs(T, d, torch.bfloat16, True, True, "none", 3)
    ref_out, ref_n = torch.empty_like(x), torch.empty_like(x)
    abi.moe_residual_norm(x, y, ref_out, ref_n, wp, wn)
    y[2] = 0
    y[4, 7] = float("inf")
    x[6, 100] = float("nan")
    out, n = torch.empty_like(x), torch.empty_like(x)
    abi.moe_residual_norm(x, y, out, n, wp, wn)
    for t in range(T):
        if t not in (2, 4, 6):
            assert torch.equal(out[t], ref_out[t]) and torch.equal(n[t], ref_n[t])
    assert torch.equal(out[2], x[2])
    assert torch.isnan(out[4, 7]) and torch.isnan(n[6]).all()


def test_no_tokens():
    z = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    abi.moe_residual_norm(z, z.clone(), z.clone(), z.clone(), w, w)
    dw = torch.full((64,), 3.0, device=DEV)
    r = torch.empty(0, device=DEV)
    abi.moe_residual_norm_bwd(z, z, z, z, z.clone(), z.clone(), None, w, w, None, 1.0, r, r, dw, dw.clone())
    assert (dw == 0).all()


def test_captured_and_on_another_stream():
    T, d, k = 70, 2880, 4
    g, x, _, wp, wn, gt = _inputs(T, d, torch.bfloat16, True, True, "channel", 11)
    y_perm = _rand(g, T * k, d, dt=x.dtype)
    rows = torch.randperm(T * k, generator=g).to(torch.int32).to(DEV)
    w = torch.rand(T, k, generator=g).to(DEV)
    bufs = lambda: [torch.zeros_like(x) for _ in range(6)] + [torch.zeros(T, device=DEV), torch.zeros(T, device=DEV)] + \
        [torch.zeros(d, device=DEV) for _ in range(3)] + [torch.zeros_like(y_perm), torch.zeros(T * k, device=DEV)]
    ws = torch.empty(abi.moe_residual_norm_bwd_workspace_size(T, d), dtype=torch.uint8, device=DEV)

    def chain(b, ws):
        y, out, n, d_x, d_y, spare, rp, rn, dwp, dwn, dg, dyp, drs = b
        abi.moe_combine_residual_norm(y_perm, rows, w, k, x, out, n, y, wp, wn, gt, 1.0, 1e-6, rp, rn)
        abi.moe_residual_norm_bwd(x, n, out, y, d_x, d_y, ws, wp, wn, gt, 1.0, rp, rn, dwp, dwn, dg)
        abi.moe_combine_weighted_bwd(d_y, y_perm, rows, w, dyp, drs)

    eager, cap = bufs(), bufs()
    chain(eager, ws)
    torch.cuda.synchronize()
    ws2 = torch.empty_like(ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        chain(cap, ws2)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(cap, ws2)
    for i in range(3):
        x.mul_(1.25)                            # new inputs for every replay
        graph.replay()
        chain(eager, ws)
        torch.cuda.synchronize()
        for a, b in zip(eager, cap):
            assert torch.equal(a, b)
