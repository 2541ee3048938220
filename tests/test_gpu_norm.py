"""The norm and its gradient on the GPU against float64, with bounds from the
number of roundings, and its operands against the quantizers' of its own y."""
import numpy as np
import pytest
import torch

import block_scaled_precision_blockwise_amd as bsq
from gpu_helpers import assert_bytes_equal, host, say, to_dev
from oracle import norm
from test_gpu_mx4 import E4M3, E5M2, E8M0, empty, u8

pytestmark = pytest.mark.gpu

f32, bf16 = torch.float32, torch.bfloat16
U = 2.0 ** -24  # half a step of float32, relative
KIND = {False: bsq.BSQ_LAYER_NORM, True: bsq.BSQ_RMS_NORM}
# one row to more rows than groups; lengths of one value, of every number of
# threads to a row, odd, and past the registers
SHAPES = [(1, 1), (1, 4096), (3, 5), (5, 64), (2, 511), (9, 512), (600, 96), (7, 1000), (4, 1024), (3, 1537), (2100, 40),
          (6, 2048), (5, 4096), (3, 4104), (2, 8192), (3, 9999), (2, 16384), (3, 16416), (2, 20001)]


def inputs(R, C, dt, seed):
    g = np.random.default_rng(seed)
    x = (g.standard_normal((R, C)) + g.standard_normal(C) * 0.5) * np.exp2(g.integers(-4, 5, (R, 1))) + 0.3
    dy = g.standard_normal((R, C))
    q = lambda v: (torch.from_numpy(v).to(dt)).double().numpy()  # noqa: E731
    w = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    return q(x), q(dy), w(1 + 0.3 * g.standard_normal(C)), w(0.3 * g.standard_normal(C))


def roundings(C):
    """Of a row's sum: what a thread adds by itself, six exchanges, up to 16 waves."""
    return (16 if C <= 16384 else -(-C // 1024)) + 6 + 16


def bounds(x, gamma, beta, rms, eps):
    """y, mean and rstd in 64 bits, and how far float32 with that many
    roundings can be off: of xn, y, mean, rstd."""
    n = roundings(x.shape[1])
    y, mean, rstd = norm.forward(x, gamma, beta, eps, rms)
    t_mean = 0 * mean if rms else (n + 1) * U * np.abs(x).mean(1)
    d = x - mean[:, None]
    t_d = t_mean[:, None] + U * np.abs(d)
    # the mean of d^2 is off by 2 |d| t_d + t_d^2 on average, and by its own roundings
    var = (d * d).mean(1) + eps
    t_var = (2 * np.abs(d) * t_d + t_d * t_d).mean(1) + (n + 4) * U * var
    rel = 0.5 * t_var / var * (1 + t_var / var) + 3 * U  # of rstd: a square root and a division
    xn = d * rstd[:, None]
    t_xn = (rstd[:, None] * t_d + np.abs(xn) * (rel[:, None] + U)) * (1 + 2 * rel[:, None])
    t_y = np.abs(gamma) * (t_xn + U * np.abs(xn)) + U * np.abs(y)
    t_y += U * np.abs(xn * gamma)
    return (y, mean, rstd), (t_xn, t_y * (1 + 4 * U), t_mean, rstd * rel * (1 + rel))


def held(got, want, tol, dt, what):
    tol = tol * 1.01 + 1e-37 + (2.0 ** -8 * (np.abs(want) + tol) if dt == bf16 else 0.0)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), (what, float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt", [f32, bf16])
@pytest.mark.parametrize("R, C", SHAPES)
def test_norm(R, C, dt, rms):
    say("norm", R, C, dt, rms)
    eps = 1e-5
    x, dy, gamma, beta = inputs(R, C, dt, R + C)
    if rms:
        beta = 0 * beta
    dev = lambda v, t=f32: torch.from_numpy(v).to("cuda", t)  # noqa: E731
    xd, gd, bd = dev(x, dt), dev(gamma), None if rms else dev(beta)
    y, mean, rstd = empty(R, C, dtype=dt), empty(R, dtype=f32), empty(R, dtype=f32)
    bsq.bsq_norm_mx(xd, y=y, gamma=gd, beta=bd, mean=mean, rstd=rstd, eps=eps, kind=KIND[rms])
    want, tol = bounds(x, gamma, beta, rms, eps)
    held(y, want[0], tol[1], dt, "y")
    held(mean, want[1], tol[2], f32, "mean")
    held(rstd, want[2], tol[3], f32, "rstd")
    # the gradient, from the norm's own mean and rstd
    dx, dg, db = empty(R, C, dtype=dt), empty(C, dtype=f32), empty(C, dtype=f32)
    space = empty(bsq.bsq_norm_backward_workspace_bytes(R, C))
    kw = dict(mean=None if rms else mean, gamma=gd, kind=KIND[rms])
    bsq.bsq_norm_backward(xd, dev(dy, dt), rstd, dx, dgamma=dg, dbeta=db, workspace=space, **kw)
    wx, wg, wb = norm.backward(x, dy, gamma, eps, rms)
    n, t_xn = roundings(C), tol[0] * 1.01
    xn, d = (x - want[1][:, None]) * want[2][:, None], dy * gamma
    s1, s2 = (d * xn).mean(1, keepdims=True), (0 if rms else 1) * d.mean(1, keepdims=True)
    t1 = (np.abs(d) * t_xn).mean(1, keepdims=True) + (n + 4) * U * np.abs(d * xn).mean(1, keepdims=True)
    t2 = (n + 3) * U * np.abs(d).mean(1, keepdims=True)
    inner = U * 4 * (np.abs(d) + np.abs(xn * s1) + np.abs(s2)) + t_xn * np.abs(s1) + (np.abs(xn) + t_xn) * t1 + t2
    r = want[2][:, None]
    held(dx, wx, r * inner * 1.01 + np.abs(wx) * (tol[3][:, None] / r + 2 * U) * 1.01, dt, "dx")
    # rows of a group, the groups' eight shares, and their joining
    m = -(-R // 32) + 64 + 16 + 2
    held(dg, wg, (np.abs(dy) * t_xn).sum(0) + (m + 1) * U * np.abs(dy * xn).sum(0), f32, "dgamma")
    held(db, wb, m * U * np.abs(dy).sum(0), f32, "dbeta")
    # without the weights' gradients, and one of them alone: the same bytes
    again, one = empty(R, C, dtype=dt), empty(C, dtype=f32)
    bsq.bsq_norm_backward(xd, dev(dy, dt), rstd, again, **kw)
    assert torch.equal(again.view(torch.int16), dx.view(torch.int16))
    bsq.bsq_norm_backward(xd, dev(dy, dt), rstd, again, dbeta=one, workspace=space, **kw)
    assert torch.equal(again.view(torch.int16), dx.view(torch.int16)) and torch.equal(one, db)


@pytest.mark.parametrize("rms", [False, True])
def test_gradient_against_differences(rms):
    R, C, h = 4, 192, 1e-5
    x, dy, gamma, beta = inputs(R, C, f32, 3)
    dev = lambda v: torch.from_numpy(v).to("cuda", f32)  # noqa: E731
    _, mean, rstd = norm.forward(x, gamma, beta, 1e-5, rms)
    dx, dg, db = empty(R, C, dtype=f32), empty(C, dtype=f32), empty(C, dtype=f32)
    bsq.bsq_norm_backward(dev(x), dev(dy), dev(rstd), dx, mean=dev(mean), gamma=dev(gamma), dgamma=dg, dbeta=db,
                          workspace=empty(bsq.bsq_norm_backward_workspace_bytes(R, C)), kind=KIND[rms])
    g = np.random.default_rng(0)
    f = lambda x, a, b: float((norm.forward(x, a, b, 1e-5, rms)[0] * dy).sum())  # noqa: E731
    for _ in range(5):
        vx, vg, vb = g.standard_normal((R, C)), g.standard_normal(C), g.standard_normal(C)
        want = (f(x + h * vx, gamma + h * vg, beta + h * vb) - f(x - h * vx, gamma - h * vg, beta - h * vb)) / (2 * h)
        terms = [(t.double().cpu().numpy(), v) for t, v in ((dx, vx), (dg, vg), (db, vb))]
        got = sum(float((t * v).sum()) for t, v in terms)
        # gradients good to 2^-17 of their size (held closer above), differences to h^2 and 1e-15 / h of the sum
        size = sum(float(np.abs(t * v).sum()) for t, v in terms)
        assert abs(got - want) <= 2.0 ** -17 * size + 1e-6, (got, want)


@pytest.mark.parametrize("dt", [f32, bf16])
@pytest.mark.parametrize("code", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("R, C", [(1, 32), (5, 96), (1, 4096), (7, 1056), (3, 2080), (130, 128), (3, 16384), (2, 16416)])
def test_operand_is_the_quantizers_of_y(R, C, code, dt):
    """The codes are those that the quantizer gives of the float32 y; of a
    bfloat16 x those of its values in float32."""
    say("norm operand", R, C, code, dt)
    x, _, gamma, beta = inputs(R, C, dt, 2 * R + C)
    x[0, : min(C, 64)] *= 2.0 ** -20
    x = torch.from_numpy(x).to("cuda", dt)
    gd, bd = (torch.from_numpy(v).to("cuda", f32) for v in (gamma, beta))
    new = lambda: ((empty(R, C // 2) if code == "e2m1" else empty(R, C, dtype={"e4m3": E4M3, "e5m2": E5M2}[code])),  # noqa: E731
                   empty(R, C // 32, dtype=E8M0))
    a, y = new(), empty(R, C, dtype=f32)
    bsq.bsq_norm_mx(x.float(), y=y, codes=a[0], scales=a[1], gamma=gd, beta=bd)
    q = new()
    if code == "e2m1":
        bsq.bsq_quant_fp4(y, *q)
    else:
        bsq.bsq_quant_mx(y, *q, 1, bsq.BSQ_E5M2 if code == "e5m2" else bsq.BSQ_E4M3)
    b, yb = new(), empty(R, C, dtype=dt)
    bsq.bsq_norm_mx(x, codes=b[0], scales=b[1], gamma=gd, beta=bd)  # without y
    for got in (a, b):
        for v, w, n in zip(got, q, ("codes", "scales")):
            assert_bytes_equal(host(v.view(u8)), host(w.view(u8)), n)
    bsq.bsq_norm_mx(x, y=yb, gamma=gd, beta=bd)  # without codes
    assert torch.equal(yb, y.to(dt))


def test_no_rows_and_no_weights():
    x, z = empty(0, 64, dtype=f32), empty(0, dtype=f32)
    dg, db = empty(64, dtype=f32), empty(64, dtype=f32)
    bsq.bsq_norm_mx(x, y=x, mean=z, rstd=z)
    bsq.bsq_norm_backward(x, x, z, x, mean=z, dgamma=dg, dbeta=db, workspace=empty(16))
    assert not dg.any() and not db.any()
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(5, 64, generator=g, device="cuda")
    y, w = empty(5, 64, dtype=f32), empty(5, 64, dtype=f32)
    bsq.bsq_norm_mx(x, y=y)
    bsq.bsq_norm_mx(x, y=w, gamma=torch.ones(64, device="cuda"), beta=torch.zeros(64, device="cuda"))
    assert torch.equal(y, w)


@pytest.mark.parametrize("C", [96, 1000, 4096, 16416])
def test_infinities_and_nan_show_in_their_row_alone(C):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(6, C, generator=g, device="cuda")
    clean = empty(6, C, dtype=f32)
    bsq.bsq_norm_mx(x, y=clean)
    x[1, 3], x[3, C - 1], x[4, 0] = float("nan"), float("inf"), float("-inf")
    y = empty(6, C, dtype=f32)
    coded = C % 32 == 0
    codes, scales = (empty(6, C // 2), empty(6, C // 32, dtype=E8M0)) if coded else (None, None)
    bsq.bsq_norm_mx(x, y=y, codes=codes, scales=scales)
    for r in (0, 2, 5):
        assert torch.equal(y[r], clean[r])
    for r in (1, 3, 4):
        assert torch.isnan(y[r]).all()
        if coded:
            assert bool((scales.view(u8)[r] == 255).all())


@pytest.mark.parametrize("dt", [f32, bf16])
@pytest.mark.parametrize("R, C", [(5, 96), (2100, 64), (7, 1001), (700, 4096), (3, 16384), (40, 16416), (3, 20001)])
def test_in_place(R, C, dt):
    """y in x's place, dx in x's or dy's: the same bytes as elsewhere."""
    say("norm in place", R, C, dt)
    x, dy, gamma, beta = inputs(R, C, dt, R + C)
    x, dy = (torch.from_numpy(v).to("cuda", dt) for v in (x, dy))
    gd, bd = (torch.from_numpy(v).to("cuda", f32) for v in (gamma, beta))
    coded = C % 32 == 0
    new = lambda: (empty(R, C, dtype=E4M3), empty(R, C // 32, dtype=E8M0)) if coded else (None, None)  # noqa: E731
    (q, s), (qi, si) = new(), new()
    y, yi, mean, rstd = empty(R, C, dtype=dt), x.clone(), empty(R, dtype=f32), empty(R, dtype=f32)
    bsq.bsq_norm_mx(x, y=y, codes=q, scales=s, gamma=gd, beta=bd, mean=mean, rstd=rstd)
    bsq.bsq_norm_mx(yi, y=yi, codes=qi, scales=si, gamma=gd, beta=bd)
    assert torch.equal(y, yi)
    if coded:
        assert torch.equal(q.view(u8), qi.view(u8)) and torch.equal(s.view(u8), si.view(u8))
    space = empty(bsq.bsq_norm_backward_workspace_bytes(R, C))
    outs = []
    for place in ("own", "x", "dy"):
        xi, di = x.clone(), dy.clone()
        dx = {"own": empty(R, C, dtype=dt), "x": xi, "dy": di}[place]
        dg, db = empty(C, dtype=f32), empty(C, dtype=f32)
        bsq.bsq_norm_backward(xi, di, rstd, dx, mean=mean, gamma=gd, dgamma=dg, dbeta=db, workspace=space)
        outs.append((dx, dg, db))
    for got in outs[1:]:
        for a, b in zip(got, outs[0]):
            assert torch.equal(a, b)
