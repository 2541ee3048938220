"""The norm on rows that hold infinities or NaN, and on rows whose sums or squares do not fit float32: every kernel,
both kinds."""
import numpy as np
import pytest
import torch

import block_scaled_precision_blockwise_amd as bsq
from gpu_helpers import say
from oracle import norm
from test_gpu_mx4 import E4M3, E5M2, E8M0, empty, gen, u8
from test_gpu_norm import KIND, U, bounds, held, roundings

pytestmark = pytest.mark.gpu

f32, bf16 = torch.float32, torch.bfloat16
CODES = {"none": None, "e4m3": E4M3, "e5m2": E5M2, "e2m1": u8}


def same(a, b):
    return torch.equal(a.view(u8), b.view(u8))


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt", [f32, bf16])
@pytest.mark.parametrize("C, code", [(C, code) for C in (96, 1000, 1024, 2048, 4096, 8192, 16384, 16416, 20001)
                                     for code in CODES if code == "none" or C % 32 == 0])  # codes come in whole blocks
def test_infinities_and_nan_make_their_whole_row_nan(C, code, dt, rms):
    """In y, in codes of 8 bits, as the scales of 4-bit ones and in rstd; the other rows are as without them."""
    say("norm of infinities and NaN", C, code, dt, rms)
    R, bad = 7, (1, 3, 4, 6)
    x = torch.randn(R, C, generator=gen(C), device="cuda").to(dt)
    beta = torch.randn(C, generator=gen(1), device="cuda")
    outs = []
    for marked in (False, True):
        if marked:
            x[1, 3], x[3, C - 1], x[4, 0] = float("nan"), float("inf"), float("-inf")
            x[6, 5], x[6, 50] = float("inf"), float("-inf")
        y, rstd = empty(R, C, dtype=dt), empty(R, dtype=f32)
        q = s = None
        if code != "none":
            q, s = empty(R, C // 2 if code == "e2m1" else C, dtype=CODES[code]), empty(R, C // 32, dtype=E8M0)
        bsq.bsq_norm_mx(x, y=y, codes=q, scales=s, beta=beta, rstd=rstd, kind=KIND[rms])
        outs.append((y, rstd, q, s))
    for r in range(R):
        y, rstd, q, s = (None if t is None else t[r] for t in outs[1])
        if r not in bad:
            assert all(same(t[r:r + 1], w[r:r + 1]) for t, w in zip(outs[1], outs[0]) if t is not None), r
            continue
        assert bool(torch.isnan(y).all()) and bool(torch.isnan(rstd)), r
        if code == "e2m1":
            assert bool((s.view(u8) == 255).all()), r
        elif code != "none":
            assert bool(torch.isnan(q.float()).all()), r


# ------------------------------------------- rows that pass float32 on the way --

ROWS = ("largest", "one against the rest", 100, 64, 0, -62, -90, -118)  # of which powers of two


def rows(C, dt, seed):
    """Rows of every magnitude."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((len(ROWS), C))
    for r, e in enumerate(ROWS):
        if e == "largest":
            x[r] = g.uniform(-3.3e38, 3.3e38, C)
        elif e == "one against the rest":
            x[r], x[r, C // 2] = -3.3e38, 3.3e38
        else:
            x[r] = (x[r] + 0.25) * 2.0 ** e
    return torch.from_numpy(x).to(dt).double().numpy()


@pytest.mark.parametrize("eps", [0.0, 1e-5, 1e-30])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt", [f32, bf16])
@pytest.mark.parametrize("C", [5, 64, 512, 1000, 2048, 4096, 8192, 9999, 16384, 16416, 20001])
def test_rows_whose_sums_or_squares_pass_float32(C, dt, rms, eps):
    """Squares above 2^128 and below 2^-149, sums and differences above the largest: the bounds of other rows hold."""
    say("norm of large and small rows", C, dt, rms, eps)
    eps = float(np.float32(eps))
    x = rows(C, dt, C)
    R = x.shape[0]
    g = np.random.default_rng(1)
    w = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    gamma, beta = w(1 + 0.3 * g.standard_normal(C)), w(0.3 * g.standard_normal(C))
    dev = lambda v, t=f32: torch.from_numpy(v).to("cuda", t)  # noqa: E731
    xd, gd = dev(x, dt), dev(gamma)
    y, mean, rstd = empty(R, C, dtype=dt), empty(R, dtype=f32), empty(R, dtype=f32)
    bsq.bsq_norm_mx(xd, y=y, gamma=gd, beta=dev(beta), mean=mean, rstd=rstd, eps=eps, kind=KIND[rms])
    want, tol = bounds(x, gamma, beta, rms, eps)
    for got, v, t, kind, what in ((y, want[0], tol[1], dt, "y"), (mean, want[1], tol[2], f32, "mean"),
                                  # rstd of the largest rows is subnormal
                                  (rstd, want[2], tol[3] + 2.0 ** -149, f32, "rstd")):
        for r in range(R):  # what `held` adds for all is too much for some
            err, t_r = np.abs(got[r].double().cpu().numpy() - v[r]), t[r] * 1.01
            t_r = t_r + (2.0 ** -8 * (np.abs(v[r]) + t_r) if kind == bf16 else 0.0)
            assert np.all(err <= t_r), (what, ROWS[r], float(np.max(err - t_r)))
    # in place: the row is read again
    xi = xd.clone()
    bsq.bsq_norm_mx(xi, y=xi, gamma=gd, beta=dev(beta), eps=eps, kind=KIND[rms])
    assert same(xi, y)
    # every value the largest, and zeros
    big = float(torch.finfo(dt).max)
    x = torch.full((2, C), big, device="cuda", dtype=dt)
    x[1] = 0
    bsq.bsq_norm_mx(x, y=y[:2], mean=mean[:2], rstd=rstd[:2], eps=1e-5, kind=KIND[rms])
    n = roundings(C)
    if rms:
        assert bool(((y[0].double() - 1).abs() <= (n + 8) * U + (2.0 ** -8 if dt == bf16 else 0)).all())
    else:
        assert abs(float(mean[0]) / big - 1) <= (n + 1) * U and bool(torch.isfinite(y[0]).all())
    assert not y[1].any() and abs(float(rstd[1]) * 1e-5 ** 0.5 - 1) < 1e-6


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt", [f32, bf16])
@pytest.mark.parametrize("C", [5, 64, 512, 1000, 2048, 4096, 8192, 9999, 16384, 16416, 20001])
def test_gradients_of_rows_whose_differences_pass_float32(C, dt, rms):
    """x - mean above the largest, rstd next to the smallest: from the norm's own mean and rstd, dx to the bounds of other
    rows, and the weights' gradients."""
    say("gradients of large and small rows", C, dt, rms)
    eps = 1e-30
    x = rows(C, dt, C)
    R = x.shape[0]
    g = np.random.default_rng(2)
    # of a size that brings dx, as large as dy / x, well inside float32
    dy = g.standard_normal((R, C)) * 2.0 ** np.array([[62 if isinstance(e, str) else e // 2] for e in ROWS])
    dy = torch.from_numpy(dy).to(dt).double().numpy()
    gamma = (1 + 0.3 * g.standard_normal(C)).astype(np.float32).astype(np.float64)
    dev = lambda v, t=f32: torch.from_numpy(v).to("cuda", t)  # noqa: E731
    xd, gd = dev(x, dt), dev(gamma)
    mean, rstd = empty(R, dtype=f32), empty(R, dtype=f32)
    bsq.bsq_norm_mx(xd, mean=mean, rstd=rstd, eps=eps, kind=KIND[rms])
    dx, dg, db = empty(R, C, dtype=dt), empty(C, dtype=f32), empty(C, dtype=f32)
    bsq.bsq_norm_backward(xd, dev(dy, dt), rstd, dx, mean=None if rms else mean, gamma=gd, dgamma=dg, dbeta=db,
                          workspace=empty(bsq.bsq_norm_backward_workspace_bytes(R, C)), kind=KIND[rms])
    eps = float(np.float32(eps))
    want, tol = bounds(x, gamma, 0 * gamma, rms, eps)
    wx, wg, wb = norm.backward(x, dy, gamma, eps, rms)
    n, r = roundings(C), want[2][:, None]
    xn, d = (x - want[1][:, None]) * r, dy * gamma
    t_r = tol[3][:, None] / r + 2.0 ** -149 / r  # rstd may be subnormal
    t_xn = tol[0] * 1.01 + np.abs(xn) * 2.0 ** -149 / r
    s1, s2 = (d * xn).mean(1, keepdims=True), (0 if rms else 1) * d.mean(1, keepdims=True)
    t1 = (np.abs(d) * t_xn).mean(1, keepdims=True) + (n + 4) * U * np.abs(d * xn).mean(1, keepdims=True)
    t2 = (n + 3) * U * np.abs(d).mean(1, keepdims=True)
    inner = U * 4 * (np.abs(d) + np.abs(xn * s1) + np.abs(s2)) + t_xn * np.abs(s1) + (np.abs(xn) + t_xn) * t1 + t2
    t_x = (r * inner * 1.01 + np.abs(wx) * (t_r + 2 * U)) * 1.02
    t_x += 2.0 ** -8 * (np.abs(wx) + t_x) if dt == bf16 else 0.0
    err = np.abs(dx.double().cpu().numpy() - wx)
    for i in range(R):
        assert np.all(err[i] <= t_x[i]), ("dx", ROWS[i], float((err[i] - t_x[i]).max()))
    # sums over the rows: up to R of a group, 16 shares and their joining
    held(dg, wg, (np.abs(dy) * t_xn).sum(0) + (R + 35) * U * np.abs(dy * xn).sum(0), f32, "dgamma")
    held(db, wb, (R + 34) * U * np.abs(dy).sum(0), f32, "dbeta")


# --------------------------------------------------------------- long rows --

@pytest.mark.parametrize("dt", [f32, bf16])
@pytest.mark.parametrize("C", [16385, 300001, (1 << 22) + 32])
def test_long_rows_far_from_zero(C, dt):
    """The mean is that of the row to its own rounding and to those of sums of x - mean, however many values there are:
    a row of one value is zeros."""
    say("norm of long rows far from zero", C, dt)
    g = np.random.default_rng(C)
    x = np.stack([np.full(C, 1000.1), np.full(C, -0.3), 1000.0 + g.standard_normal(C), 20.0 + 1e-3 * g.standard_normal(C)])
    x = torch.from_numpy(x).to(dt).double().numpy()
    y, mean, rstd = empty(4, C, dtype=f32), empty(4, dtype=f32), empty(4, dtype=f32)
    bsq.bsq_norm_mx(torch.from_numpy(x).to("cuda", f32), y=y, mean=mean, rstd=rstd)
    want, m, r = norm.forward(x, eps=float(np.float32(1e-5)))
    n = roundings(C)
    d = np.abs(x - m[:, None])
    t_first = (n + 1) * U * np.abs(x).mean(1)  # of the first mean, from which the second's differences are taken
    t_mean = U * np.abs(m) + (n + 4) * U * (d.mean(1) + t_first)
    assert np.all(np.abs(mean.double().cpu().numpy() - m) <= t_mean), np.abs(mean.double().cpu().numpy() - m) / t_mean
    # the variance: sums of (x - first mean)^2, less the square of what that is off
    var = (d * d).mean(1) + 1e-5
    t_d = U * (d + t_first[:, None])
    t_var = ((2 * d * t_d + t_d * t_d).mean(1) + 2 * (n + 6) * U * ((d * d).mean(1) + t_first ** 2) +
             2 * t_first * (n + 4) * U * (d.mean(1) + t_first) + 4 * U * var)
    rel = 0.5 * t_var / var * (1 + 2 * t_var / var) + 3 * U
    assert np.all(np.abs(rstd.double().cpu().numpy() - r) <= r * rel)
    t_y = (r * t_mean)[:, None] * (1 + rel[:, None]) + np.abs(want) * (rel[:, None] + 4 * U)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= t_y * 1.01)
