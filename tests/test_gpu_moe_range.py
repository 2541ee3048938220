"""Expert-layer operators at the ends of their range, against oracle/moe.py:
scores that are nothing in 32 or in 64 bits, biases that rule experts out,
NaN.

Bounds.  Forward: scores and weights are made in 64 bits to a relative 2^-38
and rounded once, half a step of 2^-24 relative, or of the least number of 32
bits.  Gradient, in 32 bits: an exponential's argument is off by half a step
of itself, which becomes a relative error of the result (at most 104 steps: a
larger argument gives less than the least number); beside it at most 32
roundings (exponentials, sums over the lanes, divisions, products); three such
factors in a term and as much again for the sums that are taken off it.
"""
import numpy as np
import pytest

import block_scaled_precision_blockwise_amd as bsq
from oracle import formats as F
from oracle import moe as OE

from gpu_helpers import filled, host, say, to_dev

pytestmark = pytest.mark.gpu

TINY = 1e-37  # below this float32 results are denormal
LEAST = 2.0 ** -149
FEW, MANY = 37, 2051  # a wave to a token, and four tokens to a wave


def _torch():
    import torch
    return torch


def _logits(x, bf16):
    """(device tensor, the float64 values it holds)."""
    torch = _torch()
    x = np.asarray(x, np.float32)
    if not bf16:
        return to_dev(x), x.astype(np.float64)
    bits = F.encode_bf16(x)
    return to_dev(bits.view(np.int16)).view(torch.bfloat16), F.decode_bf16(bits).astype(np.float64)


def _values(t):
    h = host(t)
    return F.decode_bf16(h).astype(np.float64) if h.dtype == np.uint16 else h.astype(np.float64)


def _within(got, want, bound, what):
    got = np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), f"{what}: not finite at {np.argwhere(~np.isfinite(got))[:3].tolist()}"
    bad = np.argwhere(~(np.abs(got - want) <= bound))
    if len(bad):
        i = tuple(bad[0])
        raise AssertionError(f"{what}: {len(bad)} of {got.size} outside; first {i}: {got[i]!r} for {want[i]!r}, "
                             f"bound {np.broadcast_to(bound, got.shape)[i]!r}")


def _span(x, ids):
    """Relative error of a gradient's exponentials (see above)."""
    top = x.max(1, keepdims=True)
    chosen = np.take_along_axis(x, np.where((ids >= 0) & (ids < x.shape[1]), ids, 0).astype(np.int64), 1)
    far = np.maximum(np.abs(np.where(np.isfinite(x), x - np.where(np.isfinite(top), top, 0.0), 0.0)).max(1),
                     np.where(np.isfinite(chosen), np.ptp(np.where(np.isfinite(chosen), chosen, 0.0), axis=1)[:, None],
                              0.0).max(1))
    return (2 * np.minimum(far, 104.0)[:, None] + 32) * 2.0 ** -24


def _check_backward(x, bf16, ids, ds=None, sigmoid=False, renorm=True, scale=2.5, seed=0):
    torch = _torch()
    dx, xv = _logits(x, bf16)
    rng = np.random.default_rng(seed + 7)
    dw = rng.standard_normal(ids.shape).astype(np.float32)
    dl = filled(xv.shape, dx.dtype, float("nan"))
    bsq.bsq_moe_route_backward(dx, to_dev(np.asarray(ids, np.int32)), to_dev(dw), dl,
                               dscores=None if ds is None else to_dev(ds), score=int(sigmoid), renorm=renorm, scale=scale)
    want, size = OE.route_backward(xv, ids, dw, ds, sigmoid, renorm, scale)
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    _within(_values(dl), want, 6 * _span(xv, np.asarray(ids)) * size + half * np.abs(want) + TINY, "dlogits")
    if renorm and ids.shape[1] > 1:
        assert np.abs(want).max() > 0.01  # the case has a gradient to lose


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("far", [60, 86, 88.5, 90, 100, 110, 200, 700, 740, 3000])
def test_route_gradient_of_chosen_scores_that_are_nothing_in_32_bits(T, sigmoid, far):
    """Softmax: a bias has steered the choice to experts `far` below the row's
    largest logit.  Sigmoid: every logit is near -far.  The weights p / sum
    are ordinary numbers, and so are their gradients."""
    say("route gradient far", T, sigmoid, far)
    rng = np.random.default_rng(int(far) + T)
    for E, k, bf16 in ((5, 2, False), (96, 6, False), (256, 8, True), (20, 1, False), (320, 12, False)):
        x = rng.standard_normal((T, E)) - far
        if not sigmoid:
            x[:, E - 2:] += far  # never chosen
        ids = np.stack([rng.permutation(E - 2 if E > 5 else 3)[:k] for _ in range(T)]).astype(np.int32)
        ds = (rng.standard_normal((T, E)) * 0.1).astype(np.float32) if E != 96 else None
        _check_backward(x, bf16, ids, ds, sigmoid, seed=E)
        _check_backward(x, bf16, ids, ds, sigmoid, renorm=False, seed=E)


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_gradient_beside_masked_logits_and_ids_that_are_none(T, sigmoid):
    say("route gradient masked", T, sigmoid)
    rng = np.random.default_rng(T)
    E, k = 24, 4
    x = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    x[0::6] = -np.inf                                   # a row of nothing
    np.put_along_axis(x[1::6], ids[1::6].astype(np.int64), -np.inf, 1)   # nothing chosen is left
    np.put_along_axis(x[2::6], ids[2::6, :2].astype(np.int64), -np.inf, 1)
    np.put_along_axis(x[3::6], ids[3::6, 1:2].astype(np.int64), -1e9, 1)
    np.put_along_axis(x[4::6], ids[4::6].astype(np.int64), x[4::6, :k] - 95.0, 1)
    ids[::5, 0] = -1
    ids[1::5, 1] = E
    for ds in (None, (rng.standard_normal((T, E)) * 0.1).astype(np.float32)):
        _check_backward(x, False, ids, ds, sigmoid, seed=1)


def _check_forward(x, bf16, k, bias=None, full=True, **kw):
    torch = _torch()
    dx, xv = _logits(x, bf16)
    T, E = xv.shape
    sigmoid = kw.pop("sigmoid", False)
    ids, w = filled((T, k), torch.int32, -7), filled((T, k), torch.float32, float("nan"))
    scores = filled((T, E), torch.float32, float("nan")) if full else None
    bsq.bsq_moe_route(dx, ids, w, bias=None if bias is None else to_dev(np.asarray(bias, np.float32)), scores=scores,
                      score=int(sigmoid), **kw)
    rid, rw, rp = OE.route(xv, k, bias=None if bias is None else np.asarray(bias, np.float32), sigmoid=sigmoid, **kw)
    assert np.array_equal(host(ids), rid), np.argwhere(host(ids) != rid)[:4].tolist()
    half = 2.0 ** -24 * (1 + 2.0 ** -10)
    _within(_values(w), rw, half * np.abs(rw) + LEAST * kw.get("scale", 1.0), "weights")
    if full:
        _within(_values(scores), rp, half * rp + LEAST, "scores")
    return rid, rw


FORWARD = [(256, 8, True, dict(groups=8, top_groups=4, group_top=2, scale=2.5)), (256, 8, False, {}),
           (128, 6, False, dict(groups=4, top_groups=2)), (40, 5, False, dict(renorm=False)), (20, 1, False, {}),
           (320, 8, False, {}), (60, 9, False, {}), (96, 4, False, dict(groups=3, top_groups=2))]


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,k,bf16,opts", FORWARD)
def test_route_is_rounded_once(T, sigmoid, E, k, bf16, opts):
    """Scores and weights to half a step of 32 bits, also where a few logits
    are far from the rest."""
    say("route rounded once", T, sigmoid, E, k, bf16, opts)
    rng = np.random.default_rng(E + k)
    x = rng.standard_normal((T, E)) * 1.5
    x[0::5, ::3] = -1e9
    x[1::5, 0] = -3e38
    x[2::5, :E // 2] -= 60.0
    x[3::5, 1::2] -= 690.0
    _check_forward(x, bf16, k, (rng.standard_normal(E) * 0.1).astype(np.float32), sigmoid=sigmoid, **opts)
    _check_forward(x, bf16, k, sigmoid=sigmoid, **opts)


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("far", [90, 200, 690, 705, 720, 735, 760, 3000])
@pytest.mark.parametrize("E,k,bf16,opts", FORWARD)
def test_route_weights_of_chosen_scores_that_are_nothing(T, sigmoid, far, E, k, bf16, opts):
    """A bias steers the choice to half of the experts, whose logits lie `far`
    below the row's largest (softmax) or zero (sigmoid): p / sum is ordinary
    where p itself is less than 64 bits hold."""
    say("route weights far", T, sigmoid, far, E, k, bf16, opts)
    rng = np.random.default_rng(E + far)
    x = rng.standard_normal((T, E)) - far
    bias = np.zeros(E, np.float32)
    bias[E // 2:] = 4.0
    if not sigmoid:
        x[:, :E // 2] += far
    rid, rw = _check_forward(x, bf16, k, bias, sigmoid=sigmoid, **opts)
    assert np.all(rid >= E // 2)
    if opts.get("renorm", True):
        assert np.allclose(rw.sum(1), opts.get("scale", 1.0))


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,groups", [(24, 1), (256, 1), (256, 8), (300, 3), (512, 4)])
@pytest.mark.parametrize("k", [4, 8, 12])
def test_route_choice_between_scores_that_are_nearly_nothing(T, sigmoid, E, groups, k):
    """Fewer ordinary logits than choices; the rest -inf (score 0), and some far
    below (scores of 1e-295 and less, the least numbers of 64 bits among them),
    which come before the -inf ones in the order of their size."""
    say("route nearly nothing", T, sigmoid, E, groups, k)
    rng = np.random.default_rng(E + groups)
    x = np.full((T, E), -np.inf)
    far = -(np.array([691.0, 693, 695, 697, 699, 701, 703, 705]) if sigmoid else
            np.array([691.0, 703, 716, 730, 738, 740, 742, 744]))
    for t in range(T):
        at = rng.permutation(E)
        x[t, at[:8]] = far[rng.permutation(8)]
        if not sigmoid or t % 2:
            x[t, at[8]] = 0.0
        x[t, at[9:11]] = (-800.0, -1e9)
    for g in (1, 2) if groups > 1 else (1,):
        opts = dict(groups=groups, top_groups=max(1, groups // 2), group_top=g) if groups > 1 else {}
        _check_forward(x, False, k, sigmoid=sigmoid, full=False, **opts)
        _check_forward(x, False, k, np.zeros(E, np.float32), sigmoid=sigmoid, renorm=False, **opts)


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("E,groups,k", [(40, 1, 4), (40, 1, 9), (256, 8, 8), (256, 8, 12), (300, 1, 8), (24, 3, 3), (1000, 1, 2)])
def test_route_shows_nan(T, E, groups, k):
    """Softmax: a row with NaN or +inf has NaN scores, weights and gradients.
    Sigmoid: a NaN logit has a NaN score and comes last; +inf has the score 1.
    By whichever kernel; the rows beside them are as without."""
    torch = _torch()
    say("route NaN", T, E, groups, k)
    rng = np.random.default_rng(E + k)
    x = rng.standard_normal((T, E)).astype(np.float32)
    x[1::7, 3] = np.nan
    x[2::7, 5] = np.inf
    x[3::7, 1:] = -np.inf
    x[3::7, 0] = np.nan
    x[4::7] = np.nan
    bad = np.zeros(T, bool)
    for r in range(1, 5):
        bad[r::7] = True
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for sigmoid in (False, True):
        ids, w, p = filled((T, k), torch.int32, -7), filled((T, k), torch.float32, 7.0), filled((T, E), torch.float32, 7.0)
        kw = dict(groups=groups, top_groups=max(1, groups // 2)) if groups > 1 else {}
        bsq.bsq_moe_route(to_dev(x), ids, w, scores=p, score=int(sigmoid), **kw)
        dl = filled((T, E), torch.float32, 7.0)
        bsq.bsq_moe_route_backward(to_dev(x), ids, to_dev(dw), dl, score=int(sigmoid))
        i, w, p, dl = host(ids), host(w), host(p), host(dl)
        assert i.min() >= 0 and i.max() < E and all(len(set(r)) == k for r in i.tolist())
        if not sigmoid:
            assert np.all(np.isnan(p[bad])) and np.all(np.isnan(w[bad])) and np.all(np.isnan(dl[bad]))
            assert np.all(np.isfinite(p[~bad])) and np.all(np.isfinite(w[~bad])) and np.all(np.isfinite(dl[~bad]))
            continue
        assert np.array_equal(np.isnan(p), np.isnan(x)) and np.array_equal(np.isnan(dl), np.isnan(x) | (
            np.isnan(np.take_along_axis(x, i.astype(np.int64), 1)).any(1)[:, None] & _asked(i, E)))
        assert np.all(p[2::7, 5] == 1.0) and np.all(np.isfinite(w[1::7])) and np.all(np.isfinite(w[2::7]))
        assert not np.any(i[1::7] == 3) and np.all(np.isnan(w[4::7]))


def _asked(ids, E):
    m = np.zeros((len(ids), E), bool)
    np.put_along_axis(m, ids.astype(np.int64), True, 1)
    return m


PAYLOADS = [0x7FC00000, 0x7FFFFFFF, 0xFFFFFFFF, 0xFFC00001, 0x7FFF8000]


@pytest.mark.parametrize("bits", PAYLOADS)
def test_nan_stays_nan_in_bfloat16(bits):
    """A NaN of any payload, on its way to a bfloat16 output."""
    torch = _torch()
    say("NaN in bfloat16", hex(bits))
    nan = np.array([bits], np.uint32).view(np.float32)
    w = np.ones((5, 2), np.float32)
    w[2, 1:] = nan
    y = torch.randn(10, 64, device="cuda").bfloat16()
    pos = torch.arange(10, dtype=torch.int32, device="cuda").view(5, 2)
    out = torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda")
    bsq.bsq_moe_combine(y, pos, out, weights=to_dev(w))
    want = np.zeros((5, 64), bool)
    want[2] = True
    assert np.array_equal(torch.isnan(out).cpu().numpy(), want)
    for T in (5, MANY):
        x = torch.randn(T, 16, device="cuda").bfloat16()
        dw = np.ones((T, 2), np.float32)
        dw[2, 1:] = nan
        ids = torch.arange(2, dtype=torch.int32, device="cuda").repeat(T, 1)
        dl = torch.zeros(T, 16, dtype=torch.bfloat16, device="cuda")
        bsq.bsq_moe_route_backward(x, ids, to_dev(dw), dl, renorm=False)
        assert torch.isnan(dl[2]).all() and not torch.isnan(dl[3:]).any() and not torch.isnan(dl[:2]).any()


@pytest.mark.parametrize("e5m2", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("bits", PAYLOADS)
def test_nan_stays_nan_in_codes_and_products(bits, bf16, e5m2):
    """NaN in a token or in the gate's input is a NaN code (of both operands
    and of the checkpoint), NaN in the product's row and in the gradient; blocks
    and rows without one are as they were."""
    torch = _torch()
    say("NaN codes", hex(bits), bf16, e5m2)
    dt = torch.bfloat16 if bf16 else torch.float32
    fp8 = torch.float8_e5m2 if e5m2 else torch.float8_e4m3fn
    cd = bsq.BSQ_E5M2 if e5m2 else bsq.BSQ_E4M3
    raw = np.array([bits >> 16], np.uint16).view(np.int16) if bf16 else np.array([bits], np.uint32).view(np.int32)
    R, C = 128, 256
    x = torch.randn(R, C, device="cuda").to(dt)

    def put(t, r, c):
        t.view(torch.int16 if bf16 else torch.int32)[r, c] = int(raw[0])

    def codes(t, T, H, k=1, weights=None):
        o = [filled(s, torch.uint8, 0x55) for s in ((T, H), (T, H // 32), (H, T), (H, T // 32))]
        rows = torch.arange(T, dtype=torch.int32, device="cuda")
        bsq.bsq_moe_gather_mx(t, rows, k, *o, weights=weights, code_dtype=cd)
        return o

    nan = lambda c: torch.isnan(c.view(fp8).float())  # noqa: E731
    plain = codes(x, R, C)
    put(x, 70, 100)
    for weights in (None, torch.ones(R, 1, device="cuda")):
        got = codes(x, R, C, weights=weights)
        m = torch.zeros(R, C, dtype=torch.bool, device="cuda")
        m[70, 100] = True
        assert torch.equal(nan(got[0]), m) and torch.equal(nan(got[2]).t(), m)
        m[70, 96:128] = True
        assert torch.equal(got[0][~m], plain[0][~m])
        m[70] = False
        m[64:96, 100] = True
        assert torch.equal(got[2].t()[~m], plain[2].t()[~m])
    if not e5m2:
        for out_dt in (torch.float32, torch.bfloat16):
            b, sb = torch.full((1, 32, C), 0x38, dtype=torch.uint8, device="cuda"), filled((1, 32, C // 32), torch.uint8, 127)
            out = torch.zeros(R, 32, dtype=out_dt, device="cuda")
            bsq.bsq_moe_matmul(got[0], got[1], b, sb, torch.tensor([0, R], dtype=torch.int32, device="cuda"), out)
            m = torch.zeros(R, 32, dtype=torch.bool, device="cuda")
            m[70] = True
            assert torch.equal(torch.isnan(out), m)
    # the gate: g at (9, 5), u at (90, 40)
    gu = torch.randn(R, C, device="cuda").to(dt)
    put(gu, 9, 5)
    put(gu, 90, 128 + 40)
    u8 = lambda *s: filled(s, torch.uint8, 0x55)  # noqa: E731
    h, hs, ht, hts, kept, ks = u8(R, 128), u8(R, 4), u8(128, R), u8(128, R // 32), u8(R, C), u8(R, C // 32)
    bsq.bsq_swiglu_mx(gu, h, hs, ht, hts, kept, ks, code_dtype=cd)
    m = torch.zeros(R, 128, dtype=torch.bool, device="cuda")
    m[9, 5] = m[90, 40] = True
    assert torch.equal(nan(h), m) and torch.equal(nan(ht).t(), m) and torch.equal(nan(kept), torch.isnan(gu))
    h2, hs2 = u8(R, 128), u8(R, 4)
    bsq.bsq_swiglu_mx(gu, h2, hs2, code_dtype=cd)
    assert torch.equal(h2, h) and torch.equal(hs2, hs)
    dh = torch.randn(R, 128, device="cuda").to(dt)
    put(dh, 50, 7)
    dgu = torch.zeros(R, C, dtype=dt, device="cuda")
    bsq.bsq_swiglu_mx_backward(kept, ks, dh, dgu, code_dtype=cd)
    m[50, 7] = True
    bad = torch.isnan(dgu)
    assert torch.equal(bad[:, :128], m)          # dg: from g, u or dh
    m[90, 40] = False
    assert torch.equal(bad[:, 128:], m)          # du: from g or dh


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("E", [60, 100, 250, 500, 1000])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_by_every_kernel(T, E, bf16, sigmoid):
    """Widths up to 64, 128, 256, 512 and 1024, few tokens and many, few
    choices (up to 8) and more (past 16 in the gradient)."""
    say("route every kernel", T, E, bf16, sigmoid)
    rng = np.random.default_rng(E)
    x = rng.standard_normal((T, E)) * 1.5
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    ds = (rng.standard_normal((T, E)) * 0.1).astype(np.float32)
    for k in (5, 12, 17):
        ids, _ = _check_forward(x, bf16, k, bias, full=k != 12, sigmoid=sigmoid, scale=2.5)
        _check_backward(x, bf16, ids, ds if k != 12 else None, sigmoid, seed=k)


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,groups,k", [(16, 4, 3), (64, 8, 8), (256, 8, 8), (256, 16, 4), (24, 3, 5), (64, 8, 12)])
def test_route_of_groups_whose_experts_a_bias_rules_out(T, sigmoid, E, groups, k):
    """A group's worth is the sum of its two largest: -inf with fewer than two
    experts left, equal to that of a group with none, so the lowest index."""
    say("route groups ruled out", T, sigmoid, E, groups, k)
    rng = np.random.default_rng(E + k)
    x = rng.standard_normal((T, E)) * 1.5
    per = E // groups
    for left in range(3):  # experts left in each group but the last
        bias = np.full(E, -np.inf, np.float32)
        bias[(groups - 1) * per:] = 0.0
        for g in range(1, groups - 1):
            bias[g * per + rng.permutation(per)[:left]] = 0.25
        for top in sorted({1, 2, groups // 2, groups - 1}):
            if k <= top * per:
                _check_forward(x, False, k, bias, sigmoid=sigmoid, groups=groups, top_groups=top, group_top=2)
