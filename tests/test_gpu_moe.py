"""The expert-layer operators on the GPU against oracle/moe.py (64 bits).

Whole numbers, codes and scales of gathered rows are equal.  Floating
outputs: a float32 result carries 2^-24 relative for each rounding on its
way, as counted at each bound below; a bfloat16 output one more half step
(2^-8); products the bound of the other block-scaled products
(1e-4 sum |a b|, plus the matrix core's group-of-8 allowance).
"""
import numpy as np
import pytest

import block_scaled_precision_blockwise_amd as bsq
from oracle import formats as F
from oracle import moe as OE
from oracle import quantize as OQ

from gpu_helpers import assert_bytes_equal, empty, filled, host, say, to_dev

pytestmark = pytest.mark.gpu

TINY = 1e-37  # below this float32 results are denormal


def _torch():
    import torch
    return torch


def _bf16(a):
    """float32 values rounded to bfloat16: (bits for the device, values)."""
    bits = F.encode_bf16(np.asarray(a, np.float32))
    return bits, F.decode_bf16(bits).astype(np.float64)


def _dev_values(a, bf16):
    """(device tensor, the float64 values it holds)."""
    torch = _torch()
    if bf16:
        bits, v = _bf16(a)
        return to_dev(bits.view(np.int16)).view(torch.bfloat16), v
    a = np.asarray(a, np.float32)
    return to_dev(a), a.astype(np.float64)


def _values(t):
    """float64 values of a device tensor (float32, bfloat16)."""
    h = host(t)
    return F.decode_bf16(h).astype(np.float64) if h.dtype == np.uint16 else h.astype(np.float64)


def _within(got, want, bound, what):
    got = np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), f"{what}: not finite at {np.argwhere(~np.isfinite(got))[:3].tolist()}"
    bad = np.argwhere(np.abs(got - want) > bound)
    if len(bad):
        i = tuple(bad[0])
        raise AssertionError(f"{what}: {len(bad)} of {got.size} outside; first {i}: {got[i]!r} for {want[i]!r}, "
                             f"bound {np.broadcast_to(bound, got.shape)[i]!r}")


# --------------------------------------------------------------- routing --

def _span(x):
    """Relative error of a float32 score, in units of 2^-24: the exponent's
    argument x - max is off by half a step of its size, which the exponential
    turns into a relative error; beside it at most 32 roundings (exponential,
    sum over the lanes, division, product)."""
    x = np.where(np.isfinite(x), x, 0.0)
    return (np.abs(x).max(1, keepdims=True) * 2 + 32) * 2.0 ** -24


def _route(x, bf16, k, bias=None, train=True, full=True, seed=0, **kw):
    torch = _torch()
    dx, xv = _dev_values(x, bf16)
    T, E = x.shape
    ids, w = filled((T, k), torch.int32, -7), filled((T, k), torch.float32, float("nan"))
    scores = filled((T, E), torch.float32, float("nan")) if full else None
    db = None if bias is None else to_dev(np.asarray(bias, np.float32))
    score = bsq.BSQ_SIGMOID if kw.pop("sigmoid", False) else bsq.BSQ_SOFTMAX
    bsq.bsq_moe_route(dx, ids, w, bias=db, scores=scores, score=score, **kw)
    okw = dict(groups=kw.get("groups", 1), top_groups=kw.get("top_groups", 1), group_top=kw.get("group_top", 1),
               renorm=kw.get("renorm", True), scale=kw.get("scale", 1.0), sigmoid=score == bsq.BSQ_SIGMOID)
    rid, rw, rp = OE.route(xv, k, bias=None if bias is None else np.asarray(bias, np.float32), **okw)
    assert np.array_equal(host(ids), rid), np.argwhere(host(ids) != rid)[:4].tolist()
    tol = _span(xv)
    _within(_values(w), rw, 3 * tol * np.abs(rw) + TINY, "weights")
    if full:
        _within(_values(scores), rp, tol * rp + TINY, "scores")
    if not train:
        return
    rng = np.random.default_rng(seed + 1000)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    ds = (rng.standard_normal((T, E)) * 0.1).astype(np.float32) if full else None
    dl = filled((T, E), dx.dtype, float("nan"))
    bsq.bsq_moe_route_backward(dx, ids, to_dev(dw), dl, dscores=None if ds is None else to_dev(ds), score=score,
                               renorm=okw["renorm"], scale=okw["scale"])
    want, size = OE.route_backward(xv, rid, dw, ds, okw["sigmoid"], okw["renorm"], okw["scale"])
    _within(_values(dl), want, 6 * tol * size + (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(want) + TINY, "dlogits")


ROUTES = [  # T, E, k, bf16, options
    (1, 1, 1, False, {}), (1, 2, 2, True, dict(sigmoid=True)), (3, 7, 3, False, {}), (65, 64, 8, True, {}),
    (5, 65, 4, False, dict(sigmoid=True, renorm=False)), (130, 128, 8, True, dict(scale=2.5)),
    (67, 256, 8, False, dict(sigmoid=True, groups=8, top_groups=4, group_top=2, scale=2.5)),
    (67, 256, 8, True, dict(groups=8, top_groups=4, group_top=2)),
    (33, 256, 6, True, dict(groups=8, top_groups=3, group_top=1)),
    (9, 21, 5, False, dict(groups=7, top_groups=2, group_top=2)), (9, 250, 8, True, dict(groups=2, top_groups=1)),
    (17, 96, 8, False, dict(groups=4, top_groups=2, group_top=2, sigmoid=True)),
    (4, 64, 64, False, {}), (4, 1000, 33, True, dict(sigmoid=True)), (3, 1024, 64, False, dict(groups=64, top_groups=9)),
    (700, 256, 8, False, dict(sigmoid=True, renorm=False)), (10, 512, 4, True, {}),
    (64, 32, 4, True, dict(sigmoid=True)), (31, 16, 2, False, {}), (20, 8, 1, False, {}),
]


@pytest.mark.parametrize("T,E,k,bf16,opts", ROUTES)
@pytest.mark.parametrize("biased", [False, True])
def test_route(T, E, k, bf16, opts, biased):
    say("route", T, E, k, bf16, opts, biased)
    rng = np.random.default_rng(T * 1009 + E * 31 + k)
    x = rng.standard_normal((T, E)) * 1.5
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if biased else None
    _route(x, bf16, k, bias, full=(T + E) % 2 == 0 or T > 60, seed=T, **dict(opts))


@pytest.mark.parametrize("E", [24, 64, 256, 320])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_takes_the_lowest_index_of_equals(E, sigmoid):
    """Logits of few values: most choices are between equals."""
    say("route equals", E, sigmoid)
    rng = np.random.default_rng(E)
    x = rng.integers(-2, 3, (50, E)).astype(np.float32)
    _route(x, True, 8, sigmoid=sigmoid)
    _route(x, False, 6, sigmoid=sigmoid, groups=8, top_groups=3, group_top=2)


@pytest.mark.parametrize("E", [64, 256])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups", [1, 8])
def test_route_tells_scores_apart_past_float32(E, sigmoid, groups):
    """A bias that nearly cancels the scores: what is left to choose by lies
    below a float32 step of the scores."""
    say("route close", E, sigmoid, groups)
    rng = np.random.default_rng(E + groups)
    x = (rng.standard_normal((1, E)) * 1.5).astype(np.float32).repeat(40, 0)
    bias = (0.5 - OE.scores(x[:1], sigmoid)[0]).astype(np.float32)
    _route(x, False, 8, bias, sigmoid=sigmoid, groups=groups, top_groups=max(1, groups // 2),
           group_top=2 if groups > 1 else 1)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,groups", [(40, 1), (64, 4), (256, 8)])
def test_route_with_logits_that_are_masked(sigmoid, E, groups):
    """-inf logits score zero; a row of nothing else has weights, scores and
    gradients of zero, and its ids are still different experts."""
    say("route masked", sigmoid, E, groups)
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((12, E)) * 2).astype(np.float32)
    x[0, :] = -np.inf
    x[1, 1:] = -np.inf
    x[2, : E // 2] = -np.inf
    x[3, ::2] = -np.inf
    x[4, :] = -60.0   # softmax even, sigmoid near zero
    x[5, :] = 80.0
    x[6, 0] = -3e38
    _route(x, False, 6, sigmoid=sigmoid, groups=groups, top_groups=max(1, groups // 2))
    x[:, 3] = -np.inf
    b = np.zeros(E, np.float32)
    b[5] = -np.inf  # a bias that rules an expert out
    _route(x, False, 4, b, sigmoid=sigmoid, groups=groups, top_groups=max(1, groups // 2))


@pytest.mark.parametrize("E", [40, 256])
def test_route_ids_are_experts_whatever_the_logits(E):
    torch = _torch()
    say("route NaN", E)
    x = torch.randn(64, E, device="cuda")
    x[0] = float("nan")
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3, :] = float("inf")
    for kw in (dict(), dict(score=bsq.BSQ_SIGMOID), dict(groups=4, top_groups=2, group_top=2)):
        ids, w = filled((64, 8), torch.int32, -7), empty((64, 8), torch.float32)
        bsq.bsq_moe_route(x, ids, w, **kw)
        got = host(ids)
        assert got.min() >= 0 and got.max() < E and all(len(set(r)) == 8 for r in got.tolist())


def test_route_backward_passes_over_ids_that_are_none():
    torch = _torch()
    say("route backward none")
    rng = np.random.default_rng(4)
    x = rng.standard_normal((6, 20)).astype(np.float32)
    ids = np.array([[0, 1], [-1, 3], [20, 4], [-1, -1], [19, 1000], [5, 6]], np.int32)
    dw = rng.standard_normal((6, 2)).astype(np.float32)
    for sigmoid in (False, True):
        dl = filled((6, 20), torch.float32, float("nan"))
        bsq.bsq_moe_route_backward(to_dev(x), to_dev(ids), to_dev(dw), dl, score=int(sigmoid))
        want, size = OE.route_backward(x, ids, dw, None, sigmoid)
        _within(_values(dl), want, 6 * _span(x) * size + TINY, "dlogits")


MANY = 2051  # tokens enough for the kernels that put four in a wave, and three left over


@pytest.mark.parametrize("E,k,bf16,opts", [
    (256, 8, True, dict(sigmoid=True, groups=8, top_groups=4, group_top=2, scale=2.5)),
    (256, 8, False, dict(groups=8, top_groups=3, group_top=1)), (256, 1, True, {}), (255, 8, False, dict(sigmoid=True)),
    (250, 7, True, dict(groups=2, top_groups=1, renorm=False)), (128, 8, True, {}), (129, 5, False, {}),
    (64, 6, True, dict(sigmoid=True, groups=16, top_groups=5, group_top=2)), (65, 2, True, dict(sigmoid=True)),
    (96, 8, False, dict(groups=4, top_groups=2, group_top=2)), (8, 8, True, {}), (3, 2, False, dict(sigmoid=True)),
    (1, 1, True, {}), (126, 4, True, dict(groups=2, top_groups=2, sigmoid=True)),
    (256, 9, True, {}), (192, 16, False, dict(sigmoid=True)), (60, 3, False, dict(groups=3, top_groups=2)),
    (512, 8, True, dict(groups=8, top_groups=4)), (1000, 8, False, dict(sigmoid=True)), (260, 6, True, {})])
@pytest.mark.parametrize("biased", [False, True])
def test_route_of_many_tokens(E, k, bf16, opts, biased):
    say("route many", E, k, bf16, opts, biased)
    rng = np.random.default_rng(E * 31 + k)
    x = rng.standard_normal((MANY, E)) * 1.5
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if biased else None
    _route(x, bf16, k, bias, full=(E + k) % 2 == 0, seed=E, **dict(opts))


@pytest.mark.parametrize("T", [37, MANY])
@pytest.mark.parametrize("E", [24, 64, 256, 320])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_of_equals_with_a_bias(T, E, sigmoid):
    """Few logits and few biases: equal sums of equal and of different terms,
    and experts that are left out next to equals that are chosen."""
    say("route equals biased", T, E, sigmoid)
    rng = np.random.default_rng(E)
    x = rng.integers(-1, 2, (T, E)).astype(np.float32)
    bias = (rng.integers(0, 2, E) * 0.25).astype(np.float32)
    _route(x, True, 8, bias, sigmoid=sigmoid)
    _route(x, False, 6, None, sigmoid=sigmoid, groups=8, top_groups=3, group_top=2)
    _route(x, False, 5, bias, sigmoid=sigmoid, groups=4, top_groups=2, group_top=1)


@pytest.mark.parametrize("E", [64, 256, 512])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups", [1, 8])
def test_route_of_many_tells_scores_apart_past_float32(E, sigmoid, groups):
    """A bias that cancels the scores but for what lies below a float32 step."""
    say("route close many", E, sigmoid, groups)
    rng = np.random.default_rng(E + groups)
    x = (rng.standard_normal((1, E)) * 1.5).astype(np.float32).repeat(MANY, 0)
    x[1::2] = np.roll(x[1::2], 1, axis=1)
    bias = (0.5 - OE.scores(x[:1], sigmoid)[0]).astype(np.float32)
    _route(x, False, 8, bias, train=False, sigmoid=sigmoid, groups=groups, top_groups=max(1, groups // 2),
           group_top=2 if groups > 1 else 1)


@pytest.mark.parametrize("T", [64, MANY])
@pytest.mark.parametrize("E", [40, 256, 300])
def test_route_tells_scores_of_neighbouring_logits_apart(T, E):
    """Logits next to each other in float32 where the sigmoid is flat: scores
    that differ by a part in 2^48."""
    say("route neighbours", T, E)
    rng = np.random.default_rng(E)
    at = np.float32(20.0) + np.arange(E, dtype=np.float32) * np.float32(2.0 ** -19)
    x = np.stack([rng.permutation(at) for _ in range(T)])
    _route(x, False, 8, sigmoid=True)
    _route(x, False, 8)


@pytest.mark.parametrize("E,groups", [(40, 1), (64, 4), (256, 8), (400, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_of_many_with_logits_that_are_masked(E, groups, sigmoid):
    say("route masked many", E, groups, sigmoid)
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((MANY, E)) * 2).astype(np.float32)
    x[0::13, :] = -np.inf
    x[1::13, 1:] = -np.inf
    x[2::13, : E // 2] = -np.inf
    x[3::13, ::2] = -np.inf
    x[4::13, :] = -60.0
    x[5::13, :] = 80.0
    x[6::13, 0] = -3e38
    x[7::13, 3:] = -1e9
    x[8::13, 2:] -= 700.0
    _route(x, False, 6, sigmoid=sigmoid, groups=groups, top_groups=max(1, groups // 2))
    b = np.zeros(E, np.float32)
    b[5] = -np.inf
    b[6] = 3.0
    _route(x, False, 4, b, sigmoid=sigmoid, groups=groups, top_groups=max(1, groups // 2), group_top=2)


@pytest.mark.parametrize("E", [40, 256, 500])
def test_route_ids_of_many_are_experts_whatever_the_logits(E):
    torch = _torch()
    say("route NaN many", E)
    x = torch.randn(MANY, E, device="cuda")
    x[0::9] = float("nan")
    x[1::9, 5] = float("nan")
    x[2::9, 7] = float("inf")
    x[3::9, :] = float("inf")
    for kw in (dict(), dict(score=bsq.BSQ_SIGMOID), dict(groups=4, top_groups=2, group_top=2)):
        ids, w = filled((MANY, 8), torch.int32, -7), empty((MANY, 8), torch.float32)
        bsq.bsq_moe_route(x, ids, w, **kw)
        got = host(ids)
        assert got.min() >= 0 and got.max() < E and all(len(set(r)) == 8 for r in got.tolist())


def test_route_backward_of_many_passes_over_ids_that_are_none():
    torch = _torch()
    say("route backward none many")
    rng = np.random.default_rng(6)
    x = rng.standard_normal((MANY, 20)).astype(np.float32)
    ids = np.stack([rng.permutation(24)[:3] for _ in range(MANY)]).astype(np.int32)
    ids[ids >= 22] = -1
    dw = rng.standard_normal((MANY, 3)).astype(np.float32)
    for sigmoid in (False, True):
        dl = filled((MANY, 20), torch.float32, float("nan"))
        bsq.bsq_moe_route_backward(to_dev(x), to_dev(ids), to_dev(dw), dl, score=int(sigmoid))
        want, size = OE.route_backward(x, ids, dw, None, sigmoid)
        _within(_values(dl), want, 6 * _span(x) * size + TINY, "dlogits")


# ------------------------------------------------------------------ rows --

@pytest.mark.parametrize("n,E,align", [(0, 4, 128), (1, 1, 1), (1, 256, 128), (63, 5, 32), (128, 256, 1), (1000, 8, 128),
                                       (1024, 1024, 1), (1025, 3, 1), (4099, 1000, 32), (8192, 64, 128), (8193, 17, 1),
                                       (70001, 37, 128), (300000, 256, 1), (300001, 2, 7)])
def test_plan(n, E, align):
    torch = _torch()
    say("plan", n, E, align)
    rng = np.random.default_rng(n + E)
    ids = np.minimum(rng.integers(0, E, n), rng.integers(0, E, n)).astype(np.int32)  # low experts more often
    if n > 60:
        ids[rng.integers(0, n, n // 20)] = rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], n // 20)
    cap = bsq.bsq_moe_capacity(n, E, align) + (0 if n % 2 else align)
    outs = [filled((s,), torch.int32, -9) for s in (E + 1, E, cap, n)]
    ws = empty((bsq.bsq_moe_plan_workspace_bytes(n, E),), torch.uint8)
    for _ in range(2):
        bsq.bsq_moe_plan(to_dev(ids), *outs, ws, align=align)
        for name, g, r in zip(("offsets", "counts", "rows", "pos"), outs, OE.plan(ids, E, align, cap)):
            assert np.array_equal(host(g), r), (name, np.argwhere(host(g) != r)[:4].tolist())


def _planned(T, E, k, align, seed, none=0.0):
    """choices [T, k], and the order of their rows (numpy)."""
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32).reshape(T, k)
    if none:
        ids[rng.random((T, k)) < none] = -1
    cap = bsq.bsq_moe_capacity(T * k, E, align)
    return (ids, cap, *OE.plan(ids, E, align, cap))


@pytest.mark.parametrize("T,H,E,k,align,bf16,e5m2,weighted", [
    (1, 32, 4, 1, 32, True, False, False), (5, 96, 8, 3, 32, False, False, True), (70, 160, 5, 2, 128, True, True, True),
    (200, 256, 16, 4, 128, True, False, False), (33, 64, 3, 3, 32, False, True, False), (300, 2048, 7, 2, 128, True, False, True)])
def test_gather(T, H, E, k, align, bf16, e5m2, weighted):
    torch = _torch()
    say("gather", T, H, E, k, align, bf16, e5m2, weighted)
    ids, cap, offsets, counts, rows, pos = _planned(T, E, k, align, T + H, none=0.1)
    rng = np.random.default_rng(T)
    x = (rng.standard_normal((T, H)) * np.exp(rng.uniform(-8, 8, (T, 1)))).astype(np.float32)
    x[0, :32] = 0.0
    dx, xv = _dev_values(x, bf16)
    w = rng.random((T, k)).astype(np.float32) if weighted else None
    fmt = F.E5M2 if e5m2 else F.E4M3
    v = OE.gather(xv.astype(np.float32), rows, k, w)
    want = (*OQ.mx_axis(v, 1, fmt), *OQ.mx_axis(v, 0, fmt))
    outs = [filled(s.shape, torch.uint8, 0x55) for s in want]
    cd = bsq.BSQ_E5M2 if e5m2 else bsq.BSQ_E4M3
    dw = None if w is None else to_dev(w)
    bsq.bsq_moe_gather_mx(dx, to_dev(rows), k, *outs, weights=dw, code_dtype=cd)
    for name, g, r in zip(("codes", "scales", "codes_t", "scales_t"), outs, want):
        assert_bytes_equal(host(g), r, name)
    # either half alone writes the same
    some = [filled(s.shape, torch.uint8, 0x55) for s in want]
    bsq.bsq_moe_gather_mx(dx, to_dev(rows), k, some[0], some[1], weights=dw, code_dtype=cd)
    bsq.bsq_moe_gather_mx(dx, to_dev(rows), k, codes_t=some[2], scales_t=some[3], weights=dw, code_dtype=cd)
    for name, g, r in zip(("codes", "scales", "codes_t", "scales_t"), some, want):
        assert_bytes_equal(host(g), r, name + " alone")


@pytest.mark.parametrize("e5m2", [False, True])
@pytest.mark.parametrize("bf16,order", [(True, "pattern"), (True, "mixed"), (False, "mixed")])
def test_gather_codes_every_value_as_the_quantizer_does(e5m2, bf16, order):
    """Every bfloat16 but NaN (infinities among them), next to its neighbours
    and next to any other, along rows and down columns."""
    torch = _torch()
    say("gather every value", e5m2, bf16, order)
    bits = np.arange(65536, dtype=np.uint32)
    bits = bits[(bits & 0x7FFF) <= 0x7F80]
    bits = np.concatenate([bits, bits[:-len(bits) % 4096 or None][: -len(bits) % 4096]]).astype(np.uint16)
    if order == "mixed":
        bits = np.random.default_rng(1).permutation(bits)
    T, H = len(bits) // 64, 64
    x = to_dev(bits.view(np.int16).reshape(T, H)).view(torch.bfloat16)
    if not bf16:
        x = x.float()
    cd = bsq.BSQ_E5M2 if e5m2 else bsq.BSQ_E4M3
    rows = torch.arange(T, dtype=torch.int32, device="cuda")
    shapes = ((T, H), (T, H // 32), (H, T), (H, T // 32))
    got, want = ([filled(s, torch.uint8, 0x55) for s in shapes] for _ in range(2))
    bsq.bsq_moe_gather_mx(x, rows, 1, *got, code_dtype=cd)
    bsq.bsq_quant_mx(x, want[0], want[1], 1, cd)
    bsq.bsq_quant_mx(x, want[2], want[3], 0, cd)
    for name, g, r in zip(("codes", "scales", "codes_t", "scales_t"), got, want):
        assert_bytes_equal(host(g), host(r), name)


@pytest.mark.parametrize("T,H,k,bf16,weighted", [(300, 416, 2, True, False), (300, 416, 2, True, True),
                                                 (1000, 160, 3, False, False), (257, 128, 1, True, False)])
def test_gather_over_several_tiles(T, H, k, bf16, weighted):
    torch = _torch()
    say("gather tiles", T, H, k, bf16, weighted)
    ids, cap, offsets, counts, rows, pos = _planned(T, 5, k, 32, T + H, none=0.1)
    rng = np.random.default_rng(T)
    dx, xv = _dev_values(rng.standard_normal((T, H)) * np.exp(rng.uniform(-8, 8, (T, 1))), bf16)
    w = rng.random((T, k)).astype(np.float32) if weighted else None
    v = OE.gather(xv.astype(np.float32), rows, k, w)
    want = (*OQ.mx_axis(v, 1, F.E4M3), *OQ.mx_axis(v, 0, F.E4M3))
    outs = [filled(s.shape, torch.uint8, 0x55) for s in want]
    bsq.bsq_moe_gather_mx(dx, to_dev(rows), k, *outs, weights=None if w is None else to_dev(w))
    for name, g, r in zip(("codes", "scales", "codes_t", "scales_t"), outs, want):
        assert_bytes_equal(host(g), r, name)


def test_gather_of_rows_that_point_nowhere():
    torch = _torch()
    say("gather nowhere")
    x = np.ones((3, 32), np.float32)
    rows = np.full(32, -1, np.int32)
    rows[:5] = [5, 6, 2 ** 31 - 1, -2 ** 31, 0]  # T k = 6: 6 is past the end
    outs = [filled(s, torch.uint8, 0x55) for s in ((32, 32), (32, 1))]
    bsq.bsq_moe_gather_mx(to_dev(x), to_dev(rows), 2, *outs)
    want = OQ.mx(OE.gather(x, rows, 2))
    assert_bytes_equal(host(outs[0]), want[0], "codes")
    assert_bytes_equal(host(outs[1]), want[1], "scales")


@pytest.mark.parametrize("T,H,E,k,bf16,weighted", [
    (1, 8, 4, 1, True, True), (3, 24, 8, 5, False, True), (70, 136, 5, 2, True, False), (129, 2048, 16, 8, True, True),
    (40, 520, 70, 64, True, True), (50, 1000, 12, 3, False, False), (9, 4104, 6, 6, True, True)])
def test_combine(T, H, E, k, bf16, weighted):
    torch = _torch()
    say("combine", T, H, E, k, bf16, weighted)
    ids, cap, offsets, counts, rows, pos = _planned(T, E, k, 1, T + H, none=0.1)
    rng = np.random.default_rng(H)
    pos = pos.copy()
    pos[0, 0] = rng.choice([-1, cap, 2 ** 31 - 1])
    y, yv = _dev_values(rng.standard_normal((cap, H)), bf16)
    w = rng.standard_normal((T, k)).astype(np.float32) if weighted else None
    out = filled((T, H), y.dtype, float("nan"))
    bsq.bsq_moe_combine(y, to_dev(pos), out, weights=None if w is None else to_dev(w))
    want, size = OE.combine(yv, pos, w)
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    _within(_values(out), want, k * 2.0 ** -24 * size + half * np.abs(want) * (1 + 2.0 ** -10) + TINY, "out")
    dout, dv = _dev_values(rng.standard_normal((T, H)), bf16)
    dw = filled((T, k), torch.float32, float("nan"))
    bsq.bsq_moe_combine_backward(y, to_dev(pos), dout, dw)
    want, size = OE.combine_backward(yv, pos, dv)
    # a lane adds H / 64 products one after another, six halvings join the lanes
    _within(_values(dw), want, (H / 64 + 16) * 2.0 ** -24 * size + TINY, "dweights")


# -------------------------------------------------------------- products --

def _operand(rng, shape, fmt, wild=False):
    """(codes, scales, values) as the quantizer makes them of normal values."""
    x = rng.standard_normal(shape).astype(np.float32)
    if wild:
        x *= np.exp(rng.uniform(-6, 6, (*shape[:-1], 1))).astype(np.float32)
    c, s = OQ.mx(x, fmt)
    v = F.decode(c, fmt).astype(np.float64) * F.decode_e8m0(s).astype(np.float64).repeat(32, -1)
    return c, s, v


def _product_bound(want, total, group, bf16):
    return 1e-4 * total + 2.0 ** -9 * group + (2.0 ** -8 if bf16 else 0.0) * np.abs(want) + TINY


def _check_product(lengths, T, N, K, k, e5m2=False, bf16=True, gather=True, tail=0, seed=0, align=1):
    """Segments of the given lengths, rows of random choices (some none)."""
    torch = _torch()
    rng = np.random.default_rng(seed + N + K)
    E = len(lengths)
    offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    cap = int(offsets[-1]) + tail
    rows = rng.integers(0, T * k, cap).astype(np.int32)
    rows[rng.random(cap) < 0.1] = -1
    fmt = F.E5M2 if e5m2 else F.E4M3
    a, sa, av = _operand(rng, (T, K), fmt, wild=True)
    if gather and T > 1:
        a[0], av[0] = 0x7F, 0.0  # NaN codes in a row that no choice takes
        rows[(rows >= 0) & (rows < k)] = -1
    b, sb, bv = _operand(rng, (E, N, K), F.E4M3)
    out = filled((cap, N), torch.bfloat16 if bf16 else torch.float32, float("nan"))
    kw = dict(rows=to_dev(rows), k=k) if gather else {}
    args = (to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(offsets), out)
    cd = bsq.BSQ_E5M2 if e5m2 else bsq.BSQ_E4M3
    bsq.bsq_moe_matmul(*args, a_dtype=cd, **kw)
    want, total, group = OE.product(av, bv, offsets, cap, rows if gather else None, k)
    _within(_values(out), want, _product_bound(want, total, group, bf16), "product")
    first = host(out).copy()
    out.fill_(float("nan"))
    bsq.bsq_moe_matmul(*args, a_dtype=cd, **kw)
    assert np.array_equal(first, host(out)), "two runs differ"


PRODUCTS = [  # lengths, T, N, K, k, options
    ([1], 1, 16, 128, 1, {}), ([0, 1, 0, 3], 4, 80, 256, 2, {}), ([3, 17, 0, 1, 16, 40], 30, 272, 384, 3, dict(tail=9)),
    ([1, 1, 1, 1, 1, 1, 1, 1], 8, 528, 1152, 1, dict(e5m2=True)), ([33, 15, 64, 65], 50, 144, 640, 2, dict(bf16=False)),
    ([100, 70, 0, 131, 200], 60, 272, 384, 2, dict(tail=50)), ([129, 127, 128], 90, 128, 128, 1, dict(e5m2=True, tail=1)),
    ([260, 64], 100, 176, 1024, 4, dict(bf16=False, e5m2=True)), ([700, 513, 900], 300, 272, 384, 2, dict(tail=3)),
    ([1100, 30], 200, 528, 640, 1, dict(e5m2=True)), ([600], 100, 16, 2048, 2, dict(bf16=False)),
    ([0, 0, 0], 5, 64, 128, 1, dict(tail=40)), ([2] * 70, 40, 48, 256, 1, {}), ([1, 0] * 150, 40, 32, 128, 1, {}),
    ([5, 9], 14, 4096, 256, 1, {}), ([16, 32, 8], 60, 1040, 128, 1, dict(gather=False, tail=4)),
    ([300, 400], 700, 80, 256, 1, dict(gather=False)), ([7, 12], 10, 64, 256, 1, dict(gather=False)),
]


@pytest.mark.parametrize("lengths,T,N,K,k,opts", PRODUCTS)
def test_matmul(lengths, T, N, K, k, opts):
    say("moe matmul", len(lengths), sum(lengths), T, N, K, k, opts)
    _check_product(lengths, T, N, K, k, **opts)


@pytest.mark.parametrize("N,lengths", [
    # 64 x 64 tiles, 64 x 128 in three stages and in two, by how many there are; 64 x 64 for 17 to 31 rows an expert
    (784, [300, 0, 500, 3]), (1296, [300, 0, 500, 3]), (2576, [300, 0, 500, 3]), (720, [25, 0, 64, 1] * 5)])
@pytest.mark.parametrize("K,opts", [(128, dict(bf16=False)), (384, dict(e5m2=True, tail=3)), (512, dict(gather=False)),
                                    (256, dict(e5m2=True, bf16=False))])
def test_matmul_by_number_of_tiles(N, lengths, K, opts):
    T = sum(lengths) if not opts.get("gather", True) else 90
    say("moe matmul tiles", len(lengths), sum(lengths), T, N, K, opts)
    _check_product(lengths, T, N, K, 1 if T > 90 else 2, **opts)


def test_matmul_without_tokens_or_contraction_writes_zeros():
    torch = _torch()
    say("moe matmul empty")
    off = to_dev(np.array([0, 5, 9], np.int32))
    b, sb = empty((2, 32, 128), torch.uint8), empty((2, 32, 4), torch.uint8)
    out = filled((10, 32), torch.float32, float("nan"))
    bsq.bsq_moe_matmul(empty((0, 128), torch.uint8), empty((0, 4), torch.uint8), b, sb, off, out,
                       rows=to_dev(np.zeros(10, np.int32)))
    assert np.all(host(out) == 0)
    out.fill_(float("nan"))
    bsq.bsq_moe_matmul(empty((4, 0), torch.uint8), empty((4, 0), torch.uint8), empty((2, 32, 0), torch.uint8),
                       empty((2, 32, 0), torch.uint8), off, out)
    assert np.all(host(out) == 0)


@pytest.mark.parametrize("cap,E", [(40, 3), (300, 3), (2000, 3)])
def test_matmul_with_offsets_and_rows_out_of_range(cap, E):
    """Index arrays that no plan writes: nothing is read or written out of
    range (the outputs beside the array keep their values)."""
    torch = _torch()
    say("moe matmul wild indexes", cap)
    rng = np.random.default_rng(cap)
    T, N, K, k = 20, 80, 256, 2
    a, sa, _ = _operand(rng, (T, K), F.E4M3)
    b, sb, _ = _operand(rng, (E, N, K), F.E4M3)
    guard = filled((cap + 64, N), torch.bfloat16, 3.0)
    for off in ([0, 2 ** 31 - 1, -5, cap], [-2 ** 31, cap // 2, cap + 1000, 2 ** 31 - 1], [cap, 0, cap, 0]):
        rows = rng.choice(np.array([-2 ** 31, -1, 0, T * k - 1, T * k, 2 ** 31 - 1]), cap).astype(np.int32)
        bsq.bsq_moe_matmul(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(np.array(off, np.int32)), guard[:cap],
                           rows=to_dev(rows), k=k)
        assert np.all(_values(guard[cap:]) == 3.0)


@pytest.mark.parametrize("blocks,N,K,e5m2,bf16", [
    ([1], 16, 16, False, False), ([2, 0, 1, 3], 80, 272, True, True), ([0, 0], 32, 48, False, True),
    ([5, 4], 272, 144, True, False), ([1, 0, 2] * 45, 48, 272, True, True), ([3, 2], 2048, 32, False, True)])
def test_wgrad(blocks, N, K, e5m2, bf16):
    torch = _torch()
    say("wgrad", len(blocks), sum(blocks), N, K, e5m2, bf16)
    rng = np.random.default_rng(N + K)
    offsets = (128 * np.concatenate([[0], np.cumsum(blocks)])).astype(np.int32)
    cap = max(128, int(offsets[-1])) + 128
    fmt = F.E5M2 if e5m2 else F.E4M3
    dy, sd, dv = _operand(rng, (N, cap), fmt)
    x, sx, xv = _operand(rng, (K, cap), F.E4M3)
    out = filled((len(blocks), N, K), torch.bfloat16 if bf16 else torch.float32, float("nan"))
    args = (to_dev(dy), to_dev(sd), to_dev(x), to_dev(sx), to_dev(offsets), out)
    cd = bsq.BSQ_E5M2 if e5m2 else bsq.BSQ_E4M3
    bsq.bsq_moe_wgrad(*args, dyt_dtype=cd)
    want, total, group = OE.wgrad(dv, xv, offsets)
    _within(_values(out), want, _product_bound(want, total, group, bf16), "dW")
    first = host(out).copy()
    out.fill_(float("nan"))
    bsq.bsq_moe_wgrad(*args, dyt_dtype=cd)
    assert np.array_equal(first, host(out)), "two runs differ"


LONG = [700, 0, 513, 1, 900, 1200, 3, 880]


@pytest.mark.parametrize("lengths,T,N,K,k,opts", [
    # more big tiles than workgroups that go through them
    (LONG, 1400, 3344, 256, 3, dict(tail=5)), (LONG, 900, 3344, 128, 5, dict(e5m2=True, bf16=False)),
    (LONG, 4200, 3344, 128, 1, dict(gather=False, tail=300)),
    ([500, 0, 300, 1, 200, 257, 30, 12], 650, 4624, 640, 2, dict(tail=2)),
    # contractions of 1, 2, 3 and more steps, odd and even, around the four that share their scales' load
    ([600, 1030], 815, 272, 512, 2, dict(bf16=False)), ([600, 1030], 815, 272, 640, 2, {}),
    ([1024], 512, 16, 896, 2, dict(e5m2=True)), ([513, 511], 512, 240, 1152, 2, dict(bf16=False, e5m2=True))])
def test_matmul_of_long_segments(lengths, T, N, K, k, opts):
    say("moe matmul long", len(lengths), sum(lengths), T, N, K, k, opts)
    _check_product(lengths, T, N, K, k, **opts)


@pytest.mark.parametrize("e5m2,bf16", [(True, True), (False, False)])
def test_wgrad_of_many_big_tiles(e5m2, bf16):
    """More 256 x 256 tiles than workgroups, segments of 0 to 5 steps; 30 tiles
    to an expert (nearly full chunks of 32), and 6 (few of one)."""
    say("wgrad big", e5m2, bf16)
    test_wgrad([3, 0, 1, 2, 5, 1, 0, 2, 1, 4], 1296, 1056, e5m2, bf16)
    test_wgrad([1, 0, 2] * 15, 528, 272, e5m2, bf16)


def test_wgrad_of_long_contractions():
    """Segments of up to 9 steps, around the four that share their scales' load."""
    say("wgrad long")
    test_wgrad([9, 7, 6, 8, 0, 4, 1, 3, 2], 1296, 1056, True, True)


@pytest.mark.parametrize("blocks,N,K", [
    # 64 x 64 tiles, 64 x 128, 128 x 128 (one to a CU, then more), by how many there are
    ([5, 0, 4], 1040, 272), ([3, 0, 1, 6], 1040, 272), ([1, 2, 0, 5, 3, 1], 1040, 272), ([1, 0, 2, 1] * 25, 80, 272)])
@pytest.mark.parametrize("e5m2,bf16", [(True, True), (False, False), (True, False), (False, True)])
def test_wgrad_of_few_tiles(blocks, N, K, e5m2, bf16):
    say("wgrad few tiles", e5m2, bf16)
    test_wgrad(blocks, N, K, e5m2, bf16)


@pytest.mark.parametrize("bf16", [True, False])
def test_swiglu_of_infinite_values(bf16):
    """silu(inf) u = inf u, which takes the block's largest code; -inf has no
    value (-inf 0): its block is left out here, and the rest is as without it."""
    torch = _torch()
    say("swiglu infinite", bf16)
    rng = np.random.default_rng(8)
    x = rng.standard_normal((64, 256)).astype(np.float32)
    dt = torch.bfloat16 if bf16 else torch.float32
    gu = to_dev(x).to(dt)
    plain = [filled(s, torch.uint8, 0x55) for s in ((64, 128), (64, 4), (128, 64), (128, 2))]
    bsq.bsq_swiglu_mx(gu, *plain)
    gu[3, 5] = float("inf")
    gu[40, 70] = -float("inf")
    got = [filled(s, torch.uint8, 0x55) for s in ((64, 128), (64, 4), (128, 64), (128, 2))]
    bsq.bsq_swiglu_mx(gu, *got)
    h, want = host(got[0]), host(plain[0])
    assert h[3, 5] == (0x7E if float(gu[3, 5 + 128]) > 0 else 0xFE)
    keep = np.ones((64, 128), bool)
    keep[3, 0:32] = False
    keep[40, 64:96] = False
    assert np.array_equal(h[keep], want[keep])
    keep_t = np.ones((128, 64), bool)
    keep_t[5, 0:32] = False
    keep_t[70, 32:64] = False
    assert host(got[2])[5, 3] == h[3, 5] and np.array_equal(host(got[2])[keep_t], host(plain[2])[keep_t])


# ------------------------------------------------------------------ gate --

# h of float32 arithmetic: the exponential (2 steps), 1 + e, the division
# (2 steps) and two products, each at most 2^-23 relative
H_OFF = 8 * 2.0 ** -23


def _check_codes(codes, scales, h, fmt, what):
    """codes and scales of values within H_OFF of h: the block exponent lies
    between those of the block's smallest and largest maximum, each value
    between the encodings of its own two bounds."""
    top = np.abs(h).reshape(*h.shape[:-1], -1, 32).max(-1)
    E = scales.astype(np.int64) - 127
    lo = np.maximum(top * (1 - H_OFF), 0)
    hi = top * (1 + H_OFF)
    floor = float(np.float32(1e-10))
    fmax = F.fmax(fmt)
    assert np.all(np.maximum(lo, floor) <= fmax * np.exp2(E.astype(np.float64))), what + ": a block's scale is too small"
    assert np.all(np.maximum(hi, floor) > fmax * np.exp2(E.astype(np.float64) - 1)), what + ": a block's scale is too large"
    got = F.decode(codes, fmt).astype(np.float64)
    unit = np.exp2(-E.astype(np.float64)).repeat(32, -1)
    a, b = h * (1 - H_OFF) * unit, h * (1 + H_OFF) * unit
    enc = lambda v: F.decode(F.encode(np.clip(v, -fmax, fmax).astype(np.float32), fmt), fmt).astype(np.float64)  # noqa: E731
    u, v = enc(np.minimum(a, b) - np.abs(a) * 2.0 ** -23), enc(np.maximum(a, b) + np.abs(a) * 2.0 ** -23)
    bad = np.argwhere((got < u) | (got > v))
    assert len(bad) == 0, (what, len(bad), bad[:3].tolist(), got[tuple(bad[0])], u[tuple(bad[0])], v[tuple(bad[0])])


@pytest.mark.parametrize("R,Fd,bf16,e5m2,train", [
    (1, 32, True, False, False), (32, 32, True, False, True), (33, 96, False, False, False), (96, 160, True, True, True),
    (160, 256, False, False, True), (320, 2048, True, False, True), (31, 2048, True, False, False), (128, 64, False, True, True)])
def test_swiglu(R, Fd, bf16, e5m2, train):
    torch = _torch()
    say("swiglu", R, Fd, bf16, e5m2, train)
    rng = np.random.default_rng(R + Fd)
    x = (rng.standard_normal((R, 2 * Fd)) * np.exp(rng.uniform(-3, 3, (R, 1)))).astype(np.float32)
    x[0, :8] = [0.0, -0.0, 100.0, -100.0, 88.8, -88.8, 1e-30, -1e-30]
    if R > 4:
        x[4] = 0.0
    gu, v = _dev_values(x, bf16)
    fmt = F.E5M2 if e5m2 else F.E4M3
    cd = bsq.BSQ_E5M2 if e5m2 else bsq.BSQ_E4M3
    u8 = lambda *s: filled(s, torch.uint8, 0x55)  # noqa: E731
    h, hs = u8(R, Fd), u8(R, Fd // 32)
    want = OE.swiglu(v[:, :Fd], v[:, Fd:])
    if not train:
        bsq.bsq_swiglu_mx(gu, h, hs, code_dtype=cd)
        _check_codes(host(h), host(hs), want, fmt, "h")
        return
    ht, hts, kept, ks = u8(Fd, R), u8(Fd, R // 32), u8(R, 2 * Fd), u8(R, 2 * Fd // 32)
    bsq.bsq_swiglu_mx(gu, h, hs, ht, hts, kept, ks, code_dtype=cd)
    _check_codes(host(h), host(hs), want, fmt, "h")
    _check_codes(host(ht), host(hts), np.ascontiguousarray(want.T), fmt, "ht")
    rk = OQ.mx(v.astype(np.float32), fmt)
    assert_bytes_equal(host(kept), rk[0], "kept")
    assert_bytes_equal(host(ks), rk[1], "kept scales")
    # each output alone, the same bytes
    for parts in (dict(ht=ht.clone(), ht_scales=hts.clone()), dict(kept=kept.clone(), kept_scales=ks.clone())):
        h2, hs2 = u8(R, Fd), u8(R, Fd // 32)
        for p in parts.values():
            p.fill_(0x55)
        bsq.bsq_swiglu_mx(gu, h2, hs2, code_dtype=cd, **parts)
        assert_bytes_equal(host(h2), host(h), "h of a part")
        for p, whole in zip(parts.values(), (ht, hts) if "ht" in parts else (kept, ks)):
            assert_bytes_equal(host(p), host(whole), "a part")
    dh, dv = _dev_values(rng.standard_normal((R, Fd)), bf16)
    dgu = filled((R, 2 * Fd), dh.dtype, float("nan"))
    bsq.bsq_swiglu_mx_backward(kept, ks, dh, dgu, code_dtype=cd)
    kv = F.decode(rk[0], fmt).astype(np.float64) * F.decode_e8m0(rk[1]).astype(np.float64).repeat(32, -1)
    g, u = kv[:, :Fd], kv[:, Fd:]
    dg, du = OE.swiglu_backward(g, u, dv)
    s, q = OE.scores(g, True), OE.scores(-g, True)
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    # 1 - s is off by a step of s, which g multiplies
    off_g = H_OFF * np.abs(dv * u * s) * (1 + np.abs(g)) * 2
    off_u = H_OFF * np.abs(dv * g * s)
    got = _values(dgu)
    _within(got[:, :Fd], dg, off_g + half * (np.abs(dg) + off_g) + TINY, "dg")
    _within(got[:, Fd:], du, off_u + half * (np.abs(du) + off_u) + TINY, "du")


# ----------------------------------------------- streams, graphs, offsets --

def _layer(T, H, Fd, E, k, seed=0):
    """A small expert layer: its buffers, and one forward and backward pass
    through every operator, as a training step makes them."""
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    cap = bsq.bsq_moe_capacity(T * k, E, 128)
    x, dout, logits = rand(T, H).bfloat16(), rand(T, H).bfloat16(), rand(T, E)

    def weight(n, m):
        c, s = u8(E, n, m), u8(E, n, m // 32)
        bsq.bsq_quant_mx((rand(E * n, m) * 0.05), c.view(E * n, m), s.view(E * n, m // 32))
        return c, s

    w1, w2 = weight(2 * Fd, H), weight(H, Fd)
    w1t, w2t = weight(H, 2 * Fd), weight(Fd, H)
    b = dict(ids=i32(T, k), w=torch.zeros(T, k, device="cuda"), off=i32(E + 1), cnt=i32(E), rows=i32(cap), pos=i32(T, k),
             ws=u8(bsq.bsq_moe_plan_workspace_bytes(T * k, E)), xc=u8(cap, H), xs=u8(cap, H // 32), xt=u8(H, cap),
             xts=u8(H, cap // 32), gu=bf(cap, 2 * Fd), h=u8(cap, Fd), hs=u8(cap, Fd // 32), ht=u8(Fd, cap),
             hts=u8(Fd, cap // 32), kept=u8(cap, 2 * Fd), ks=u8(cap, 2 * Fd // 32), y=bf(cap, H), out=bf(T, H),
             dw=torch.zeros(T, k, device="cuda"), dl=torch.zeros(T, E, device="cuda"), dy=u8(cap, H), dys=u8(cap, H // 32),
             dyt=u8(H, cap), dyts=u8(H, cap // 32), dW2=bf(E, H, Fd), dh=bf(cap, Fd), dgu=bf(cap, 2 * Fd),
             dguc=u8(cap, 2 * Fd), dgus=u8(cap, 2 * Fd // 32), dgut=u8(2 * Fd, cap), dguts=u8(2 * Fd, cap // 32),
             dW1=bf(E, 2 * Fd, H), dxr=bf(cap, H), dx=bf(T, H))
    e5 = bsq.BSQ_E5M2

    def step():
        bsq.bsq_moe_route(logits, b["ids"], b["w"], score=bsq.BSQ_SIGMOID, scale=2.5)
        bsq.bsq_moe_plan(b["ids"], b["off"], b["cnt"], b["rows"], b["pos"], b["ws"], align=128)
        bsq.bsq_moe_gather_mx(x, b["rows"], k, b["xc"], b["xs"], b["xt"], b["xts"])
        bsq.bsq_moe_matmul(b["xc"], b["xs"], *w1, b["off"], b["gu"])
        bsq.bsq_swiglu_mx(b["gu"], b["h"], b["hs"], b["ht"], b["hts"], b["kept"], b["ks"])
        bsq.bsq_moe_matmul(b["h"], b["hs"], *w2, b["off"], b["y"])
        bsq.bsq_moe_combine(b["y"], b["pos"], b["out"], weights=b["w"])
        bsq.bsq_moe_combine_backward(b["y"], b["pos"], dout, b["dw"])
        bsq.bsq_moe_route_backward(logits, b["ids"], b["dw"], b["dl"], score=bsq.BSQ_SIGMOID, scale=2.5)
        bsq.bsq_moe_gather_mx(dout, b["rows"], k, b["dy"], b["dys"], b["dyt"], b["dyts"], weights=b["w"], code_dtype=e5)
        bsq.bsq_moe_wgrad(b["dyt"], b["dyts"], b["ht"], b["hts"], b["off"], b["dW2"], dyt_dtype=e5)
        bsq.bsq_moe_matmul(b["dy"], b["dys"], *w2t, b["off"], b["dh"], a_dtype=e5)
        bsq.bsq_swiglu_mx_backward(b["kept"], b["ks"], b["dh"], b["dgu"])
        bsq.bsq_quant_mx(b["dgu"], b["dguc"], b["dgus"], code_dtype=e5)
        bsq.bsq_quant_mx(b["dgu"], b["dgut"], b["dguts"], axis=0, code_dtype=e5)
        bsq.bsq_moe_wgrad(b["dgut"], b["dguts"], b["xt"], b["xts"], b["off"], b["dW1"], dyt_dtype=e5)
        bsq.bsq_moe_matmul(b["dguc"], b["dgus"], *w1t, b["off"], b["dxr"], a_dtype=e5)
        bsq.bsq_moe_combine(b["dxr"], b["pos"], b["dx"])

    return dict(x=x, dout=dout, logits=logits), b, step


def _snapshot(b):
    torch = _torch()
    torch.cuda.synchronize()
    return {n: t.clone() for n, t in b.items() if n != "ws"}


def _same(a, b, what):
    torch = _torch()
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), f"{what}: {n} differs"


def test_a_layers_step_replays_as_a_graph():
    torch = _torch()
    T, H, Fd, E, k = 700, 256, 384, 6, 2
    say("layer graph", T, H, Fd, E, k)
    ins, b, step = _layer(T, H, Fd, E, k)
    step()
    torch.cuda.synchronize()
    assert all(torch.isfinite(b[n].float()).all() for n in ("out", "dx", "dW1", "dW2", "dl"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(3):
        for t in ins.values():
            t.copy_(torch.randn(t.shape, device="cuda"))
        for n, t in b.items():
            t.zero_() if n != "ws" else t.fill_(0x7F)
        torch.cuda.synchronize()
        graph.replay()
        got = _snapshot(b)
        junk = torch.randn(1 << 20, device="cuda").sum()  # unrelated eager work
        step()
        _same(got, _snapshot(b), f"replay {rep}")
        del junk


def test_a_layers_step_runs_on_the_callers_stream():
    torch = _torch()
    say("layer stream")
    ins, b, step = _layer(130, 128, 128, 5, 3, seed=1)
    step()
    want = _snapshot(b)
    for t in b.values():
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    _same(want, _snapshot(b), "side stream")


def test_products_whose_offsets_pass_32_bits():
    """A's bytes and the output's elements each pass 2^32 / 2^31: the rows at
    the far end give what the same rows give near the start."""
    torch = _torch()
    T, K, N = 1_050_000, 4224, 64
    say("far rows of A", T, K)
    a = torch.zeros(T, K, dtype=torch.uint8, device="cuda")
    sa = torch.full((T, K // 32), 127, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(0)
    c, s, _ = _operand(rng, (48, K), F.E4M3)
    b, sb, _ = _operand(rng, (2, N, K), F.E4M3)
    for at in (0, T - 48):
        a[at:at + 48], sa[at:at + 48] = to_dev(c), to_dev(s)
    off = to_dev(np.array([0, 20, 48], np.int32))
    outs = []
    for at in (0, T - 48):
        out = filled((48, N), torch.float32, float("nan"))
        rows = torch.arange(at, at + 48, dtype=torch.int32, device="cuda")
        bsq.bsq_moe_matmul(a, sa, to_dev(b), to_dev(sb), off, out, rows=rows)
        outs.append(host(out))
    assert np.array_equal(outs[0], outs[1]) and np.any(outs[0] != 0)
    del a, sa
    cap, N, K = 540_000, 4096, 128
    say("far rows of the output", cap, N)
    c, s, _ = _operand(rng, (64, K), F.E4M3)
    b, sb, _ = _operand(rng, (1, N, K), F.E4M3)
    rows = (torch.arange(cap, dtype=torch.int32, device="cuda") % 64)
    out = filled((cap, N), torch.bfloat16, float("nan"))
    bsq.bsq_moe_matmul(to_dev(c), to_dev(s), to_dev(b), to_dev(sb), to_dev(np.array([0, cap], np.int32)), out, rows=rows)
    assert torch.equal(out.view(torch.int16)[: cap // 64 * 64].view(-1, 64 * N)[-1], out.view(torch.int16)[:64].reshape(-1))
    assert torch.equal(out.view(torch.int16).view(-1, N)[-1], out.view(torch.int16)[(cap - 1) % 64])


def test_rows_whose_offsets_pass_32_bits():
    torch = _torch()
    cap, H, k = 290_016, 8192, 1
    say("far rows of y and codes", cap, H)
    x = torch.randn(64, H, device="cuda").bfloat16()
    rows = torch.arange(cap, dtype=torch.int32, device="cuda") % 64
    codes, scales = empty((cap, H), torch.uint8), empty((cap, H // 32), torch.uint8)
    codes_t, scales_t = empty((H, cap), torch.uint8), empty((H, cap // 32), torch.uint8)
    bsq.bsq_moe_gather_mx(x, rows, k, codes, scales, codes_t, scales_t)
    # 290016 = 64 * 4531 + 32: the last 32 rows are the first 32 tokens again
    assert torch.equal(codes[-32:], codes[:32]) and torch.equal(scales[-32:], scales[:32])
    assert torch.equal(codes_t[:, -32:], codes_t[:, :32]) and torch.equal(scales_t[:, -1], scales_t[:, 0])
    del codes, codes_t
    y = torch.zeros(cap, H, dtype=torch.bfloat16, device="cuda")
    y[-3:] = x[:3]
    pos = torch.tensor([[cap - 3], [cap - 2], [cap - 1]], dtype=torch.int32, device="cuda")
    out = empty((3, H), torch.bfloat16)
    bsq.bsq_moe_combine(y, pos, out)
    assert torch.equal(out, x[:3])
    dw = empty((3, 1), torch.float32)
    bsq.bsq_moe_combine_backward(y, pos, x[:3].contiguous(), dw)
    assert torch.allclose(dw[:, 0], (x[:3].double() ** 2).sum(1).float(), rtol=1e-5)
