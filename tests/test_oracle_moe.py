"""Pins of oracle/moe.py that do not come from itself: gradients against
central differences, the order of rows against its defining properties, the
ragged products against one matrix product per expert, closed forms."""
import numpy as np
import pytest

from oracle import moe as OE


def test_scores_closed_forms():
    assert np.allclose(OE.scores([[0.0, 0.0]], False), [[0.5, 0.5]])
    assert np.allclose(OE.scores([[np.log(3.0), 0.0]], False), [[0.75, 0.25]])
    assert np.allclose(OE.scores([[0.0, np.log(3.0)]], True), [[0.5, 0.75]])
    assert np.array_equal(OE.scores([[-np.inf, -np.inf]], False), [[0.0, 0.0]])
    assert np.array_equal(OE.scores([[-np.inf, 0.0]], False), [[0.0, 1.0]])


def test_route_ties_bias_and_groups():
    x = np.array([[1.0, 3.0, 3.0, 0.0, 2.0, 2.0]])
    assert OE.route(x, 3)[0].tolist() == [[1, 2, 4]]
    # the bias steers the choice, not the weight
    ids, w, p = OE.route(x, 1, bias=[0, 0, 0, 9.0, 0, 0], renorm=False, scale=2.0)
    assert ids.tolist() == [[3]] and np.allclose(w, 2.0 * p[0, 3])
    # groups (1,3) (3,0) (2,2): by the largest the first, by two the first (its index is lower) then the third
    assert OE.route(x, 2, groups=3, top_groups=1, group_top=1)[0].tolist() == [[1, 0]]
    assert OE.route(x, 4, groups=3, top_groups=2, group_top=1)[0].tolist() == [[1, 2, 0, 3]]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(sigmoid, renorm):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 7))
    ids = OE.route(x, 3, sigmoid=sigmoid)[0].astype(np.int64)
    dw, ds = rng.standard_normal((3, 3)), rng.standard_normal((3, 7))

    def loss(x):
        p = OE.scores(x, sigmoid)
        w = np.take_along_axis(p, ids, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return (w * 1.7 * dw).sum() + (p * ds).sum()

    got = OE.route_backward(x, ids, dw, ds, sigmoid, renorm, 1.7)[0]
    h = 1e-6
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = h
        assert abs((loss(x + d) - loss(x - d)) / (2 * h) - got[i]) < 1e-8


@pytest.mark.parametrize("align", [1, 32, 128])
def test_plan_is_a_stable_sort(align):
    rng = np.random.default_rng(6)
    ids = rng.integers(-1, 5, (40, 3))
    offsets, counts, rows, pos = OE.plan(ids, 5, align, 120 + 5 * (align - 1))
    flat = ids.reshape(-1)
    assert np.all(offsets % align == 0) and counts.sum() == (flat >= 0).sum()
    for e in range(5):
        seg = rows[offsets[e]:offsets[e + 1]]
        assert np.array_equal(seg[:counts[e]], np.nonzero(flat == e)[0]) and np.all(seg[counts[e]:] == -1)
    assert np.all(rows[offsets[5]:] == -1)
    held = flat >= 0
    assert np.array_equal(rows[pos.reshape(-1)[held]], np.nonzero(held)[0]) and np.all(pos.reshape(-1)[~held] == -1)


def test_combine_and_products_undo_the_order():
    """gather, one matrix per expert, weighted sum = the same token by token."""
    rng = np.random.default_rng(7)
    T, E, k, K, N = 9, 4, 2, 16, 5
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    x, b, w = rng.standard_normal((T, K)), rng.standard_normal((E, N, K)), rng.random((T, k))
    offsets, _, rows, pos = OE.plan(ids, E, 4, 40)
    y = OE.product(x, b, offsets, 40, rows, k)[0]
    out, _ = OE.combine(y, pos, w)
    want = np.stack([sum(w[t, j] * (b[ids[t, j]] @ x[t]) for j in range(k)) for t in range(T)])
    assert np.allclose(out, want, atol=1e-12)
    dout = rng.standard_normal((T, N))
    dw, _ = OE.combine_backward(y, pos, dout)
    assert np.allclose(dw, [[dout[t] @ (b[ids[t, j]] @ x[t]) for j in range(k)] for t in range(T)], atol=1e-12)
    # the gradient of sum_t dout . out with respect to each matrix: w dout x^T summed over its rows
    grad = np.zeros_like(b)
    for t in range(T):
        for j in range(k):
            grad[ids[t, j]] += w[t, j] * np.outer(dout[t], x[t])
    got = np.stack([OE.gather(dout, rows, k, w)[lo:hi].T.astype(np.float64) @
                    OE.gather(x, rows, k)[lo:hi].astype(np.float64) for lo, hi in zip(offsets[:-1], offsets[1:])])
    assert np.allclose(got, grad, atol=1e-5)


def test_wgrad_is_a_product_per_segment():
    rng = np.random.default_rng(8)
    dyt, xt = rng.standard_normal((6, 48)), rng.standard_normal((5, 48))
    out = OE.wgrad(dyt, xt, [0, 16, 16, 40])[0]
    assert np.allclose(out[0], dyt[:, :16] @ xt[:, :16].T) and np.all(out[1] == 0)
    assert np.allclose(out[2], sum(np.outer(dyt[:, r], xt[:, r]) for r in range(16, 40)))


def test_swiglu_and_its_gradient():
    assert np.allclose(OE.swiglu([0.0, np.log(3.0)], [5.0, 4.0]), [0.0, 3.0 * np.log(3.0)])
    rng = np.random.default_rng(9)
    g, u, dh = rng.standard_normal((3, 50)) * 3
    dg, du = OE.swiglu_backward(g, u, dh)
    h = 1e-6
    assert np.allclose((OE.swiglu(g + h, u) - OE.swiglu(g - h, u)) / (2 * h) * dh, dg, atol=1e-7)
    assert np.allclose((OE.swiglu(g, u + h) - OE.swiglu(g, u - h)) / (2 * h) * dh, du, atol=1e-7)
