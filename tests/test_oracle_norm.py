"""The norm's oracle: hand-made rows, and the gradient against differences."""
import numpy as np
import pytest

from oracle import norm


def test_rows():
    y, mean, rstd = norm.forward([[1.0, 3.0], [5.0, 5.0]], eps=0.0625)
    assert mean.tolist() == [2.0, 5.0]
    assert np.allclose(rstd, [1 / np.sqrt(1.0625), 4.0])
    assert np.allclose(y, [[-1 / np.sqrt(1.0625), 1 / np.sqrt(1.0625)], [0, 0]])
    y, mean, rstd = norm.forward([[3.0, 4.0]], gamma=np.array([2.0, 1.0]), beta=np.array([0.0, 1.0]), eps=0.0, rms=True)
    assert mean[0] == 0 and np.allclose(y, [[6 / np.sqrt(12.5), 4 / np.sqrt(12.5) + 1]])


@pytest.mark.parametrize("rms", [False, True])
def test_gradients_against_differences(rms):
    g = np.random.default_rng(0)
    x, dy, gamma, beta = g.standard_normal((3, 7)) + 0.5, g.standard_normal((3, 7)), g.uniform(0.5, 2, 7), g.standard_normal(7)
    f = lambda x, gamma, beta: float((norm.forward(x, gamma, beta, 1e-3, rms)[0] * dy).sum())  # noqa: E731
    args, h = (x, gamma, beta), 1e-6
    for i, grad in enumerate(norm.backward(x, dy, gamma, 1e-3, rms)):
        for at in np.ndindex(args[i].shape):
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[i][at] += h
            down[i][at] -= h
            # h^2 times a third derivative below 10^3 here, and 1e-15 / h of rounding
            assert abs((f(*up) - f(*down)) / (2 * h) - grad[at]) < 1e-7
