"""Layer and rms norm and their gradients in float64.  TEST INFRASTRUCTURE
ONLY.  Written from the definitions; the gradient is pinned by differences of
the forward."""
from __future__ import annotations

import numpy as np


def forward(x, gamma=None, beta=None, eps=1e-5, rms=False):
    """x [R, C] -> (y, mean [R], rstd [R])."""
    x = np.asarray(x, dtype=np.float64)
    mean = np.zeros(x.shape[0]) if rms else x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    return (y if beta is None else y + beta), mean, rstd


def backward(x, dy, gamma=None, eps=1e-5, rms=False):
    """Gradients of sum(forward(x) dy): (dx [R, C], dgamma [C], dbeta [C])."""
    xn, _, rstd = forward(x, eps=eps, rms=rms)
    dy = np.asarray(dy, dtype=np.float64)
    d = dy if gamma is None else dy * gamma
    dx = d - xn * (d * xn).mean(1, keepdims=True)
    if not rms:
        dx = dx - d.mean(1, keepdims=True)
    return dx * rstd[:, None], (dy * xn).sum(0), dy.sum(0)
