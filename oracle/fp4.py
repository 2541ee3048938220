"""Quantizers to 4-bit codes: float values -> (e2m1 codes, scales).  TEST
INFRASTRUCTURE ONLY.

numpy float32 arithmetic (IEEE-754, round to nearest even, true division),
codes from the table of e2m1's values.

mxfp4
    blocks of 32 along the last axis with an e8m0 scale: the rule of
    ``quantize.mx`` with fmax 6.
nvfp4
    blocks of 16 with an e4m3 scale: y = x * factor, s = e4m3(max(amax / 6,
    2^-9)) and at most 448, codes of y / s, values beyond 6 become 6.

jax.nn.scaled_matmul's Notes name the formats and no scale rule.  Pinned by
the defining inequality of the exponent, by the nearest of e2m1's values with
exact rationals, and by ties.
"""
from __future__ import annotations

import numpy as np

from . import formats as F

FMAX = 6.0
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode(v: np.ndarray) -> np.ndarray:
    """Codes (one per element) of finite float32 values, nearest, ties to the
    even code, beyond 6 the largest; the sign of zero is kept."""
    a = np.minimum(np.abs(np.asarray(v, dtype=np.float64)), FMAX)
    hi = np.searchsorted(VALUES, a, side="left")
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - VALUES[lo], VALUES[hi] - a
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | (np.signbit(v) * 8)).astype(np.uint8)


def mxfp4(x: np.ndarray):
    """x[..., C] float32 -> (packed codes [..., C / 2], E8M0 bytes [..., C / 32])."""
    x = np.asarray(x, dtype=np.float32)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = np.maximum(np.abs(b).max(-1), np.float32(1e-10)).astype(np.float64)
    m, e = np.frexp(amax / FMAX)  # amax / 6 = m 2^e, m in [1/2, 1)
    # m rounds to 1/2 only where amax is 6 times a power of two
    E = np.where(amax == FMAX * np.ldexp(0.5, e), e - 1, e)
    assert np.all(amax <= FMAX * np.ldexp(1.0, E)) and np.all(amax > FMAX * np.ldexp(1.0, E - 1))
    codes = encode(np.ldexp(b.astype(np.float64), -E[..., None])).reshape(x.shape)
    return F.pack_e2m1(codes), (E + 127).astype(np.uint8)


def nvfp4(x: np.ndarray, factor=1.0):
    """x[..., C] float32 -> (packed codes [..., C / 2], e4m3 scale bytes [..., C / 16])."""
    y = np.asarray(x, dtype=np.float32) * np.float32(factor)
    b = y.reshape(*y.shape[:-1], y.shape[-1] // 16, 16)
    s = np.clip(np.abs(b).max(-1) / np.float32(6.0), np.float32(2.0 ** -9), np.float32(448.0))
    scales = F.encode(s, F.E4M3)
    codes = encode(b / F.decode(scales, F.E4M3).astype(np.float32)[..., None]).reshape(y.shape)
    return F.pack_e2m1(codes), scales
