"""Pins of the 4-bit quantizers' oracle."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import formats as F
from oracle import fp4


def test_encode_is_the_nearest_value_ties_to_even():
    g = np.random.default_rng(0)
    mids = (fp4.VALUES[1:] + fp4.VALUES[:-1]) / 2
    near = np.concatenate([np.nextafter(mids.astype(np.float32), np.float32(s)) for s in (0, 9)])
    v = np.concatenate([mids, near, fp4.VALUES, g.uniform(0, 7, 500)]).astype(np.float32)
    v = np.concatenate([v, -v])
    for x, c in zip(v, fp4.encode(v)):
        a = min(abs(Fraction(float(x))), Fraction(6))
        d = [abs(a - Fraction(t)) for t in fp4.VALUES.tolist()]
        best = [i for i in range(8) if d[i] == min(d)]
        want = best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0)
        assert (c & 7) == want and bool(c & 8) == bool(np.signbit(x)), x
    assert fp4.encode(np.float32([mids[0], mids[1], 100.0, -0.0])).tolist() == [0, 2, 7, 8]


@pytest.mark.parametrize("seed", range(3))
def test_mxfp4_scale_is_the_least_power_of_two(seed):
    g = np.random.default_rng(seed)
    x = (g.standard_normal((7, 96)) * np.exp2(g.integers(-60, 60, (7, 1)))).astype(np.float32)
    x[0, :32] = 0
    x[1, 32:64] = np.float32(6 * 2.0 ** 5) * (np.arange(32) == 3)
    x[2, :32] = np.nextafter(np.float32(6 * 2.0 ** -7), np.float32(1)) * (np.arange(32) == 0)
    codes, scales = fp4.mxfp4(x)
    E = scales.astype(int) - 127
    amax = np.maximum(np.abs(x.reshape(7, 3, 32)).max(-1), np.float32(1e-10)).astype(np.float64)
    assert np.all(amax <= 6 * 2.0 ** E) and np.all(amax > 6 * 2.0 ** (E - 1))
    assert E[1, 1] == 5 and E[2, 0] == -6
    top = np.abs(F.decode_e2m1(F.unpack_e2m1(codes))).reshape(7, 3, 32).max(-1)
    assert np.all((top >= 3) | (amax <= np.float64(np.float32(1e-10))))


def test_nvfp4():
    x = np.zeros((3, 32), np.float32)
    x[0, :16] = np.arange(16) - 8.0          # amax 8, 8 / 6 = 1.333 -> 1.375 in e4m3
    x[1, 16:] = 1e-6                         # below the smallest scale
    x[2, 3] = 1e6                            # above the largest
    codes, scales = fp4.nvfp4(x)
    s = F.decode(scales, F.E4M3)
    assert s[0, 0] == 1.375 and s[0, 1] == 2.0 ** -9 and s[1, 1] == 2.0 ** -9 and s[2, 0] == 448
    v = F.decode_e2m1(F.unpack_e2m1(codes))
    # -8 / 1.375 = -5.82 -> -6, -5 / 1.375 = -3.64 -> -4, 1 / 1.375 = 0.73 -> 0.5
    assert v[0, 0] == -6 and v[0, 3] == -4 and v[0, 9] == 0.5 and v[2, 3] == 6 and not v[1].any()
    c2, s2 = fp4.nvfp4(x / 4, 4.0)
    assert np.array_equal(c2, codes) and np.array_equal(s2, scales)
