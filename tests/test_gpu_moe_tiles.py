"""The ragged products' kernels by the tiles that they take: index arrays that
no plan writes, in front of each of them."""
import numpy as np
import pytest

import block_scaled_precision_blockwise_amd as bsq
from oracle import formats as F
from oracle import quantize as OQ

from gpu_helpers import filled, say, to_dev

pytestmark = pytest.mark.gpu

GUARD = 64  # rows kept on both sides of an output


def _torch():
    import torch
    return torch


def _codes(rng, shape, fmt=F.E4M3):
    c, s = OQ.mx(rng.standard_normal(shape).astype(np.float32), fmt)
    return to_dev(c), to_dev(s)


def _guarded(n, shape, dtype):
    """(the whole buffer of `n` outputs of `shape`, the outputs between its guards)."""
    t = filled((n + 2 * GUARD, *shape), dtype, 3.0)
    return t, t[GUARD:GUARD + n]


def _offsets(rng, E, cap):
    """Offsets that do not ascend, and such as are out of range."""
    up = np.array([i % 2 * cap for i in range(E + 1)])
    return [up, cap - up, np.array([i % 2 * (2 ** 31 - 1) for i in range(E + 1)]),
            rng.integers(-2 ** 31, 2 ** 31, E + 1), rng.integers(-5, cap + 5, E + 1), np.full(E + 1, cap + 3),
            np.full(E + 1, -1), np.array([cap] + [0] * E)]


WILD = [  # E, cap, N, K: by the tile that the sizes take
    pytest.param(3, 300, 80, 256, id="32x64"), pytest.param(3, 803, 784, 256, id="64x64"),
    pytest.param(3, 803, 1296, 128, id="64x128 three stages"), pytest.param(3, 803, 2576, 256, id="64x128"),
    pytest.param(20, 450, 720, 128, id="64x64 few rows"), pytest.param(3, 2001, 5136, 384, id="256x256"),
    pytest.param(130, 2001, 272, 256, id="many segments")]


@pytest.mark.parametrize("E,cap,N,K", WILD)
def test_matmul_keeps_inside_its_arrays(E, cap, N, K):
    torch = _torch()
    rng = np.random.default_rng(cap + N)
    T, k = cap, 2
    a, sa = _codes(rng, (T, K))
    b, sb = _codes(rng, (E, N, K))
    whole, out = _guarded(cap, (N,), torch.bfloat16)
    for i, off in enumerate(_offsets(rng, E, cap)):
        for with_rows in (True, False):
            say("wild offsets", E, cap, N, K, i, with_rows)
            rows = rng.choice(np.array([-2 ** 31, -1, 0, T * k - 1, T * k, 2 ** 31 - 1]), cap).astype(np.int32)
            kw = dict(rows=to_dev(rows), k=k) if with_rows else {}
            bsq.bsq_moe_matmul(a, sa, b, sb, to_dev(off.astype(np.int32)), out, **kw)
            assert torch.all(whole[:GUARD] == 3.0) and torch.all(whole[-GUARD:] == 3.0)


@pytest.mark.parametrize("E,cap,N,K", [
    pytest.param(3, 768, 80, 272, id="64x64"), pytest.param(3, 768, 1296, 272, id="64x128"),
    pytest.param(6, 768, 1040, 272, id="128x128"), pytest.param(8, 2048, 1536, 1536, id="256x256"),
    pytest.param(4, 6144, 2048, 2048, id="256x256 dealt")])
def test_wgrad_keeps_inside_its_arrays(E, cap, N, K):
    torch = _torch()
    rng = np.random.default_rng(cap + N)
    dy, sd = _codes(rng, (N, cap))
    x, sx = _codes(rng, (K, cap))
    whole = filled((E + 2, N, K), torch.bfloat16, 3.0)
    for i, off in enumerate(_offsets(rng, E, cap)):
        say("wgrad wild offsets", E, cap, N, K, i)
        bsq.bsq_moe_wgrad(dy, sd, x, sx, to_dev(off.astype(np.int32)), whole[1:-1])
        assert torch.all(whole[0] == 3.0) and torch.all(whole[-1] == 3.0)
        assert torch.isfinite(whole).all()
    # not multiples of 128: cut down to one
    off = np.sort(rng.integers(0, cap + 1, E + 1)).astype(np.int32)
    say("wgrad unaligned offsets", E, cap, N, K)
    bsq.bsq_moe_wgrad(dy, sd, x, sx, to_dev(off), whole[1:-1])
    got = whole[1:-1].clone()
    bsq.bsq_moe_wgrad(dy, sd, x, sx, to_dev(off // 128 * 128), whole[1:-1])
    assert torch.equal(got.view(torch.int16), whole[1:-1].contiguous().view(torch.int16)) and torch.any(got != 0)
