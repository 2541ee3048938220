"""The norm on rows that hold infinities or NaN: every kernel, both kinds, every operand."""
import pytest
import torch

import block_scaled_precision_blockwise_amd as bsq
from gpu_helpers import say
from test_gpu_mx4 import E4M3, E5M2, E8M0, empty, gen, u8
from test_gpu_norm import KIND

pytestmark = pytest.mark.gpu

f32, bf16 = torch.float32, torch.bfloat16
CODES = {"none": None, "e4m3": E4M3, "e5m2": E5M2, "e2m1": u8}


def same(a, b):
    return torch.equal(a.view(u8), b.view(u8))


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt", [f32, bf16])
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("C", [96, 1000, 1024, 2048, 4096, 8192, 16384, 16416, 20001])
def test_infinities_and_nan_make_their_whole_row_nan(C, code, dt, rms):
    """In y, in codes of 8 bits, as the scales of 4-bit ones and in rstd; the other rows are as without them."""
    if code != "none" and C % 32:
        pytest.skip("codes come in whole blocks")
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
