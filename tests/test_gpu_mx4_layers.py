"""Steps of layers in 4 bits that tests/test_gpu_mx4_use.py does not take: streams that are named."""
import pytest
import torch

import block_scaled_precision_blockwise_amd as bsq
from gpu_helpers import say
from test_gpu_mx4 import E8M0, empty, exact_operand, u8
from test_gpu_mx4_use import randn

pytestmark = pytest.mark.gpu
f32, bf16 = torch.float32, torch.bfloat16


# ------------------------------------------------------------------ streams --

def calls():
    """(name, call(stream), its outputs) of each call on 4-bit operands and of the norm."""
    M, K, N = 64, 288, 208
    x, dy, gamma = randn(M, K, seed=1), randn(M, K, seed=2), 1 + 0.1 * randn(K, seed=3)
    codes, scales = empty(M, K // 2), empty(M, K // 32, dtype=E8M0)
    yield "bsq_quant_fp4", lambda s: bsq.bsq_quant_fp4(x, codes, scales, stream=s), (codes, scales)
    (a, sa), (b, sb) = exact_operand((1, M, K), "e4m3", 4), exact_operand((1, N, K), "e2m1", 5)
    out = empty(1, M, N, dtype=f32)
    yield "bsq_scaled_matmul_mxfp4", lambda s: bsq.bsq_scaled_matmul_mxfp4(a, b, sa, sb, out, stream=s), (out,)
    offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    rows = empty(M, N, dtype=bf16)
    yield ("bsq_moe_matmul_mxfp4", lambda s: bsq.bsq_moe_matmul_mxfp4(a[0], sa[0], b, sb, offsets, rows, stream=s),
           (rows,))
    y, mean, rstd = empty(M, K, dtype=f32), empty(M, dtype=f32), empty(M, dtype=f32)
    yield "bsq_norm_mx", lambda s: bsq.bsq_norm_mx(x, y=y, gamma=gamma, mean=mean, rstd=rstd, stream=s), (y, mean, rstd)
    m, r = randn(M, seed=6), 1 + 0.1 * randn(M, seed=7)
    dx, dg, db = empty(M, K, dtype=f32), empty(K, dtype=f32), empty(K, dtype=f32)
    space = empty(bsq.bsq_norm_backward_workspace_bytes(M, K))
    yield ("bsq_norm_backward", lambda s: bsq.bsq_norm_backward(x, dy, r, dx, mean=m, gamma=gamma, dgamma=dg, dbeta=db,
                                                                workspace=space, stream=s), (dx, dg, db))


def test_a_named_stream_is_the_one_that_is_used():
    """The outputs are there when the named stream is done, while the current stream has yet to come through the work
    that was put on it before the call."""
    busy, named = torch.cuda.Stream(), torch.cuda.Stream()
    big = torch.zeros(1 << 28, device="cuda")
    for name, call, outs in calls():
        say("named stream", name)
        call(None)
        want = [t.clone() for t in outs]
        for t in outs:
            t.view(u8).fill_(0xFF)  # NaN in every type
        torch.cuda.synchronize()
        with torch.cuda.stream(busy):
            for _ in range(500):  # 2 GiB of traffic each, 200 ms in all
                big.add_(1.0)
            held_up = torch.cuda.Event()
            held_up.record()
            call(named)
        with torch.cuda.stream(named):
            got = [t.clone() for t in outs]
        named.synchronize()
        assert not held_up.query(), "the current stream was done first: nothing is shown"
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g.view(u8), w.view(u8)), name
