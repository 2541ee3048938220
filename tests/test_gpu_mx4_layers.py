"""Steps of layers in 4 bits that tests/test_gpu_mx4_use.py does not take: streams that are named, scales at both ends
of their range, the experts' backward pass, nvfp4 operands value by value."""
import pytest
import torch

import block_scaled_precision_blockwise_amd as bsq
from gpu_helpers import say
from mx4_sizes import DENSE
from test_gpu_mx4 import E4M3, E8M0, TABLE, decode, dense, empty, exact_operand, experts_reference, ragged, u8
from test_gpu_mx4_use import quant, randn

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
    """A named stream that is being captured takes the call into its graph, whatever the current stream: nothing is written
    until the graph is replayed.  (Streams may share a hardware queue, so that one held up may hold up the other.)"""
    named, current = torch.cuda.Stream(), torch.cuda.Stream()
    for name, call, outs in calls():
        say("named stream", name)
        call(None)
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        untouched = lambda: all(bool((t.view(u8) == 0xFF).all()) for t in outs)  # noqa: E731
        for t in outs:
            t.view(u8).fill_(0xFF)  # NaN in every type
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=named):
            with torch.cuda.stream(current):
                call(named)
        torch.cuda.synchronize()
        assert untouched(), name
        for _ in range(2):
            g.replay()
            torch.cuda.synchronize()
            for got, w in zip(outs, want):
                assert torch.equal(got.view(u8), w.view(u8)), name
            for t in outs:
                t.view(u8).fill_(0xFF)


# --------------------------------------------------------- scales far apart --

@pytest.mark.parametrize("kind", ["e2m1", "e4m3", "e5m2"])
@pytest.mark.parametrize("tile", [t for t in DENSE if t != "t256x256 batch"])
def test_scales_at_the_ends_of_their_range_cancel(tile, kind):
    """A's scales of 2^-119 under B's of 2^119, and the other way, give the product under scales of 1."""
    B, M, N, _ = DENSE[tile]
    K = 288
    a, sa = exact_operand((B, M, K), kind, 1)
    b, sb = exact_operand((B, N, K), "e2m1", 2)
    want = dense(a, sa, b, sb, f32)
    for by in (-119, 119):
        say("scales far apart", tile, kind, by)
        up, down = (sa.view(u8).int() + by).to(u8).view(E8M0), (sb.view(u8).int() - by).to(u8).view(E8M0)
        assert torch.equal(dense(a, up, b, down, f32), want)


@pytest.mark.parametrize("tile", [t for t in DENSE if t != "t256x256 batch"])
def test_what_lies_behind_the_scales_has_no_effect(tile):
    """Scales that end inside a word, between NaN scales: of the dense call and of the experts'."""
    B, M, N, _ = DENSE[tile]
    M += 1 - M % 2  # odd, for 3 scales to a row
    K = 96
    a, sa = exact_operand((B, M, K), "e4m3", 1)
    b, sb = exact_operand((B, N, K), "e2m1", 2)
    around = []
    for s in (sa, sb):
        whole = empty(s.numel() + 128, fill=0xFF)
        whole[64:64 + s.numel()] = s.view(u8).reshape(-1)
        around.append(whole[64:64 + s.numel()].view(s.shape).view(E8M0))
    say("scales between others", tile)
    assert torch.equal(dense(a, around[0], b, around[1], f32), dense(a, sa, b, sb, f32))
    T = B * M  # the same rows as segments of the batch's weights
    offsets = torch.arange(0, T + 1, M, dtype=torch.int32, device="cuda")
    outs = []
    for x, y in ((sa, sb), around):
        out = empty(T, N, dtype=f32)
        bsq.bsq_moe_matmul_mxfp4(a.view(T, K), x.reshape(T, K // 32), b, y, offsets, out)
        outs.append(out)
    assert torch.equal(*outs) and torch.equal(outs[0].view(B, M, N), dense(a, sa, b, sb, f32))


# ------------------------------------------------------------------ experts --

@pytest.mark.parametrize("align", [1, 32])
@pytest.mark.parametrize("gathers", [False, True])
@pytest.mark.parametrize("code", ["e2m1", "e4m3"])
@pytest.mark.parametrize("counts, F, H", [([30, 0, 70, 1, 44], 160, 96), ([300, 0, 433, 157, 250, 1, 240], 544, 1056)])
def test_the_experts_input_gradient(counts, F, H, code, gathers, align):
    """dX of each row is its dY times its expert's weights: the product of the transposed operand that the quantizer
    writes, contracting the weights' rows; from rows in their order, or from each token's dY."""
    E, k = len(counts), 2
    say("experts' input gradient", counts, F, H, code, gathers, align)
    cap = sum(n + -n % align for n in counts) + 5
    T = cap if not gathers else 61
    offsets, rows = ragged(counts, T, k, align, 3)
    w, dy = randn(E, F, H, seed=1, dtype=bf16) * H ** -0.5, randn(T, F, seed=2)
    (_, _), (wt, wts) = quant(w)  # codes_t [E, H, F / 2]
    if code == "e2m1":
        g, gs = quant(dy, both=False)
    else:
        g, gs = empty(T, F, dtype=E4M3), empty(T, F // 32, dtype=E8M0)
        bsq.bsq_quant_mx(dy, g, gs, 1, bsq.BSQ_E4M3)
    dx = empty(cap, H, dtype=f32)
    bsq.bsq_moe_matmul_mxfp4(g, gs, wt, wts, offsets, dx, rows=rows if gathers else None, k=k if gathers else 1)
    if not gathers:
        rows = None
    args = (offsets, rows, cap, k if gathers else 1)
    want = experts_reference(g, gs, wt, wts, *args)
    # sums of F products and, of 8-bit codes, the 13 bits that they are cut to: by the sums of magnitudes
    size = experts_reference(g.float().abs().to(E4M3) if code != "e2m1" else g & 0x77, gs, wt & 0x77, wts, *args)
    tol = ((F / 8 + F / 32 + 4) * 2.0 ** -23 + (7 * 2.0 ** -13 if code != "e2m1" else 0.0)) * size
    assert bool(((dx.double() - want).abs() <= tol).all())
    # what the codes stand for is the transposed weights, each to half a step (see the linear layer's test)
    v = w.transpose(1, 2).double()
    scale = torch.exp2(wts.view(u8).double() - 127).repeat_interleave(32, -1)
    assert bool(((decode(wt, wts) - v).abs() <= torch.maximum(v.abs() / 4, scale / 4)).all())
    # and the rows' gradient is that of sum(out c) by differences of the forward's sum, which is linear in x
    if not gathers:
        at = offsets[1] - 1  # a row of the first expert
        step = torch.randn(H, device="cuda", dtype=torch.float64)
        fwd = lambda x: float((decode(g, gs)[at] * (decode(wt[0], wts[0]).t() @ x)).sum())  # noqa: E731
        diff = fwd(step) - fwd(-step)
        got = 2 * float((dx[at].double() * step).sum())
        assert abs(diff - got) <= 2 * float((tol[at] * step.abs()).sum()) + 1e-9 * abs(diff)


# ------------------------------------------------------------------- nvfp4 --

@pytest.mark.parametrize("M, N, K", [(1, 64, 256), (48, 64, 256), (130, 272, 640)])
def test_nvfp4_operands_and_their_product_value_by_value(M, N, K):
    """Each code stands for its value to half a step, and the product is that of what the codes stand for."""
    say("nvfp4 value by value", M, N, K)
    ops = []
    for shape, seed in (((1, M, K), 1), ((1, N, K), 2)):
        t = randn(*shape, seed=seed) * 0.01
        f = 6 * 448 / t.abs().max().reshape(1)
        q, s = empty(1, shape[1], K // 2), empty(1, shape[1], K // 16, dtype=E4M3)
        bsq.bsq_quant_fp4(t, q, s, format=bsq.BSQ_NVFP4, factor=f)
        c = torch.stack([q & 15, q >> 4], -1).flatten(-2).long()
        v = TABLE.cuda().double()[c & 7]
        scale = s.double().repeat_interleave(16, -1)
        v = torch.where(c > 7, -v, v) * scale
        y = (t * f).double()
        # half a step is a fifth of the value at most (1 at 5, 0.25 at 1.25), or a quarter of the scale; the scale, a
        # sixth of the largest, is rounded by 2^-4, by which the largest may pass 6
        assert bool(((v - y).abs() <= torch.maximum(y.abs() / 5, scale / 4) * (1 + 2.0 ** -20)).all())
        ops.append((q, s, v[0]))
    (qa, sa, a), (qb, sb, b) = ops
    out = empty(1, M, N, dtype=f32)
    bsq.bsq_scaled_matmul_nvfp4(qa, qb, sa, sb, out, empty(bsq.bsq_nvfp4_workspace_bytes(1, M, N, K)))
    # a code times its scale has 6 bits: exact in the product's operands; K roundings of its float32 sums
    err = (out[0].double() - a @ b.t()).abs()
    assert bool((err <= K * 2.0 ** -23 * (a.abs() @ b.abs().t())).all())
