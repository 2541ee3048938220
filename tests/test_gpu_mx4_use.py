"""The calls on 4-bit operands and the norm as programs use them: together, in
graphs, on other streams, beside memory that is not theirs, with infinities and
NaN, with index arrays that hold anything, and their refusals."""
import ctypes

import numpy as np
import pytest
import torch

import block_scaled_precision_blockwise_amd as bsq
from gpu_helpers import assert_bytes_equal, host, say
from mx4_sizes import DENSE, RAGGED, cap_of
from oracle import fp4, norm
from test_gpu_mx4 import (E4M3, E5M2, E8M0, decode, dense, empty, exact_operand, experts, experts_reference, full_operand,
                          gen, hold, ragged, reference, u8)

pytestmark = pytest.mark.gpu
f32, bf16 = torch.float32, torch.bfloat16


def randn(*shape, seed=0, dtype=f32):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(dtype)


def quant(x, both=True, fmt=bsq.BSQ_MXFP4):
    """Operands of x [.., R, C] along its rows and, with `both`, transposed."""
    *lead, R, C = x.shape
    b, kind = (32, E8M0) if fmt == bsq.BSQ_MXFP4 else (16, E4M3)
    rows = empty(*lead, R, C // 2), empty(*lead, R, C // b, dtype=kind)
    cols = (empty(*lead, C, R // 2), empty(*lead, C, R // b, dtype=kind)) if both else (None, None)
    bsq.bsq_quant_fp4(x, *rows, *cols, format=fmt)
    return (rows, cols) if both else rows


# ---------------------------------------------------------------- together --

@pytest.mark.parametrize("code", ["e2m1", "e4m3"])
def test_a_linear_layer_forward_and_backward(code):
    """norm -> operand -> product; backward: both operands of dy, the input's
    and the weight's gradient, the norm's gradient.  Every product is that of
    the operands it was given, the gradient that of the formula in 64 bits."""
    M, K, N = 160, 288, 224
    say("4-bit linear layer", code)
    x, w, dy = randn(M, K, seed=1, dtype=bf16), randn(N, K, seed=2) * K ** -0.5, randn(M, N, seed=3, dtype=bf16)
    gamma, beta = 1 + 0.2 * randn(K, seed=4), 0.1 * randn(K, seed=5)
    (wq, ws), (wt, wts) = quant(w)
    y = empty(M, K, dtype=bf16)
    a = (empty(M, K // 2) if code == "e2m1" else empty(M, K, dtype=E4M3)), empty(M, K // 32, dtype=E8M0)
    mean, rstd = empty(M, dtype=f32), empty(M, dtype=f32)
    bsq.bsq_norm_mx(x, y=y, codes=a[0], scales=a[1], gamma=gamma, beta=beta, mean=mean, rstd=rstd)
    out = empty(1, M, N, dtype=bf16)
    bsq.bsq_scaled_matmul_mxfp4(a[0][None], wq[None], a[1][None], ws[None], out)
    hold(out[0], *reference(decode(*a), decode(wq, ws)), K, code != "e2m1", "forward")

    (g, gs), (gt, gts) = quant(dy)
    dxn, dw = empty(1, M, K, dtype=bf16), empty(1, N, K, dtype=f32)
    bsq.bsq_scaled_matmul_mxfp4(g[None], wt[None], gs[None], wts[None], dxn)  # contracts N
    hold(dxn[0], *reference(decode(g, gs), decode(wt, wts)), N, False, "dX")
    (_, _), (yt, yts) = quant(y)
    bsq.bsq_scaled_matmul_mxfp4(gt[None], yt[None], gts[None], yts[None], dw)  # contracts M
    hold(dw[0], *reference(decode(gt, gts), decode(yt, yts)), M, False, "dW")
    # the transposed operands stand for the same matrices, blocked the other way:
    # each value within half a step (a quarter of 4 or more, else of its block's 2)
    for (q, s), v in (((wt, wts), w.t()), ((gt, gts), dy.t())):
        got, scale = decode(q, s), torch.exp2(s.view(u8).double() - 127).repeat_interleave(32, -1)
        assert bool(((got - v.double()).abs() <= torch.maximum(v.double().abs() / 4, scale / 4)).all())
    dx, dgamma, dbeta = empty(M, K, dtype=bf16), empty(K, dtype=f32), empty(K, dtype=f32)
    bsq.bsq_norm_backward(x, dxn[0], rstd, dx, mean=mean, gamma=gamma, dgamma=dgamma, dbeta=dbeta,
                          workspace=empty(bsq.bsq_norm_backward_workspace_bytes(M, K)))
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    want = norm.backward(n(x), n(dxn[0]), n(gamma))
    for got, v, what in ((dx, want[0], "dx"), (dgamma, want[1], "dgamma"), (dbeta, want[2], "dbeta")):
        # roundings of 2^-24 in sums of 160 and 288 terms, and bfloat16's of dx
        err = np.abs(n(got) - v)
        assert np.all(err <= 2.0 ** -8 * np.abs(v) * (got is dx) + 1e-4 * np.abs(v).max()), what


def test_an_expert_layer_with_4_bit_weights():
    """route -> order -> W1 (tokens gathered by the product) -> gate -> W2 ->
    weighted sum, against the same steps in 64 bits on the operands in between."""
    T, H, F, E, k = 70, 96, 64, 8, 2
    say("4-bit experts")
    x, w1, w2 = randn(T, H, seed=1, dtype=bf16), randn(E, 2 * F, H, seed=2) * H ** -0.5, randn(E, H, F, seed=3) * F ** -0.5
    (q1, s1), (q2, s2) = quant(w1, both=False), quant(w2, both=False)
    ids, weights = empty(T, k, dtype=torch.int32), empty(T, k, dtype=f32)
    bsq.bsq_moe_route(randn(T, E, seed=4), ids, weights)
    cap = bsq.bsq_moe_capacity(T * k, E, 32)
    i32 = lambda *s: empty(*s, dtype=torch.int32)  # noqa: E731
    offsets, counts, rows, pos = i32(E + 1), i32(E), i32(cap), i32(T, k)
    bsq.bsq_moe_plan(ids, offsets, counts, rows, pos, empty(bsq.bsq_moe_plan_workspace_bytes(T * k, E)), align=32)
    xq, xs = quant(x, both=False)
    gu = empty(cap, 2 * F, dtype=bf16)
    bsq.bsq_moe_matmul_mxfp4(xq, xs, q1, s1, offsets, gu, rows=rows, k=k)
    want = experts_reference(xq, xs, q1, s1, offsets, rows, cap, k)
    assert bool(((gu.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all())
    h, hs = empty(cap, F, dtype=E4M3), empty(cap, F // 32, dtype=E8M0)
    bsq.bsq_swiglu_mx(gu, h, hs)
    y = empty(cap, H, dtype=bf16)
    bsq.bsq_moe_matmul_mxfp4(h, hs, q2, s2, offsets, y)
    want = experts_reference(h, hs, q2, s2, offsets, None, cap, 1)
    assert bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * want.abs().max()).all())
    out = empty(T, H, dtype=bf16)
    bsq.bsq_moe_combine(y, pos, out, weights=weights)
    want = (y.double()[pos.long()] * weights.double()[:, :, None]).sum(1)
    assert bool(((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all())


def test_nvfp4_operands_go_through_their_product():
    """The quantizer makes what bsq_scaled_matmul_nvfp4 takes; under both
    tensors' factors the product is that of the values, divided by them."""
    M, N, K = 48, 64, 256
    a, b = randn(1, M, K, seed=1) * 0.01, randn(1, N, K, seed=2, dtype=bf16)
    fa, fb = (6 * 448 / t.float().abs().max().reshape(1) for t in (a, b))
    ops = []
    for t, f in ((a, fa), (b, fb)):
        q, s = empty(1, t.shape[1], K // 2), empty(1, t.shape[1], K // 16, dtype=E4M3)
        bsq.bsq_quant_fp4(t, q, s, format=bsq.BSQ_NVFP4, factor=f)
        ops.append((q, s))
    (qa, sa), (qb, sb) = ops
    out = empty(1, M, N, dtype=f32)
    bsq.bsq_scaled_matmul_nvfp4(qa, qb, sa, sb, out, empty(bsq.bsq_nvfp4_workspace_bytes(1, M, N, K)))
    out = out[0].double() / (fa * fb).double()
    # each value within 1/4 (of 4 to 6 steps: half a step of 2, by 4) plus 2^-4 of its scale
    x, y = a[0].double(), b[0].double()
    rms = (x @ y.t()).pow(2).mean().sqrt()
    assert float((out - x @ y.t()).pow(2).mean().sqrt() / rms) < 0.25


# ------------------------------------------------------------ NaN, infinity --

ONE_OF_EACH = ["few16x16", "few32x32", "t32x64g2", "t64x64g2", "t128x128", "t256x256"]


@pytest.mark.parametrize("kind", ["e2m1", "e4m3"])
@pytest.mark.parametrize("tile", ONE_OF_EACH)
def test_nan_scales_show_in_their_row_and_column_alone(tile, kind):
    """The NaN scale of one row of A (its last block) and of one of B (its
    first): also where the contraction ends inside a step, whose rest is next to
    the scales of the row behind it."""
    B, M, N, _ = DENSE[tile]
    for K in (96, 288, 1056):
        say("NaN scales", tile, kind, K)
        a, sa = exact_operand((B, M, K), kind, 1)
        b, sb = exact_operand((B, N, K), "e2m1", 2)
        clean = dense(a, sa, b, sb, f32)
        r, c = M - 3, N - 2
        sa.view(u8)[0, r, -1] = 255
        sb.view(u8)[0, c, 0] = 255
        out = dense(a, sa, b, sb, f32)
        want = clean.clone()
        want[0, r, :] = want[0, :, c] = float("nan")
        assert torch.equal(torch.isnan(out), torch.isnan(want)), K
        assert torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0)), K


def test_nan_and_infinity_codes_of_8_bits_show_in_their_row_alone():
    for kind, bad in (("e4m3", 0x7F), ("e5m2", 0x7D), ("e5m2", 0x7C)):
        for K in (96, 544):
            a, sa = exact_operand((1, 40, K), kind, 1)
            b, sb = exact_operand((1, 48, K), "e2m1", 2)
            clean = dense(a, sa, b, sb, f32)
            a.view(u8)[0, 39, K - 1] = bad
            a.view(u8)[0, 3, 0] = bad
            out = dense(a, sa, b, sb, f32)
            rows = [i for i in range(40) if i not in (3, 39)]
            assert torch.equal(out[0, rows], clean[0, rows])
            assert not torch.isfinite(out[0, 3]).any() and not torch.isfinite(out[0, 39]).any()


@pytest.mark.parametrize("dt", [f32, bf16])
def test_quantizer_of_infinities_and_nan(dt):
    x = randn(64, 128, seed=1)
    x[0, 5], x[1, 40], x[33, 127], x[40, 0] = float("inf"), float("-inf"), float("nan"), -float("nan")
    x = x.to(dt)
    for fmt, block, nan in ((bsq.BSQ_MXFP4, 32, 255), (bsq.BSQ_NVFP4, 16, 0x7F)):
        clean = torch.where(torch.isfinite(x), x, 0)
        q = (lambda v: fp4.mxfp4(v)) if block == 32 else (lambda v: fp4.nvfp4(v))
        (c, s), (ct, st) = quant(x, fmt=fmt)
        for codes, scales, v in ((c, s, x), (ct, st, x.t().contiguous())):
            w = torch.where(torch.isfinite(v), v, 0).float().cpu().numpy()
            wc, ws = q(w)
            codes, scales, v = host(codes), host(scales.view(u8)), v.float().cpu().numpy()
            for r in range(v.shape[0]):
                for k in range(v.shape[1] // block):
                    part = v[r, block * k:block * (k + 1)]
                    got, sc = codes[r, block // 2 * k:block // 2 * (k + 1)], scales[r, k]
                    if np.isnan(part).any():
                        assert sc == nan
                    elif np.isinf(part).any():
                        one = np.stack([got & 15, got >> 4], -1).reshape(-1)[np.isinf(part)]
                        assert np.all(one == np.where(part[np.isinf(part)] > 0, 7, 15)) and sc != nan
                    else:
                        assert sc == ws[r, k] and np.array_equal(got, wc[r, block // 2 * k:block // 2 * (k + 1)])
        del clean


def test_quantizer_extremes():
    """Zero blocks, subnormals, the largest magnitudes, blocks that round to the next scale."""
    big = np.float32(3.4e38)
    x = np.zeros((32, 64), np.float32)
    x[1, :3] = 1e-45, -1e-40, 1e-38
    x[2, ::7] = big
    x[3, 1] = -big
    x[4, :2] = 6.0, np.nextafter(np.float32(6.0), np.float32(7))
    x[5, :32] = np.nextafter(np.float32(0.75), np.float32(0))
    x[5, 0] = 6
    x[6] = -0.0
    x[7, 32:] = 1e-10
    t = torch.from_numpy(x).cuda()
    for fmt, q in ((bsq.BSQ_MXFP4, fp4.mxfp4), (bsq.BSQ_NVFP4, fp4.nvfp4)):
        (c, s), (ct, st) = quant(t, fmt=fmt)
        for got, want in zip((c, s, ct, st), (*q(x), *q(np.ascontiguousarray(x.T)))):
            assert_bytes_equal(host(got.view(u8)), want, str(fmt))


# ----------------------------------------------------------- index arrays --

@pytest.mark.parametrize("tile", RAGGED)
def test_index_arrays_that_hold_anything(tile):
    """Offsets out of order, negative and past the rows, choices out of range:
    nothing but `out` is written, and rows of plain segments are right."""
    counts, align, N, _ = RAGGED[tile]
    K, k, E, cap = 96, 2, len(counts), cap_of(counts, align)
    a, sa = exact_operand((cap, K), "e4m3", 5)
    b, sb = exact_operand((E, N, K), "e2m1", 6)
    offsets, rows = ragged(counts, cap, k, align, 7)
    good = rows.clone()
    rows[1::5], rows[2::7], rows[0] = 2 ** 31 - 1, -(2 ** 31), 2 * cap  # past the choices
    good[1::5], good[2::7], good[0] = -1, -1, -1
    say("any choices", tile)
    want = experts_reference(a, sa, b, sb, offsets, good, cap, k)
    assert torch.equal(experts(a, sa, b, sb, offsets, rows, cap, k, f32).double(), want)
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bad = torch.randint(-(2 ** 31), 2 ** 31 - 1, (E + 1,), generator=g, device="cuda").to(torch.int32)
        bad[torch.rand(E + 1, generator=g, device="cuda") < 0.5] %= cap + 9
        guard = empty(cap + 2, N, dtype=f32)
        say("any offsets", tile, seed)
        bsq.bsq_moe_matmul_mxfp4(a, sa, b, sb, bad, guard[1:-1], rows=rows, k=k)
        torch.cuda.synchronize()
        assert bool((guard[0].view(torch.int32) == guard[-1].view(torch.int32)).all())
        assert bool((guard[0].view(u8) == 0xA5).all())


# ------------------------------------------------- memory, streams, graphs --

def inside(shape, dtype=u8, before=64, after=64):
    """A tensor of `shape` with bytes in front of it and behind it, and a check that those are as they were."""
    size = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    whole = empty(before + size + after)
    t = whole[before:before + size].view(dtype).view(shape)
    return t, lambda: bool((whole[:before] == 0xA5).all()) and bool((whole[before + size:] == 0xA5).all())


def test_nothing_beside_the_outputs_is_written():
    for R, C in ((1, 32), (33 * 32, 96), (160, 2080), (96, 32)):
        x = randn(R, C, seed=R)
        for fmt, b in ((bsq.BSQ_MXFP4, 32), (bsq.BSQ_NVFP4, 16)):
            for shift in (0, 1):  # scales that start anywhere
                outs = [inside((R, C // 2)), inside((R, C // b), before=64 + shift)]
                if R % b == 0:
                    outs += [inside((C, R // 2)), inside((C, R // b), before=64 + shift)]
                say("quant in memory", R, C, fmt, shift)
                bsq.bsq_quant_fp4(x, *(t for t, _ in outs), format=fmt)
                assert all(ok() for _, ok in outs)
                want = quant(x, both=False, fmt=fmt)
                assert torch.equal(outs[0][0], want[0]) and torch.equal(outs[1][0], want[1].view(u8))
                if R % b == 0:
                    want = quant(x.t().contiguous(), both=False, fmt=fmt)
                    assert torch.equal(outs[2][0], want[0]) and torch.equal(outs[3][0], want[1].view(u8))
    for tile, (B, M, N, _) in DENSE.items():
        a, sa = exact_operand((B, M, 160), "e4m3", 1)
        b, sb = exact_operand((B, N, 160), "e2m1", 2)
        for dt in (f32, bf16):
            out, ok = inside((B, M, N), dt)
            say("product in memory", tile, dt)
            bsq.bsq_scaled_matmul_mxfp4(a, b, sa, sb, out)
            assert ok()
    for R, C in ((1, 1), (5, 95), (7, 1024), (3, 4096), (2, 9000), (2, 16385)):
        x, dy = randn(R, C, seed=1), randn(R, C, seed=2)
        outs = [inside((R, C), f32), inside((R,), f32), inside((R,), f32), inside((R, C), f32), inside((C,), f32), inside((C,), f32)]
        y, mean, rstd, dx, dg, db = (t for t, _ in outs)
        ws, ok = inside((bsq.bsq_norm_backward_workspace_bytes(R, C),))
        say("norm in memory", R, C)
        bsq.bsq_norm_mx(x, y=y, mean=mean, rstd=rstd)
        bsq.bsq_norm_backward(x, dy, rstd, dx, mean=mean, dgamma=dg, dbeta=db, workspace=ws)
        assert ok() and all(o() for _, o in outs)


def layer(M=160, K=288, N=208, seed=0):
    """One pass of every call on buffers of its own: (fill(seed), run(), outputs)."""
    x, w, dy = empty(M, K, dtype=bf16), empty(N, K, dtype=f32), empty(M, K, dtype=bf16)
    gamma = empty(K, dtype=f32)
    s = dict(codes=empty(M, K // 2), scales=empty(M, K // 32, dtype=E8M0), y=empty(M, K, dtype=bf16),
             mean=empty(M, dtype=f32), rstd=empty(M, dtype=f32), wq=empty(N, K // 2), ws=empty(N, K // 32, dtype=E8M0),
             out=empty(1, M, N, dtype=f32), rows=empty(M, N, dtype=bf16), dx=empty(M, K, dtype=bf16),
             dgamma=empty(K, dtype=f32), dbeta=empty(K, dtype=f32))
    offsets = torch.tensor([0, M // 3, M], dtype=torch.int32, device="cuda")
    space = empty(bsq.bsq_norm_backward_workspace_bytes(M, K))

    def fill(seed):
        x.copy_(randn(M, K, seed=seed))
        dy.copy_(randn(M, K, seed=seed + 1))
        w.copy_(randn(N, K, seed=seed + 2))
        gamma.copy_(1 + 0.1 * randn(K, seed=seed + 3))

    def run():
        bsq.bsq_norm_mx(x, y=s["y"], codes=s["codes"], scales=s["scales"], gamma=gamma, mean=s["mean"], rstd=s["rstd"],
                        code_dtype=bsq.BSQ_E2M1)
        bsq.bsq_quant_fp4(w, s["wq"], s["ws"])
        bsq.bsq_scaled_matmul_mxfp4(s["codes"][None], s["wq"][None], s["scales"][None], s["ws"][None], s["out"])
        bsq.bsq_moe_matmul_mxfp4(s["codes"], s["scales"], s["wq"].expand(2, -1, -1).contiguous(),
                                 s["ws"].view(u8).expand(2, -1, -1).contiguous(), offsets, s["rows"])
        bsq.bsq_norm_backward(x, dy, s["rstd"], s["dx"], mean=s["mean"], gamma=gamma, dgamma=s["dgamma"], dbeta=s["dbeta"],
                              workspace=space)
    return fill, run, s


def copies(s):
    return {n: t.clone() for n, t in s.items()}


def same(a, b):
    for n in a:
        assert torch.equal(a[n].view(u8), b[n].view(u8)), n


def test_graph_replays():
    """Captured once, replayed on new inputs, with eager work between."""
    fill, run, s = layer()
    fill(1)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for rep in range(4):
        fill(10 * rep)
        g.replay()
        torch.cuda.synchronize()
        got = copies(s)
        torch.randn(1 << 20, device="cuda").sum().item()
        for t in s.values():
            t.view(u8).fill_(0x5A)
        run()
        torch.cuda.synchronize()
        same(got, s)


def test_streams_side_by_side():
    """Two passes at once on two streams give what each gives alone; a stream
    argument is obeyed; every pass gives the same bytes."""
    one, two = layer(), layer(96, 544, 1040)
    want = []
    for fill, run, s in (one, two):
        fill(3)
        run()
        torch.cuda.synchronize()
        want.append(copies(s))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(5):
        for t in (*one[2].values(), *two[2].values()):
            t.view(u8).fill_(0x5A)
        torch.cuda.synchronize()
        for st, (_, run, _) in zip(streams, (one, two)):
            with torch.cuda.stream(st):
                run()
        torch.cuda.synchronize()
        same(want[0], one[2])
        same(want[1], two[2])
    x, y = randn(4, 64), empty(4, 64, dtype=f32)
    with torch.cuda.stream(streams[0]):
        bsq.bsq_norm_mx(x, y=y, stream=streams[1])
    streams[1].synchronize()
    assert torch.isfinite(y).all()


def test_the_product_records_the_events_asked_for():
    hip = ctypes.CDLL("libamdhip64.so.7")
    ev = [ctypes.c_void_p(), ctypes.c_void_p()]
    hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p, ctypes.c_void_p]
    for e in ev:
        assert hip.hipEventCreateWithFlags(ctypes.byref(e), ctypes.c_uint(0)) == 0
    try:
        for tile in ("few16x16", "t64x64g2", "t256x256"):
            B, M, N, _ = DENSE[tile]
            a, sa = exact_operand((B, M, 128), "e2m1", 1)
            b, sb = exact_operand((B, N, 128), "e2m1", 2)
            y0 = dense(a, sa, b, sb, bf16)
            bsq.bsq_time_next_gemm(ev[0].value, ev[1].value)
            y1 = dense(a, sa, b, sb, bf16)
            torch.cuda.synchronize()
            ms = ctypes.c_float()
            assert hip.hipEventElapsedTime(ctypes.byref(ms), ev[0], ev[1]) == 0 and 0.0 < ms.value < 100.0
            assert torch.equal(y0, y1)
    finally:
        bsq.bsq_time_next_gemm(None, None)
        for e in ev:
            hip.hipEventDestroy(e)


# ---------------------------------------------------------------- refusals --

def test_binding_refusals():
    x = randn(32, 64)
    c, s = empty(32, 32), empty(32, 2)
    bad = [
        (ValueError, lambda: bsq.bsq_quant_fp4(x.t(), c, s)),                      # strides
        (ValueError, lambda: bsq.bsq_quant_fp4(x[:, ::2], c, s)),
        (ValueError, lambda: bsq.bsq_quant_fp4(x, c, None)),
        (ValueError, lambda: bsq.bsq_quant_fp4(x, empty(32, 64), s)),
        (ValueError, lambda: bsq.bsq_quant_fp4(x, c, empty(32, 4))),
        (ValueError, lambda: bsq.bsq_quant_fp4(x, c, s, format=7)),
        (ValueError, lambda: bsq.bsq_quant_fp4(x[0], c, s)),
        (ValueError, lambda: bsq.bsq_quant_fp4(randn(31, 64), codes_t=empty(64, 15), scales_t=empty(64, 0))),
        (NotImplementedError, lambda: bsq.bsq_quant_fp4(x, c, s, factor=randn(1))),
        (TypeError, lambda: bsq.bsq_quant_fp4(x.half(), c, s)),
        (TypeError, lambda: bsq.bsq_quant_fp4(x, empty(32, 32, dtype=E4M3), s)),
        (TypeError, lambda: bsq.bsq_quant_fp4(x, c, empty(32, 2, dtype=f32))),
    ]
    a, sa = exact_operand((1, 4, 64), "e2m1", 1)
    b, sb = exact_operand((1, 16, 64), "e2m1", 2)
    e, se = exact_operand((1, 4, 64), "e4m3", 3)
    out = empty(1, 4, 16, dtype=f32)
    mm = bsq.bsq_scaled_matmul_mxfp4
    bad += [
        (ValueError, lambda: mm(a, b, sa[:, :, :1].contiguous(), sb, out)),
        (ValueError, lambda: mm(a, b, sa, sb[:, :8].contiguous(), out)),
        (ValueError, lambda: mm(a, b, sa, sb, empty(1, 4, 17, dtype=f32))),
        (ValueError, lambda: mm(a.expand(2, 4, 32).contiguous(), b, sa, sb, out)),
        (ValueError, lambda: mm(a[0], b, sa, sb, out)),
        (ValueError, lambda: mm(e[:, :, :32].contiguous(), b, se, sb, out)),      # half the contraction
        (TypeError, lambda: mm(e, b, se, sb, out, lhs_dtype=bsq.BSQ_E5M2)),       # the tensor says e4m3
        (TypeError, lambda: mm(a, e, sa, se, out)),                               # 8-bit weights
        (TypeError, lambda: mm(a, b, sa, sb, out.half())),
        (ValueError, lambda: mm(a, b, empty(9)[1:].view(1, 4, 2), sb, out)),      # scales off a word
        (NotImplementedError, lambda: mm(a, b[:, :8].contiguous(), sa, sb[:, :8].contiguous(), empty(1, 4, 8, dtype=f32))),
    ]
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    moe = bsq.bsq_moe_matmul_mxfp4
    bad += [
        (ValueError, lambda: moe(a[0], sa[0], b, sb, off[:1], out[0])),
        (TypeError, lambda: moe(a[0], sa[0], b, sb, off.long(), out[0])),
        (ValueError, lambda: moe(a[0], sa[0], b, sb, off, out[0], rows=off)),
        (ValueError, lambda: moe(a[0], sa[0], b, sb, off, out[0], k=0)),
        (ValueError, lambda: moe(a[0], sa[0], b[0], sb, off, out[0])),
    ]
    y, v = empty(32, 64, dtype=f32), randn(64)
    bad += [
        (ValueError, lambda: bsq.bsq_norm_mx(x, y=empty(32, 65, dtype=f32))),
        (TypeError, lambda: bsq.bsq_norm_mx(x, y=y.to(bf16))),
        (ValueError, lambda: bsq.bsq_norm_mx(x, y=y, gamma=v[:63])),
        (TypeError, lambda: bsq.bsq_norm_mx(x, y=y, gamma=v.to(bf16))),
        (ValueError, lambda: bsq.bsq_norm_mx(x, codes=c)),
        (ValueError, lambda: bsq.bsq_norm_mx(x, codes=empty(32, 64), scales=s)),  # bytes are 4-bit codes
        (ValueError, lambda: bsq.bsq_norm_mx(x, y=y, mean=v)),
        (NotImplementedError, lambda: bsq.bsq_norm_mx(x, y=y, eps=-1.0)),
        (ValueError, lambda: bsq.bsq_norm_mx(x, y=y, kind=5)),
        (ValueError, lambda: bsq.bsq_norm_backward(x, x, v[:32].contiguous(), y)),  # layer norm without a mean
        (ValueError, lambda: bsq.bsq_norm_backward(x, x, v[:32].contiguous(), y, mean=v[:32].contiguous(), dgamma=empty(64, dtype=f32))),
        (ValueError, lambda: bsq.bsq_norm_backward(x, x[:31], v[:32].contiguous(), y, mean=v[:32].contiguous())),
    ]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            print("not refused:", i)
    # bytes with the format said are 8-bit codes
    codes8, sc = empty(32, 64), empty(32, 2)
    bsq.bsq_norm_mx(x, codes=codes8, scales=sc, code_dtype=bsq.BSQ_E4M3)
    as_e4, s2 = empty(32, 64, dtype=E4M3), empty(32, 2, dtype=E8M0)
    bsq.bsq_norm_mx(x, codes=as_e4, scales=s2)
    assert torch.equal(codes8, as_e4.view(u8)) and torch.equal(sc, s2.view(u8))
    out8 = empty(1, 4, 16, dtype=f32)
    mm(e.view(u8), b, se, sb, out8, lhs_dtype=bsq.BSQ_E4M3)
    mm(e, b, se, sb, out)
    assert torch.equal(out, out8)
