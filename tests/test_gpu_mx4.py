"""4-bit operands on the GPU: the quantizer against the oracle bit for bit, and
the products with 4-bit weights, dense and ragged, against products in 64 bits.

Where the operands are small whole multiples of powers of two every partial
sum is exact in float32 (see `exact_operands`), and the product must be the
exact one bit for bit, whatever the kernel and the order of its sums."""
import numpy as np
import pytest
import torch

import block_scaled_precision_blockwise_amd as bsq
from gpu_helpers import assert_bytes_equal, host, say, to_dev
from mx4_sizes import DENSE, RAGGED, cap_of
from oracle import fp4

pytestmark = pytest.mark.gpu

E4M3, E5M2, E8M0 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
u8 = torch.uint8


def empty(*shape, dtype=u8, fill=0xA5):
    """Device memory that holds `fill` in every byte."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.view(u8).fill_(fill) if t.numel() else None
    return t


# ------------------------------------------------------------- quantizer --

def values(shape, seed, bf16):
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape) * np.exp2(g.integers(-12, 12, (*shape[:-1], 1)))
    x[..., : min(16, shape[-1])] *= 2.0 ** -30
    flat = x.reshape(-1)
    flat[g.integers(0, flat.size, flat.size // 50 + 1)] = 0.0
    # ties between codes under a power-of-two scale, and magnitudes next to 6 2^E
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -5.0])
    flat[: 10 * (flat.size // 10)].reshape(-1, 10)[:: 7] = ties
    x = x.astype(np.float32)
    if bf16:
        x = torch.from_numpy(x).bfloat16().float().numpy()
    return x


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shape", [(1, 32), (1, 4096), (7, 96), (32, 32), (64, 160), (128, 128), (160, 2080), (3, 96, 64),
                                   (2, 288, 416)])
def test_quant(fmt, bf16, shape):
    x = values(shape, sum(shape) + bf16, bf16)
    factor = np.float32(3.7) if fmt == "nv" and shape[-1] % 64 else None
    say("quant_fp4", fmt, bf16, shape)
    block = 32 if fmt == "mx" else 16
    q = (lambda v: fp4.mxfp4(v)) if fmt == "mx" else (lambda v: fp4.nvfp4(v, 1.0 if factor is None else factor))
    d = to_dev(x).bfloat16() if bf16 else to_dev(x)
    f = None if factor is None else torch.tensor([factor], device="cuda")
    *lead, R, C = shape
    kw = dict(format=bsq.BSQ_MXFP4 if fmt == "mx" else bsq.BSQ_NVFP4, factor=f)
    want, want_t = q(x), q(np.ascontiguousarray(np.swapaxes(x, -1, -2))) if R % block == 0 else None
    rows = lambda: (empty(*lead, R, C // 2), empty(*lead, R, C // block))  # noqa: E731
    cols = lambda: (empty(*lead, C, R // 2), empty(*lead, C, R // block))  # noqa: E731
    a, t = rows(), cols()
    bsq.bsq_quant_fp4(d, *a, **kw)
    for got, w, n in zip(a, want, ("codes", "scales")):
        assert_bytes_equal(host(got), w, n)
    if want_t is None:
        with pytest.raises(ValueError):
            bsq.bsq_quant_fp4(d, None, None, empty(*lead, C, R // 2), empty(*lead, C, R // block), **kw)
        return
    bsq.bsq_quant_fp4(d, codes_t=t[0], scales_t=t[1], **kw)
    for got, w, n in zip(t, want_t, ("codes_t alone", "scales_t alone")):
        assert_bytes_equal(host(got), w, n)
    a, t = rows(), cols()
    bsq.bsq_quant_fp4(d, *a, *t, **kw)
    for got, w, n in zip((*a, *t), (*want, *want_t), ("codes", "scales", "codes_t", "scales_t")):
        assert_bytes_equal(host(got), w, n)


# ---------------------------------------------------------------- operands --

TABLE = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def decode(codes, scales):
    """What codes (packed e2m1 where they are bytes, else fp8) under E8M0 scales of 32 stand for, in 64 bits."""
    if codes.dtype == u8:
        c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
        v = TABLE.to(codes.device).double()[c & 7]
        v = torch.where(c > 7, -v, v)
    else:
        v = codes.double()
    s = scales.view(u8).double()
    return v * torch.where(s == 255, torch.nan, torch.exp2(s - 127)).repeat_interleave(32, -1)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def exact_operand(shape, kind, seed):
    """e2m1: any code; fp8: multiples of 0.5 up to 6; scales 1/2, 1, 2.  A
    product of two is a multiple of 2^-4 of at most 144 = 36 * 4, so that a sum
    of up to 4096 of them takes 24 bits, and the matrix core's groups of 8, cut
    to 13 bits below the largest product, lose nothing."""
    g = gen(seed)
    s = torch.randint(126, 129, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda").to(u8).view(E8M0)
    if kind == "e2m1":
        return torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device="cuda").to(u8), s
    v = torch.randint(-12, 13, shape, generator=g, device="cuda").float() / 2
    return v.to(E4M3 if kind == "e4m3" else E5M2), s


def full_operand(shape, kind, seed):
    """Any finite code, scales over 12 powers of two."""
    g = gen(seed)
    s = torch.randint(120, 133, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda").to(u8).view(E8M0)
    if kind == "e2m1":
        return torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device="cuda").to(u8), s
    dt = E4M3 if kind == "e4m3" else E5M2
    c = torch.randint(0, 256, shape, generator=g, device="cuda").to(u8).view(dt)
    return torch.where(torch.isfinite(c.float()), c.float(), 1.0).to(dt), s


def reference(a, b):
    """a b^T and the bound's two sums: of |a b|, and of the largest product of each 8 neighbours."""
    y, T = a @ b.t(), a.abs() @ b.abs().t()
    a8, b8 = (v.abs().reshape(v.shape[0], -1, 8).amax(-1) for v in (a, b))
    return y, T, a8 @ b8.t()


def hold(out, y, T, G, K, eight, what):
    """float32 sums: each of the K / 8 groups and each chunk's sum adds one
    rounding of at most 2^-23 of a partial sum (T bounds them).  With 8-bit
    codes 7 products of a group lose at most 2^-13 of its largest each.  One
    rounding more for bfloat16 (2^-8)."""
    tol = (K / 8 + K / 32 + 4) * 2.0 ** -23 * T + (7 * 2.0 ** -13 * G if eight else 0.0)
    if out.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs()
    err = (out.double() - y).abs()
    assert bool((err <= tol).all()), (what, float((err - tol).max()), float(err.max()))


KINDS = ["e2m1", "e4m3", "e5m2"]


def dense(a, sa, b, sb, dtype):
    out = empty(a.shape[0], a.shape[1], b.shape[1], dtype=dtype)
    bsq.bsq_scaled_matmul_mxfp4(a, b, sa, sb, out)
    return out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tile", DENSE)
def test_dense_exact_by_each_tile(tile, kind):
    B, M, N, Ks = DENSE[tile]
    for K in Ks:
        say("mxfp4 dense", tile, B, M, N, K, kind)
        a, sa = exact_operand((B, M, K), kind, 1)
        b, sb = exact_operand((B, N, K), "e2m1", 2)
        out, bf = dense(a, sa, b, sb, torch.float32), dense(a, sa, b, sb, torch.bfloat16)
        for i in range(B):
            y = decode(a[i], sa[i]) @ decode(b[i], sb[i]).t()
            assert torch.equal(out[i].double(), y), (K, i, int((out[i].double() != y).sum()))
            assert torch.equal(bf[i], y.float().bfloat16()), (K, i)


# odd rows, columns and batches, one value's block, empty contractions
SMALL = [(1, 1, 16, 32), (1, 3, 272, 96), (2, 16, 64, 160), (3, 5, 32, 64), (1, 33, 144, 256), (2, 100, 208, 416),
         (1, 129, 272, 512), (1, 300, 16, 2880), (3, 70, 96, 1056), (5, 7, 48, 0), (1, 4100, 3600, 0)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B, M, N, K", SMALL)
def test_dense_exact_small(B, M, N, K, kind):
    say("mxfp4 dense", B, M, N, K, kind)
    a, sa = exact_operand((B, M, K), kind, 1)
    b, sb = exact_operand((B, N, K), "e2m1", 2)
    y = torch.bmm(decode(a, sa), decode(b, sb).transpose(1, 2).contiguous())
    assert torch.equal(dense(a, sa, b, sb, torch.float32).double(), y)
    assert torch.equal(dense(a, sa, b, sb, torch.bfloat16), y.float().bfloat16())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B, M, N, K", [(1, 1, 272, 4096), (1, 3, 272, 9312), (1, 16, 4112, 8192), (2, 33, 144, 288), (1, 257, 528, 1312), (1, 400, 1200, 1312),
                                        (1, 1000, 1504, 1056), (1, 1700, 2000, 1056), (1, 4100, 3600, 1056)])
def test_dense_any_codes(B, M, N, K, kind):
    say("mxfp4 dense, any codes", B, M, N, K, kind)
    a, sa = full_operand((B, M, K), kind, 3)
    b, sb = full_operand((B, N, K), "e2m1", 4)
    for dt in (torch.float32, torch.bfloat16):
        out = empty(B, M, N, dtype=dt)
        bsq.bsq_scaled_matmul_mxfp4(a, b, sa, sb, out)
        for i in range(B):
            hold(out[i], *reference(decode(a[i], sa[i]), decode(b[i], sb[i])), K, kind != "e2m1", (B, M, N, K, kind))


# ------------------------------------------------------------------ ragged --

def ragged(counts, T, k, align, seed):
    """offsets [E + 1], rows [cap] of segments with `counts` choices, the rest of each segment and a tail empty."""
    g = np.random.default_rng(seed)
    offsets, rows = [0], []
    for n in counts:
        rows += g.integers(0, T * k, n).tolist() + [-1] * (-n % align)
        offsets.append(len(rows))
    rows += [-1] * 5
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return i32(offsets), i32(rows)


def experts(a, sa, b, sb, offsets, rows, cap, k, dtype):
    out = empty(cap, b.shape[1], dtype=dtype)
    bsq.bsq_moe_matmul_mxfp4(a, sa, b, sb, offsets, out, rows=rows, k=k)
    return out


def experts_reference(a, sa, b, sb, offsets, rows, cap, k):
    """Rows of segments that may lie anywhere in [0, cap), the rest zeros."""
    T = a.shape[0]
    at = torch.arange(cap, device="cuda") if rows is None else torch.where(rows >= 0, rows // k, -1).long()
    at = torch.where(at < T, at, -1)
    want = torch.zeros(cap, b.shape[1], dtype=torch.float64, device="cuda")
    x, ends = decode(a, sa), offsets.tolist()
    for e in range(b.shape[0]):
        r = at[ends[e]:ends[e + 1]]
        if r.numel() and T:
            want[ends[e]:ends[e + 1]] = torch.where((r >= 0)[:, None], x[r.clamp_min(0)], 0.0) @ decode(b[e], sb[e]).t()
    return want


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("tile", RAGGED)
def test_ragged_exact_by_each_tile(tile, own, kind):
    counts, align, N, Ks = RAGGED[tile]
    cap, k = cap_of(counts, align), 2
    T = cap - 3 if own else cap  # own rows past A's are zeros
    offsets, rows = ragged(counts, T, k, align, 7)
    assert rows.numel() == cap
    for K in Ks:
        say("mxfp4 ragged", tile, own, K, kind)
        a, sa = exact_operand((T, K), kind, 5)
        b, sb = exact_operand((len(counts), N, K), "e2m1", 6)
        args = (a, sa, b, sb, offsets, None if own else rows, cap, k)
        want = experts_reference(*args)
        assert torch.equal(experts(*args, torch.float32).double(), want), K
        assert torch.equal(experts(*args, torch.bfloat16), want.float().bfloat16()), K


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts, T, N, K, k, align", [
    ([1], 1, 16, 32, 1, 1), ([0, 1, 0, 2, 1], 3, 80, 96, 2, 1), ([3, 16, 17, 0, 1, 40], 9, 272, 160, 4, 1),
    ([5, 0, 130], 31, 144, 512, 2, 32), ([200, 7, 0, 64], 40, 208, 1056, 3, 128), ([0, 0], 4, 32, 64, 1, 1),
    ([1, 0, 2], 1, 64, 96, 4, 128), ([3, 1], 2, 48, 0, 2, 1), ([2, 2], 0, 48, 64, 1, 1), ([1] * 1024, 700, 32, 64, 3, 1),
    ([7000, 5000, 6000], 5, 1552, 32, 4000, 1), ([7000, 5000, 6000], 2, 1552, 512, 9000, 1),
    ([7000, 5000, 6000], 0, 1552, 288, 2, 1), ([7000, 5000, 6000], 9000, 1552, 0, 2, 1)])
def test_ragged_exact(counts, T, N, K, k, align, kind):
    """Few tokens chosen often, holes, a plan's alignment, no contraction, no tokens, the most experts, big tiles of
    fewer scales than they read at once."""
    say("mxfp4 ragged", len(counts), T, N, K, k, align, kind)
    a, sa = exact_operand((T, K), kind, 5)
    b, sb = exact_operand((len(counts), N, K), "e2m1", 6)
    offsets, rows = ragged(counts, max(T, 1), k, align, 7)
    args = (a, sa, b, sb, offsets, rows, rows.numel(), k)
    want = experts_reference(*args)
    assert torch.equal(experts(*args, torch.float32).double(), want)
    assert torch.equal(experts(*args, torch.bfloat16), want.float().bfloat16())


def test_ragged_own_rows():
    a, sa = exact_operand((50, 288), "e4m3", 8)
    b, sb = exact_operand((3, 48, 288), "e2m1", 9)
    offsets = torch.tensor([0, 20, 20, 41], dtype=torch.int32, device="cuda")
    out = empty(60, 48, dtype=torch.float32)
    bsq.bsq_moe_matmul_mxfp4(a, sa, b, sb, offsets, out)
    x = decode(a, sa)
    want = torch.zeros(60, 48, dtype=torch.float64, device="cuda")
    want[:20] = x[:20] @ decode(b[0], sb[0]).t()
    want[20:41] = x[20:41] @ decode(b[2], sb[2]).t()
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("T, K", [(5, 32), (0, 32), (15, 32), (16, 32), (3, 256), (1, 512)])
def test_ragged_own_rows_past_few_tokens(T, K):
    """Segments of thousands of rows, of which A has the first few."""
    say("mxfp4 ragged", T, K)
    cap, N, ends = 18000, 1552, [2, 7000, 18000]
    a, sa = exact_operand((T, K), "e2m1", 8)
    b, sb = exact_operand((3, N, K), "e2m1", 9)
    out = empty(cap, N, dtype=torch.float32)
    bsq.bsq_moe_matmul_mxfp4(a, sa, b, sb, torch.tensor([0] + ends, dtype=torch.int32, device="cuda"), out)
    want = torch.zeros(cap, N, dtype=torch.float64, device="cuda")
    if T:
        x = decode(a, sa)
        want[:min(T, 2)] = x[:2] @ decode(b[0], sb[0]).t()
        want[2:max(T, 2)] = x[2:] @ decode(b[1], sb[1]).t()
    assert torch.equal(out.double(), want)
