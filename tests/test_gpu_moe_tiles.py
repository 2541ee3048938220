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


# ------------------------------------------------ every tile, type and length --

def _wide(codes, scales, fp8):
    """float64 values of codes with a scale to each 32 along the last axis."""
    torch = _torch()
    v = codes.view(fp8).double().view(*scales.shape, 32)
    return (v * torch.exp2(scales.double() - 127.0)[..., None]).view(codes.shape)


def _close(got, a, b, bf16, what):
    """got [m, n] against a [m, k] b [n, k]^T in 64 bits: 1e-4 of the sum of
    |products|, what the matrix core cuts off a group of 8, a rounding to bfloat16."""
    torch = _torch()

    def groups(v):
        return v.abs().view(*v.shape[:-1], v.shape[-1] // 8, 8).amax(-1)

    want = a @ b.t()
    bound = 1e-4 * (a.abs() @ b.abs().t()) + 2.0 ** -9 * (groups(a) @ groups(b).t()) + 1e-37
    if bf16:
        bound += 2.0 ** -8 * want.abs()
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    bad = (off > bound).nonzero()
    assert len(bad) == 0, f"{what}: {len(bad)} of {got.numel()} outside; first {bad[0].tolist()}"


def _random_codes(g, shape, fp8):
    """Codes of normal values of unlike size, a block exponent to each 32."""
    torch = _torch()
    top = 448.0 if fp8 == torch.float8_e4m3fn else 57344.0
    c = (torch.randn(shape, generator=g, device="cuda") * (top / 6)).clamp(-top, top).to(fp8).view(torch.uint8)
    e = torch.randint(112, 122, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda", dtype=torch.int32)
    return c, e.to(torch.uint8)


# lengths, N, by the tile that they take with any K of these tests
PRODUCT_TILES = {
    "t32x64": ([3, 0, 33, 1], 144), "t64x64": ([300, 0, 500, 3], 784), "t64x128s3": ([300, 0, 500, 3], 1296),
    "t64x128": ([300, 0, 500, 3], 2576), "t256x256": ([700, 0, 1301], 9232)}
TYPES = [(False, False), (False, True), (True, False), (True, True)]  # A in e5m2, output in bfloat16


@pytest.mark.parametrize("steps", range(1, 10))
@pytest.mark.parametrize("tile", PRODUCT_TILES)
def test_matmul_of_each_tile_type_and_length(tile, steps):
    torch = _torch()
    lengths, N = PRODUCT_TILES[tile]
    K, E, k = 128 * steps, len(lengths), 2
    cap = sum(lengths) + 5
    T = cap  # more choices than rows: all rows may hold one
    g = torch.Generator(device="cuda").manual_seed(steps)
    off = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    rows = torch.randint(-T // 4, T * k, (cap,), generator=g, device="cuda").clamp(min=-1).to(torch.int32)
    b, sb = _random_codes(g, (E, N, K), torch.float8_e4m3fn)
    bv = _wide(b, sb, torch.float8_e4m3fn)
    for e5m2, bf16 in TYPES:
        say("matmul of tile", tile, K, e5m2, bf16)
        fp8 = torch.float8_e5m2 if e5m2 else torch.float8_e4m3fn
        a, sa = _random_codes(g, (T, K), fp8)
        av = _wide(a, sa, fp8)
        outs = [filled((cap, N), torch.bfloat16 if bf16 else torch.float32, float("nan")) for _ in range(2)]
        for out in outs:
            bsq.bsq_moe_matmul(a, sa, b, sb, off, out, rows=rows, k=k,
                               a_dtype=bsq.BSQ_E5M2 if e5m2 else bsq.BSQ_E4M3)
        src = torch.where((rows >= 0)[:, None], av[(rows.clamp(min=0) // k).long()], 0.0)
        at = 0
        for e, n in enumerate(lengths):
            _close(outs[0][at:at + n], src[at:at + n], bv[e], bf16, f"expert {e}")
            at += n
        assert torch.all(outs[0][at:] == 0)
        assert torch.equal(outs[0].view(torch.uint8), outs[1].view(torch.uint8)), "two runs differ"


# blocks of 128 rows of the experts' segments, blocks of cap, N, K
WGRAD_TILES = {
    "t64x64": ([9, 7, 0, 1, 3], 21, 400, 272), "t64x128s3": ([5, 0, 6, 8, 2, 4, 1, 9], 36, 400, 400),
    "t128x128s3": ([5, 0, 6, 8, 2, 4, 1, 9], 35, 656, 528), "t128x128": ([5, 0, 6, 8, 2, 4, 1, 9], 35, 784, 784),
    "t256x256": ([9, 7, 6, 8, 0, 4, 1, 3], 40, 1296, 2032), "t256x256 dealt": ([9, 5, 4, 3, 8], 40, 2032, 2000),
    "t256x256_stream": ([9, 7, 20, 0, 2], 64, 2032, 2000), "t256x256_stream one": ([1, 3, 6, 8], 56, 2048, 1936)}


@pytest.mark.parametrize("e5m2,bf16", TYPES)
@pytest.mark.parametrize("tile", WGRAD_TILES)
def test_wgrad_of_each_tile_type_and_length(tile, e5m2, bf16):
    torch = _torch()
    blocks, all_blocks, N, K = WGRAD_TILES[tile]
    E, cap = len(blocks), 128 * all_blocks
    say("wgrad of tile", tile, E, cap, N, K, e5m2, bf16)
    g = torch.Generator(device="cuda").manual_seed(N)
    fp8 = torch.float8_e5m2 if e5m2 else torch.float8_e4m3fn
    dy, sd = _random_codes(g, (N, cap), fp8)
    x, sx = _random_codes(g, (K, cap), torch.float8_e4m3fn)
    off = (torch.tensor([0] + blocks, device="cuda").cumsum(0) * 128).to(torch.int32)
    outs = [filled((E, N, K), torch.bfloat16 if bf16 else torch.float32, float("nan")) for _ in range(2)]
    for out in outs:
        bsq.bsq_moe_wgrad(dy, sd, x, sx, off, out, dyt_dtype=bsq.BSQ_E5M2 if e5m2 else bsq.BSQ_E4M3)
    dv, xv = _wide(dy, sd, fp8), _wide(x, sx, torch.float8_e4m3fn)
    at = 0
    for e, n in enumerate(blocks):
        if n:
            _close(outs[0][e], dv[:, at:at + 128 * n].contiguous(), xv[:, at:at + 128 * n].contiguous(), bf16, f"expert {e}")
        else:
            assert torch.all(outs[0][e] == 0)
        at += 128 * n
    assert torch.equal(outs[0].view(torch.uint8), outs[1].view(torch.uint8)), "two runs differ"


@pytest.mark.parametrize("bf16", [False, True])
def test_big_tiles_without_tokens_or_contraction_write_zeros(bf16):
    torch = _torch()
    E, N = 3, 9232
    off = torch.tensor([0, 700, 700, 2001], dtype=torch.int32, device="cuda")
    out = filled((2006, N), torch.bfloat16 if bf16 else torch.float32, float("nan"))
    u8 = lambda *s: filled(s, torch.uint8, 0x7F)  # noqa: E731
    for T, K in ((0, 128), (2006, 0)):
        say("big tiles empty", T, K, bf16)
        out.fill_(float("nan"))
        bsq.bsq_moe_matmul(u8(T, K), u8(T, K // 32), u8(E, N, K), u8(E, N, K // 32), off, out)
        assert torch.all(out == 0)
