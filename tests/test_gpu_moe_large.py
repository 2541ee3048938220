"""Calls on so many tokens, rows or tiles that one launch cannot
hold their threads: every block of the input repeats the first, and so has
every block of the output to."""
import pytest

import block_scaled_precision_blockwise_amd as bsq

from gpu_helpers import say

pytestmark = pytest.mark.gpu

BLOCK = 4096  # tokens


def _torch():
    import torch
    return torch


def _repeated(block, n):
    """`block` n times along its first axis."""
    return block.unsqueeze(0).expand(n, *block.shape).reshape(n * block.shape[0], *block.shape[1:])


def _repeats(t, rows, what):
    """Every `rows` rows of t are its first (compared in pieces of 2^30 bytes)."""
    torch = _torch()
    first = t[:rows].contiguous().view(torch.uint8).reshape(1, -1)
    whole = t.view(torch.uint8).reshape(-1, first.shape[1])
    step = max(1, (1 << 30) // first.shape[1])
    for i in range(0, whole.shape[0], step):
        assert torch.all(whole[i:i + step] == first), f"{what}: a block from {i} on differs"


@pytest.mark.parametrize("blocks,E,k", [(65536 + 1, 2, 1), (16384 + 1, 260, 8), (16384 + 1, 24, 4)])
def test_route_and_its_gradient_of_very_many_tokens(blocks, E, k):
    torch = _torch()
    T = blocks * BLOCK
    say("route large", T, E, k)
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = _repeated(torch.randn(BLOCK, E, generator=g, device="cuda").bfloat16(), blocks)
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    bsq.bsq_moe_route(logits, ids, w)
    want = logits[:BLOCK].float().sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids[:BLOCK].long(), want)
    _repeats(ids, BLOCK, "ids")
    _repeats(w, BLOCK, "weights")
    dw = _repeated(torch.randn(BLOCK, k, generator=g, device="cuda"), blocks)
    del w
    dl = torch.full((T, E), float("nan"), dtype=torch.bfloat16, device="cuda")
    say("route gradient large", T, E, k)
    bsq.bsq_moe_route_backward(logits, ids, dw, dl)
    assert torch.isfinite(dl[:BLOCK].float()).all()
    _repeats(dl, BLOCK, "dlogits")


def test_combine_gradient_of_very_many_tokens():
    torch = _torch()
    blocks, H = 16384 + 1, 8
    T = blocks * BLOCK
    say("combine gradient large", T, H)
    g = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randn(BLOCK, H, generator=g, device="cuda").bfloat16()
    block = torch.randn(BLOCK, H, generator=g, device="cuda").bfloat16()
    pos = _repeated(torch.arange(BLOCK, dtype=torch.int32, device="cuda").view(-1, 1), blocks)
    dw = torch.full((T, 1), float("nan"), device="cuda")
    bsq.bsq_moe_combine_backward(y, pos, _repeated(block, blocks), dw)
    assert torch.allclose(dw[:BLOCK, 0].double(), (y.double() * block.double()).sum(1), rtol=0, atol=8 * 2.0 ** -24 * 40)
    _repeats(dw, BLOCK, "dweights")


def test_gate_of_very_many_rows():
    torch = _torch()
    F = 32
    blocks = (1 << 33) // (F * BLOCK) + 1
    say("gate large", blocks * BLOCK, F)
    g = torch.Generator(device="cuda").manual_seed(2)
    gu = _repeated(torch.randn(BLOCK, 2 * F, generator=g, device="cuda").bfloat16(), blocks)
    R = gu.shape[0]
    u8 = lambda *s: torch.full(s, 0x55, dtype=torch.uint8, device="cuda")  # noqa: E731
    h, hs, kept, ks = u8(R, F), u8(R, 1), u8(R, 2 * F), u8(R, 2)
    bsq.bsq_swiglu_mx(gu, h, hs, kept=kept, kept_scales=ks)
    h1, hs1 = u8(BLOCK, F), u8(BLOCK, 1)
    bsq.bsq_swiglu_mx(gu[:BLOCK].contiguous(), h1, hs1)
    assert torch.equal(h[:BLOCK], h1) and torch.equal(hs[:BLOCK], hs1)
    for t, n in ((h, "h"), (hs, "h scales"), (kept, "kept"), (ks, "kept scales")):
        _repeats(t, BLOCK, n)


def test_gather_of_very_many_tiles():
    torch = _torch()
    H, T = 8192, 128
    cap = (1 << 36) // H + 1024
    say("gather large", cap, H)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    rows = torch.arange(cap, dtype=torch.int32, device="cuda") % T
    codes = torch.full((cap, H), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((cap, H // 32), 0x55, dtype=torch.uint8, device="cuda")
    bsq.bsq_moe_gather_mx(x, rows, 1, codes, scales)
    want = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
    bsq.bsq_quant_mx(x, *want)
    assert torch.equal(codes[:T], want[0]) and torch.equal(scales[:T], want[1])
    _repeats(codes, T, "codes")
    _repeats(scales, T, "scales")


def test_product_of_very_many_tiles():
    """Room for far more rows than the tokens say: small tiles, and more of
    them than one launch has workgroups."""
    torch = _torch()
    T, E, N, K = 64, 4, 8192, 128
    cap = (1 << 20) + 4096
    say("product large", cap, N)
    g = torch.Generator(device="cuda").manual_seed(4)

    def codes(n, m):
        c, s = torch.empty(n, m, dtype=torch.uint8, device="cuda"), torch.empty(n, m // 32, dtype=torch.uint8, device="cuda")
        bsq.bsq_quant_mx(torch.randn(n, m, generator=g, device="cuda"), c, s)
        return c, s

    a, sa = codes(T, K)
    b, sb = codes(E * N, K)
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * (cap // E)
    rows = torch.arange(cap, dtype=torch.int32, device="cuda") % T
    out = torch.full((cap, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    bsq.bsq_moe_matmul(a, sa, b.view(E, N, K), sb.view(E, N, K // 32), off, out, rows=rows, k=1)
    few = torch.full((E * T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    bsq.bsq_moe_matmul(a, sa, b.view(E, N, K), sb.view(E, N, K // 32), torch.arange(E + 1, dtype=torch.int32, device="cuda") * T,
                       few, rows=rows[:E * T].contiguous(), k=1)
    assert torch.isfinite(few.float()).all()
    for e in range(E):
        seg = out[e * (cap // E):(e + 1) * (cap // E)]
        assert torch.equal(seg[:T], few[e * T:(e + 1) * T])
        _repeats(seg, T, f"expert {e}")


@pytest.mark.parametrize("D", [4, 3])
def test_int8_codes_of_very_many_rows(D):
    torch = _torch()
    R = (1 << 24) + BLOCK
    say("int8 rows large", R, D)
    x = _repeated(torch.randn(BLOCK, D, device="cuda"), R // BLOCK)
    q, s = torch.full((R, D), 99, dtype=torch.int8, device="cuda"), torch.full((R,), float("nan"), device="cuda")
    bsq.bsq_int8_quant_rows(x, q, s)
    assert torch.allclose(q[:BLOCK].float() * s[:BLOCK, None], x[:BLOCK], rtol=0, atol=float(s[:BLOCK].max()) * 0.501)
    _repeats(q, BLOCK, "codes")
    _repeats(s, BLOCK, "scales")
