"""Refusals of the expert-layer calls, on the host and without a GPU: every
rule of include/bsq.h that a caller can break, through the C ABI with fake
addresses that are never dereferenced; and the binding's own checks."""
import pytest
import torch

import block_scaled_precision_blockwise_amd as bsq

OK, NULL, SHAPE, DTYPE, UNSUP, ALIGN, DEVICE, HIP = range(8)
P, P4 = 0x1000, 0x1004
F32, BF16, E4, E5 = bsq.BSQ_F32, bsq.BSQ_BF16, bsq.BSQ_E4M3, bsq.BSQ_E5M2
BIG = 1 << 62


@pytest.fixture(scope="module")
def L():
    if not bsq.is_built():
        import __graft_entry__
        __graft_entry__.build()
    return bsq.lib()


def _call(f, base, **change):
    args = dict(base, **change)
    return f(*args.values())


def _table(L, f, base, rows):
    """Each row: the changed arguments and the status they give."""
    for change, want in rows:
        got = _call(f, base, **change)
        assert got == want, (change, got, L.bsq_last_error())
        if want not in (OK,):
            assert L.bsq_last_error()


ROUTE = dict(T=4, E=64, k=4, groups=1, top_groups=1, group_top=1, logits=P, dt=F32, bias=P, score=0, renorm=1,
             scale=1.0, ids=P, weights=P, scores=P, stream=None)


def test_route(L):
    _table(L, L.bsq_moe_route, ROUTE, [
        ({}, DEVICE), (dict(bias=None, scores=None), DEVICE), (dict(T=0, logits=None), OK),
        (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE),
        (dict(groups=5), SHAPE), (dict(groups=0), SHAPE), (dict(groups=8, top_groups=9), SHAPE),
        (dict(groups=8, top_groups=0), SHAPE), (dict(groups=32, top_groups=1, k=3), SHAPE),
        (dict(groups=64, group_top=2, top_groups=64), SHAPE), (dict(group_top=0), SHAPE),
        (dict(groups=8, top_groups=4, group_top=2), DEVICE), (dict(group_top=3), UNSUP),
        (dict(E=1025), UNSUP), (dict(E=1024, k=64), DEVICE), (dict(E=1024, k=65), UNSUP),
        (dict(E=128, groups=128, top_groups=128), UNSUP), (dict(T=1 << 31), UNSUP),
        (dict(dt=42), DTYPE), (dict(score=2), DTYPE), (dict(score=-1), DTYPE), (dict(dt=bsq.BSQ_I8), UNSUP),
        (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL),
        (dict(logits=P4), ALIGN), (dict(bias=P4), ALIGN), (dict(scores=P4), ALIGN), (dict(ids=P4), ALIGN)])


def test_route_backward(L):
    base = dict(T=4, E=64, k=4, logits=P, dt=BF16, score=1, renorm=1, scale=1.0, ids=P, dw=P, ds=P, dl=P, stream=None)
    _table(L, L.bsq_moe_route_backward, base, [
        ({}, DEVICE), (dict(ds=None), DEVICE), (dict(T=0, logits=None), OK), (dict(T=-1), SHAPE),
        (dict(k=65), SHAPE), (dict(k=0), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), UNSUP), (dict(T=1 << 31), UNSUP),
        (dict(E=128, k=65), UNSUP), (dict(dt=9), DTYPE), (dict(score=7), DTYPE), (dict(dt=E4), UNSUP),
        (dict(dw=None), NULL), (dict(dl=None), NULL), (dict(ids=None), NULL), (dict(ds=P4), ALIGN),
        (dict(dl=P4), ALIGN)])


def test_capacity_and_workspace(L):
    assert bsq.bsq_moe_capacity(100, 8, 1) == 100
    assert bsq.bsq_moe_capacity(100, 8, 128) == 1152          # 100 + 8 * 127 = 1116, up to 128s
    assert bsq.bsq_moe_capacity(3, 8, 128) == 384             # no more segments than choices
    assert bsq.bsq_moe_capacity(0, 8, 128) == 0
    assert bsq.bsq_moe_capacity(-1, 8, 1) == 0 and bsq.bsq_moe_capacity(1, 0, 1) == 0
    assert bsq.bsq_moe_capacity(BIG, BIG, BIG) == 2 ** 63 - 1
    assert bsq.bsq_moe_plan_workspace_bytes(0, 8) >= 16 and bsq.bsq_moe_plan_workspace_bytes(-1, 8) == 0
    assert bsq.bsq_moe_plan_workspace_bytes(1 << 40, 8) == 2 ** 64 - 1
    for n in (1, 1024, 1025, 65536, 10 ** 7):
        assert bsq.bsq_moe_plan_workspace_bytes(n, 256) <= max(16, 4 * 256 * (min(256, -(-n // 1024)) + 1))


def test_plan(L):
    base = dict(n=100, E=8, align=128, cap=1116, ids=P, offsets=P, counts=P, rows=P, pos=P, ws=P, wb=1 << 20,
                stream=None)
    _table(L, L.bsq_moe_plan, base, [
        ({}, DEVICE), (dict(cap=1115), SHAPE), (dict(n=-1), SHAPE), (dict(E=0), SHAPE), (dict(align=0), SHAPE),
        (dict(cap=-1), SHAPE), (dict(wb=15), SHAPE), (dict(E=1025), UNSUP), (dict(n=1 << 31), UNSUP),
        (dict(cap=1 << 31), UNSUP), (dict(align=1 << 40), UNSUP), (dict(n=0, cap=0, ids=None, pos=None, rows=None, ws=None), DEVICE),
        (dict(ids=None), NULL), (dict(offsets=None), NULL), (dict(counts=None), NULL), (dict(rows=None), NULL),
        (dict(pos=None), NULL), (dict(ws=None), NULL), (dict(rows=P4), ALIGN)])


def test_gather(L):
    base = dict(T=10, H=64, cap=128, k=2, x=P, dt=BF16, rows=P, w=P, cd=E4, codes=P, scales=P, ct=P, st=P, stream=None)
    _table(L, L.bsq_moe_gather_mx, base, [
        ({}, DEVICE), (dict(w=None), DEVICE), (dict(ct=None, st=None, cap=127), DEVICE),
        (dict(codes=None, scales=None), DEVICE), (dict(codes=None, scales=None, ct=None, st=None), OK),
        (dict(cap=0), OK), (dict(H=0), OK), (dict(T=0, x=None), DEVICE), (dict(T=-1), SHAPE), (dict(k=0), SHAPE),
        (dict(H=48), SHAPE), (dict(cap=127), SHAPE), (dict(cap=1 << 31), UNSUP), (dict(T=BIG), UNSUP),
        (dict(dt=42), DTYPE), (dict(cd=42), DTYPE), (dict(dt=E4), UNSUP), (dict(cd=F32), UNSUP),
        (dict(codes=None), NULL), (dict(st=None), NULL), (dict(x=None), NULL), (dict(rows=None), NULL),
        (dict(codes=P4), ALIGN), (dict(w=P4), ALIGN), (dict(x=P4), ALIGN)])


def test_combine(L):
    base = dict(T=10, H=64, cap=128, k=2, y=P, dt=BF16, pos=P, w=P, out=P, stream=None)
    _table(L, L.bsq_moe_combine, base, [
        ({}, DEVICE), (dict(w=None), DEVICE), (dict(cap=0, y=None), DEVICE), (dict(T=0), OK), (dict(H=0), OK),
        (dict(T=-1), SHAPE), (dict(H=60), SHAPE), (dict(k=0), SHAPE), (dict(dt=42), DTYPE), (dict(dt=E5), UNSUP),
        (dict(T=1 << 31), UNSUP), (dict(cap=1 << 31), UNSUP), (dict(H=1 << 60), UNSUP),
        (dict(y=None), NULL), (dict(pos=None), NULL), (dict(out=None), NULL), (dict(w=P4), ALIGN), (dict(out=P4), ALIGN)])
    base = dict(T=10, H=64, cap=128, k=2, y=P, dt=F32, pos=P, dout=P, dw=P, stream=None)
    _table(L, L.bsq_moe_combine_backward, base, [
        ({}, DEVICE), (dict(T=0), OK), (dict(H=0, y=None, dout=None), DEVICE), (dict(H=60), SHAPE), (dict(k=0), SHAPE),
        (dict(dt=42), DTYPE), (dict(dt=E5), UNSUP), (dict(dw=None), NULL), (dict(dout=None), NULL), (dict(dout=P4), ALIGN)])


def test_matmul(L):
    base = dict(T=10, cap=64, E=4, N=128, K=256, k=2, a=P, ad=E5, sa=P, b=P, bd=E4, sb=P, offsets=P, rows=P, out=P,
                od=BF16, stream=None)
    _table(L, L.bsq_moe_matmul, base, [
        ({}, DEVICE), (dict(rows=None), DEVICE), (dict(K=0, a=None, b=None, sa=None, sb=None), DEVICE),
        (dict(T=0, a=None, b=None, sa=None, sb=None), DEVICE), (dict(cap=0), OK), (dict(N=0), OK),
        (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(k=0), SHAPE), (dict(cap=-1), SHAPE),
        (dict(K=64), UNSUP), (dict(N=24), UNSUP), (dict(E=1025), UNSUP), (dict(bd=E5), UNSUP), (dict(ad=F32), UNSUP),
        (dict(od=E4), UNSUP), (dict(od=42), DTYPE), (dict(ad=42), DTYPE), (dict(cap=1 << 31), UNSUP),
        (dict(K=1 << 25), UNSUP), (dict(T=(1 << 31) - 1, K=1 << 20), UNSUP), (dict(N=1 << 30, K=1 << 20), UNSUP),
        (dict(cap=(1 << 31) - 1, N=1 << 20), UNSUP),
        (dict(out=None), NULL), (dict(offsets=None), NULL), (dict(a=None), NULL), (dict(b=None), NULL),
        (dict(sa=None), NULL), (dict(sb=None), NULL), (dict(sb=P + 2), ALIGN), (dict(a=P4), ALIGN), (dict(rows=P4), ALIGN)])


def test_wgrad(L):
    base = dict(cap=256, E=4, N=128, K=256, dy=P, dd=E5, sd=P, x=P, xd=E4, sx=P, offsets=P, out=P, od=BF16, stream=None)
    _table(L, L.bsq_moe_wgrad, base, [
        ({}, DEVICE), (dict(cap=0, dy=None, x=None, sd=None, sx=None), DEVICE), (dict(N=0), OK), (dict(K=0), OK),
        (dict(cap=-128), SHAPE), (dict(cap=64), SHAPE), (dict(E=0), SHAPE), (dict(N=24), UNSUP), (dict(K=24), UNSUP),
        (dict(E=1025), UNSUP), (dict(xd=E5), UNSUP), (dict(dd=bsq.BSQ_I8), UNSUP), (dict(od=42), DTYPE),
        (dict(cap=1 << 31), UNSUP), (dict(cap=1 << 30, N=1 << 10), UNSUP), (dict(out=None), NULL), (dict(dy=None), NULL),
        (dict(sx=None), NULL), (dict(offsets=None), NULL), (dict(out=P4), ALIGN), (dict(sd=P + 2), ALIGN)])


def test_swiglu(L):
    base = dict(R=64, F=64, gu=P, dt=BF16, cd=E4, h=P, hs=P, ht=P, hts=P, kept=P, ks=P, stream=None)
    _table(L, L.bsq_swiglu_mx, base, [
        ({}, DEVICE), (dict(ht=None, hts=None, R=63), DEVICE), (dict(kept=None, ks=None), DEVICE), (dict(R=0), OK),
        (dict(F=0), OK), (dict(R=-1), SHAPE), (dict(F=48), SHAPE), (dict(R=63), SHAPE), (dict(R=BIG), UNSUP),
        (dict(dt=42), DTYPE), (dict(dt=E4), UNSUP), (dict(cd=BF16), UNSUP), (dict(hts=None), NULL),
        (dict(ks=None), NULL), (dict(h=None), NULL), (dict(hs=None), NULL), (dict(gu=None), NULL), (dict(gu=P4), ALIGN),
        (dict(kept=P4), ALIGN)])
    base = dict(R=63, F=64, kept=P, cd=E4, ks=P, dh=P, dt=BF16, dgu=P, stream=None)
    _table(L, L.bsq_swiglu_mx_backward, base, [
        ({}, DEVICE), (dict(R=0), OK), (dict(F=48), SHAPE), (dict(dt=42), DTYPE), (dict(cd=F32), UNSUP),
        (dict(kept=None), NULL), (dict(ks=None), NULL), (dict(dh=None), NULL), (dict(dgu=None), NULL), (dict(dgu=P4), ALIGN)])


def test_binding_refuses_tensors_off_the_gpu():
    t = torch.zeros
    i = lambda *s: t(*s, dtype=torch.int32)  # noqa: E731
    b = lambda *s: t(*s, dtype=torch.uint8)  # noqa: E731
    calls = [lambda: bsq.bsq_moe_route(t(4, 8), i(4, 2), t(4, 2)),
             lambda: bsq.bsq_moe_route_backward(t(4, 8), i(4, 2), t(4, 2), t(4, 8)),
             lambda: bsq.bsq_moe_plan(i(4, 2), i(9), i(8), i(8), i(4, 2), b(64)),
             lambda: bsq.bsq_moe_gather_mx(t(4, 32), i(32), 2, b(32, 32), b(32, 1)),
             lambda: bsq.bsq_moe_combine(t(8, 32), i(4, 2), t(4, 32)),
             lambda: bsq.bsq_moe_combine_backward(t(8, 32), i(4, 2), t(4, 32), t(4, 2)),
             lambda: bsq.bsq_moe_matmul(b(4, 128), b(4, 4), b(2, 16, 128), b(2, 16, 4), i(3), t(8, 16)),
             lambda: bsq.bsq_moe_wgrad(b(16, 128), b(16, 4), b(16, 128), b(16, 4), i(3), t(2, 16, 16)),
             lambda: bsq.bsq_swiglu_mx(t(4, 64), b(4, 32), b(4, 1)),
             lambda: bsq.bsq_swiglu_mx_backward(b(4, 64), b(4, 2), t(4, 32), t(4, 64))]
    for c in calls:
        with pytest.raises(ValueError, match="GPU"):
            c()
