"""Refusals of the calls on 4-bit operands and of the norm, on the host and
without a GPU: every rule of include/bsq.h that a caller can break, through the
C ABI with fake addresses that are never dereferenced; and the binding's own
checks."""
import pytest
import torch

import block_scaled_precision_blockwise_amd as bsq
from test_moe_abi import ALIGN, BIG, BF16, DEVICE, DTYPE, E4, E5, F32, NULL, OK, P, P4, SHAPE, UNSUP, L, _table  # noqa: F401

E2 = bsq.BSQ_E2M1
MX, NV = bsq.BSQ_MXFP4, bsq.BSQ_NVFP4


def test_quant_fp4(L):  # noqa: F811
    base = dict(B=2, rows=64, cols=96, src=P, dt=BF16, format=MX, factor=None, codes=P, scales=P, ct=P, st=P, stream=None)
    _table(L, L.bsq_quant_fp4, base, [
        ({}, DEVICE), (dict(codes=None, scales=None), DEVICE), (dict(ct=None, st=None), DEVICE),
        (dict(ct=None, st=None, rows=7), DEVICE), (dict(format=NV, rows=48, cols=16), DEVICE),
        (dict(format=NV, factor=P), DEVICE), (dict(scales=P + 1, st=P + 3), DEVICE),
        (dict(codes=None, scales=None, ct=None, st=None), OK), (dict(B=0), OK), (dict(rows=0), OK), (dict(cols=0), OK),
        (dict(B=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(cols=-32), SHAPE), (dict(cols=48), SHAPE),
        (dict(rows=48), SHAPE), (dict(format=NV, rows=40), SHAPE), (dict(format=NV, cols=24), SHAPE),
        (dict(dt=42), DTYPE), (dict(format=2), DTYPE), (dict(format=-1), DTYPE), (dict(dt=E4), UNSUP), (dict(dt=E2), UNSUP),
        (dict(factor=P), UNSUP), (dict(B=BIG), UNSUP), (dict(B=1, rows=1 << 40, cols=32), UNSUP),
        (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(ct=None), NULL), (dict(st=None), NULL), (dict(src=None), NULL),
        (dict(src=P4), ALIGN), (dict(codes=P4), ALIGN), (dict(ct=P4), ALIGN), (dict(format=NV, factor=P + 2), ALIGN)])


PRODUCT = [
    (dict(ad=E4), DEVICE), (dict(ad=E5, od=BF16), DEVICE), (dict(K=32), DEVICE), (dict(K=16), SHAPE), (dict(K=-32), SHAPE),
    (dict(N=-16), SHAPE), (dict(N=24), UNSUP), (dict(N=0), OK), (dict(K=0, a=None, b=None, sa=None, sb=None), DEVICE),
    (dict(ad=F32), UNSUP), (dict(ad=bsq.BSQ_E8M0), UNSUP), (dict(od=E2), UNSUP), (dict(ad=42), DTYPE), (dict(od=-1), DTYPE),
    (dict(K=1 << 25), UNSUP), (dict(N=1 << 31), UNSUP), (dict(N=1 << 30, K=1 << 20), UNSUP),
    (dict(a=None), NULL), (dict(b=None), NULL), (dict(sa=None), NULL), (dict(sb=None), NULL), (dict(out=None), NULL),
    (dict(a=P4), ALIGN), (dict(b=P4), ALIGN), (dict(out=P4), ALIGN), (dict(sa=P + 2), ALIGN), (dict(sb=P + 1), ALIGN),
    (dict(sa=P4, sb=P4), DEVICE)]


def test_scaled_matmul(L):  # noqa: F811
    base = dict(B=2, M=3, N=48, K=96, a=P, ad=E2, b=P, sa=P, sb=P, out=P, od=F32, stream=None)
    _table(L, L.bsq_scaled_matmul_mxfp4, base, [({}, DEVICE)] + PRODUCT + [
        (dict(B=0), OK), (dict(M=0), OK), (dict(B=-1), SHAPE), (dict(M=-1), SHAPE), (dict(B=65536), UNSUP),
        (dict(M=1 << 31), UNSUP), (dict(M=1 << 30, K=1 << 10), UNSUP), (dict(B=1, M=1 << 30, N=1 << 20), UNSUP),
        (dict(B=65535, M=1 << 24, N=16), UNSUP)])


def test_moe_matmul(L):  # noqa: F811
    base = dict(T=10, cap=64, E=4, N=48, K=96, k=2, a=P, ad=E2, sa=P, b=P, sb=P, offsets=P, rows=P, out=P, od=F32,
                stream=None)
    _table(L, L.bsq_moe_matmul_mxfp4, base, [({}, DEVICE)] + PRODUCT + [
        (dict(rows=None), DEVICE), (dict(T=0, a=None, b=None, sa=None, sb=None), DEVICE), (dict(cap=0), OK),
        (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(k=0), SHAPE), (dict(cap=-1), SHAPE), (dict(E=1025), UNSUP),
        (dict(T=1 << 31), UNSUP), (dict(T=1 << 30, K=1 << 10), UNSUP), (dict(cap=(1 << 31) - (1 << 16) + 1), UNSUP),
        (dict(cap=(1 << 31) - (1 << 16), N=1 << 10), UNSUP), (dict(k=1 << 31), UNSUP), (dict(offsets=None), NULL),
        (dict(rows=P4), ALIGN), (dict(offsets=P4), ALIGN)])


def test_norm(L):  # noqa: F811
    base = dict(R=5, C=96, x=P, dt=BF16, kind=0, eps=1e-5, gamma=P, beta=P, y=P, cd=E2, codes=P, scales=P, mean=P, rstd=P,
                stream=None)
    _table(L, L.bsq_norm_mx, base, [
        ({}, DEVICE), (dict(cd=E4, kind=1), DEVICE), (dict(gamma=None, beta=None, mean=None, rstd=None), DEVICE),
        (dict(codes=None, scales=None, cd=42, C=95), DEVICE), (dict(y=None), DEVICE), (dict(R=0), OK), (dict(C=0), OK),
        (dict(R=-1), SHAPE), (dict(C=-1), SHAPE), (dict(C=95), SHAPE), (dict(C=(1 << 24) + 32), UNSUP), (dict(R=BIG), UNSUP),
        (dict(dt=42), DTYPE), (dict(cd=42), DTYPE), (dict(kind=2), DTYPE), (dict(kind=-1), DTYPE), (dict(dt=E4), UNSUP),
        (dict(cd=F32), UNSUP), (dict(eps=-1.0), UNSUP), (dict(eps=float("nan")), UNSUP), (dict(x=None), NULL),
        (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(x=P4), ALIGN), (dict(y=P4), ALIGN),
        (dict(codes=P4), ALIGN), (dict(gamma=P4), ALIGN), (dict(beta=P4), ALIGN), (dict(mean=P + 2), ALIGN),
        (dict(rstd=P + 1), ALIGN), (dict(mean=P4, rstd=P4), DEVICE)])
    base = dict(R=5, C=95, x=P, dy=P, dt=F32, kind=0, gamma=P, mean=P, rstd=P, dx=P, dg=P, db=P, ws=P, wb=1 << 20, stream=None)
    _table(L, L.bsq_norm_backward, base, [
        ({}, DEVICE), (dict(kind=1, mean=None), DEVICE), (dict(gamma=None), DEVICE), (dict(dg=None), DEVICE),
        (dict(dg=None, db=None, ws=None, wb=0), DEVICE), (dict(R=0, x=None, dy=None, dx=None, mean=None, rstd=None), DEVICE),
        (dict(R=0, dg=None, db=None), OK), (dict(C=0), OK), (dict(R=-1), SHAPE), (dict(wb=8 * 95 * 5 - 1), SHAPE),
        (dict(wb=8 * 95 * 5), DEVICE), (dict(C=(1 << 24) + 1), UNSUP), (dict(dt=42), DTYPE), (dict(kind=3), DTYPE),
        (dict(dt=E5), UNSUP), (dict(x=None), NULL), (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(mean=None), NULL),
        (dict(rstd=None), NULL), (dict(ws=None), NULL), (dict(dx=P4), ALIGN), (dict(gamma=P4), ALIGN), (dict(dg=P + 2), ALIGN),
        (dict(db=P + 2), ALIGN), (dict(rstd=P + 2), ALIGN), (dict(ws=P4), ALIGN)])


def test_workspace():
    f = bsq.bsq_norm_backward_workspace_bytes
    assert f(0, 64) == 16 and f(3, 64) == 8 * 64 * 3 and f(10 ** 6, 64) == 8 * 64 * 1024
    assert f(-1, 64) == 0 and f(1, -1) == 0 and f(1, (1 << 24) + 1) == 2 ** 64 - 1


def test_binding_refuses_tensors_off_the_gpu():
    t = torch.zeros
    i = lambda *s: t(*s, dtype=torch.int32)  # noqa: E731
    b = lambda *s: t(*s, dtype=torch.uint8)  # noqa: E731
    calls = [lambda: bsq.bsq_quant_fp4(t(32, 64), b(32, 32), b(32, 2)),
             lambda: bsq.bsq_scaled_matmul_mxfp4(b(1, 4, 32), b(1, 16, 32), b(1, 4, 2), b(1, 16, 2), t(1, 4, 16)),
             lambda: bsq.bsq_moe_matmul_mxfp4(b(4, 32), b(4, 2), b(2, 16, 32), b(2, 16, 2), i(3), t(8, 16)),
             lambda: bsq.bsq_norm_mx(t(4, 64), y=t(4, 64)),
             lambda: bsq.bsq_norm_backward(t(4, 64), t(4, 64), t(4), t(4, 64), mean=t(4))]
    for c in calls:
        with pytest.raises(ValueError, match="GPU"):
            c()
    with pytest.raises(TypeError):
        bsq.bsq_norm_mx([1.0, 2.0])
