"""The largest sizes of the expert-layer calls, on the host and without a GPU:
what is beyond them is refused before a device is looked for."""
import pytest

import block_scaled_precision_blockwise_amd as bsq

OK, NULL, SHAPE, DTYPE, UNSUP, ALIGN, DEVICE, HIP = range(8)
P = 0x1000  # an address that is never dereferenced
F32, BF16, E4, E5 = bsq.BSQ_F32, bsq.BSQ_BF16, bsq.BSQ_E4M3, bsq.BSQ_E5M2


@pytest.fixture(scope="module")
def L():
    if not bsq.is_built():
        import __graft_entry__
        __graft_entry__.build()
    return bsq.lib()


def _call(f, base, change):
    return f(*dict(base, **change).values())


MATMUL = dict(T=10, cap=64, E=4, N=16, K=256, k=2, a=P, ad=E4, sa=P, b=P, bd=E4, sb=P, offsets=P, rows=P, out=P,
              od=BF16, stream=None)


@pytest.mark.parametrize("rows,T", [(P, 10), (None, 1 << 29)])
def test_rows_of_a_product(L, rows, T):
    most = (1 << 31) - (1 << 16)
    for cap, want in ((most, DEVICE), (most + 1, UNSUP), ((1 << 31) - 1, UNSUP)):
        assert _call(L.bsq_moe_matmul, MATMUL, dict(cap=cap, rows=rows, T=T, K=128)) == want, cap
