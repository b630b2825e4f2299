"""The operators of include/rmsnorm_serving.h without a GPU: refusals (all before the library
touches CUDA)."""
import pytest

from rmsnorm_fwd_bwd_gb300 import binding as B
from rmsnorm_fwd_bwd_gb300 import build as build_mod

OK, NULL, SHAPE, DTYPE, EPS, ALIGN, WORKSPACE, ARG = 0, 1, 2, 3, 4, 5, 6, 9


@pytest.fixture(scope="module", autouse=True)
def library():
    build_mod.build()


def weight(**kw):
    a = dict(w=0x100000, ldw=256, codes=0x200000, ldcodes=256, scales=0x300000, ldscales=2, N=300, K=256, dtype=2,
             pow2=0, stream=0)
    a.update(kw)
    return B.rmsnorm_quant_weight(**a)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=3)), (DTYPE, dict(dtype=-1)), (ARG, dict(pow2=2)), (SHAPE, dict(N=-1)), (SHAPE, dict(K=0)),
    (SHAPE, dict(N=(1 << 20) + 1)), (SHAPE, dict(K=(1 << 20) + 1, ldw=1 << 21, ldcodes=1 << 21, ldscales=1 << 14)),
    (SHAPE, dict(ldw=255)), (SHAPE, dict(ldcodes=255)), (SHAPE, dict(ldscales=1)), (OK, dict(N=0, w=None, codes=None)),
    (NULL, dict(w=None)), (NULL, dict(codes=None)), (NULL, dict(scales=None)), (ALIGN, dict(w=0x100001)),
    (ALIGN, dict(scales=0x300002)), (ARG, dict(codes=0x100000)), (ARG, dict(codes=0x100000 + 299 * 512)),
    (ARG, dict(scales=0x200000)), (ARG, dict(scales=0x100010)),
])
def test_quant_weight_refusals(want, kw):
    assert weight(**kw) == want


def matmul(**kw):
    a = dict(a=0x1000000, lda=256, a_scales=0x2000000, ldas=2, b=0x3000000, ldb=256, b_scales=0x4000000, ldbs=2,
             bias=0x5000000, y=0x6000000, ldy=300, M=20, N=300, K=256, dtype=2, group=128, stream=0)
    a.update(kw)
    return B.rmsnorm_quant_matmul(**a)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=3)), (ARG, dict(group=64)), (ARG, dict(group=-128)), (SHAPE, dict(M=-1)), (SHAPE, dict(N=0)),
    (SHAPE, dict(K=0)), (SHAPE, dict(N=(1 << 20) + 1)), (SHAPE, dict(M=1 << 31)), (SHAPE, dict(lda=255)),
    (SHAPE, dict(ldas=1)), (SHAPE, dict(group=0, ldas=0)), (SHAPE, dict(ldb=255)), (SHAPE, dict(ldbs=1)),
    (SHAPE, dict(ldy=299)), (OK, dict(M=0, a=None, y=None)), (NULL, dict(a=None)), (NULL, dict(a_scales=None)),
    (NULL, dict(b=None)), (NULL, dict(b_scales=None)), (NULL, dict(y=None)), (ALIGN, dict(a_scales=0x2000001)),
    (ALIGN, dict(b_scales=0x4000002)), (ALIGN, dict(bias=0x5000001)), (ALIGN, dict(y=0x6000001)),
    (ARG, dict(y=0x1000000)), (ARG, dict(y=0x3000000 + 256 * 299 + 254)), (ARG, dict(y=0x5000000 + 2)),
    (ARG, dict(y=0x4000008)), (ARG, dict(y=0x2000000 - 100)),
])
def test_quant_matmul_refusals(want, kw):
    assert matmul(**kw) == want
