"""The operators of include/rmsnorm_serving.h on the GPU, against their formulas in 64 bits.

Bounds, with u = 2^-24. A code times a code has 8 significant bits and is exact in fp32. The
tensor cores add the 128 products of a block one after the other in fp32; each addition is
taken to lose up to a unit in the last place (truncation), 2 u of the magnitudes that went
in: 256 u of the sum of the magnitudes in all. The product of a pair of scales is off by u, a
multiply-add per block by u, the sums of up to 8 blocks of a cluster by u each, and the bias by
u. One rounding to y's type is half a step. The smallest results are off by half of the
least subnormal.
"""
import pytest
import torch

from rmsnorm_fwd_bwd_gb300 import binding as B
from tests import fused_ref as ref

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
DTYPES = ["float32", "float16", "bfloat16"]
U = ref.U
SHAPES = [(1, 128, 128), (1, 1, 1), (3, 7, 5), (16, 256, 384), (17, 130, 1000), (33, 400, 512), (64, 1024, 2048), (100, 300, 129),
          (128, 640, 1152), (129, 256, 128), (200, 1000, 640), (300, 700, 4099), (513, 520, 136), (7, 6144, 4096)]


@pytest.fixture(autouse=True)
def _clean():
    assert torch.cuda.is_available()
    B.rmsnorm_device_error(clear=True)
    yield
    assert B.rmsnorm_device_error(clear=True) == 0


def codes(rows, cols, seed, layout="dense", scale=60.0):
    """Random codes in a buffer of codes that no call may read as operands (NaN); (view, pitch)."""
    g = torch.Generator().manual_seed(seed)
    v = (torch.randn(rows, cols, generator=g) * scale).clamp(-448, 448).to(F8)
    pitch, start = {"dense": (cols, 0), "padded": (-(-cols // 16) * 16 + 32, 0), "shifted": (cols + 3, 5),
                    "odd pitch": (cols + 1, 16)}[layout]
    buf = torch.full((start + rows * pitch + 64,), 0x7F, dtype=torch.uint8)
    out = buf[start:start + rows * pitch].view(rows, pitch)
    out[:, :cols] = v.view(torch.uint8)
    return buf.cuda().view(F8)[start:start + rows * pitch].view(rows, pitch)[:, :cols], pitch


def spread(s, rows, cols, group_rows=128):
    return s.double().repeat_interleave(group_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def product_inputs(M, N, K, group, seed=0, layout="dense"):
    a, lda = codes(M, K, seed, layout)
    b, ldb = codes(N, K, seed + 1, layout)
    g = torch.Generator().manual_seed(seed + 2)
    n, k = -(-N // 128), -(-K // 128)
    sa = torch.exp(torch.randn(M, k if group else 1, generator=g)).cuda() * 0.01
    sb = torch.exp(torch.randn(n, k, generator=g)).cuda() * 0.003
    return a, lda, b, ldb, sa, sb


def product(a, lda, b, ldb, sa, sb, dtype, group, bias=None, y=None, stream=None):
    M, N = a.shape[0], b.shape[0]
    if y is None:
        y = torch.full((M, N + 3), 7.0, dtype=ref.TYPES[dtype], device="cuda")
    st = B.rmsnorm_quant_matmul(a, lda, sa, sa.shape[1], b, ldb, sb, sb.shape[1], bias, y, y.stride(0), M, N, a.shape[1],
                                dtype, group, stream)
    assert st == 0
    return y


def product_bound(a, b, sa, sb, group, bias=None):
    """y in 64 bits and the bound on its error before the rounding."""
    M, K = a.shape
    N = b.shape[0]
    fa = a.double() * (sa.double().repeat_interleave(128, 1)[:, :K] if group else sa.double())
    fb = b.double() * spread(sb, N, K)
    want, mag = fa @ fb.t(), fa.abs() @ fb.abs().t()
    if bias is not None:
        want, mag = want + bias.double(), mag + bias.double().abs()
    return want, (256 + -(-K // 128) + 8 + 3) * U * mag


def check_product(a, b, sa, sb, dtype, group, y, bias=None):
    want, err = product_bound(a, b, sa, sb, group, bias)
    N = b.shape[0]
    ref.assert_close(y[:, :N], want, err + ref.rounding(want.abs() + err, ref.TYPES[dtype]), "y")
    assert (y[:, N:] == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul_shapes(M, N, K, group, dtype):
    a, lda, b, ldb, sa, sb = product_inputs(M, N, K, group)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(5)).to(ref.TYPES[dtype]).cuda() if N % 2 == 0 else None
    check_product(a, b, sa, sb, dtype, group, product(a, lda, b, ldb, sa, sb, dtype, group, bias), bias)


@pytest.mark.parametrize("layout", ["padded", "shifted", "odd pitch"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul_layouts(M, N, K, layout):
    a, lda, b, ldb, sa, sb = product_inputs(M, N, K, 128, 3, layout)
    check_product(a, b, sa, sb, "bfloat16", 128, product(a, lda, b, ldb, sa, sb, "bfloat16", 128))


@pytest.mark.parametrize("layout", ["padded", "shifted"])
@pytest.mark.parametrize("M,N,K", [(5, 300, 700), (40, 129, 1000), (100, 256, 640), (260, 300, 300)])
def test_matmul_of_whole_numbers_is_exact(M, N, K, layout):
    # sums of small whole numbers times powers of two, in any order: every entry has its place
    g = torch.Generator().manual_seed(11)
    a, lda = codes(M, K, 0, layout)
    b, ldb = codes(N, K, 1, layout)
    a.copy_(torch.randint(-4, 5, (M, K), generator=g).float())
    b.copy_(torch.randint(-4, 5, (N, K), generator=g).float())
    sa = 2.0 ** torch.randint(-2, 3, (M, -(-K // 128)), generator=g).float().cuda()
    sb = 2.0 ** torch.randint(-2, 3, (-(-N // 128), -(-K // 128)), generator=g).float().cuda()
    y = product(a, lda, b, ldb, sa, sb, "float32", 128)
    assert torch.equal(y[:, :N].double(), product_bound(a, b, sa, sb, 128)[0])


# --------------------------------------------------------------------------- #
# weights
# --------------------------------------------------------------------------- #
def quant_weight(w, ldw, N, K, dtype, pow2, pad=3):
    c = torch.full((N, K + pad), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((-(-N // 128), -(-K // 128) + 1), 7.0, device="cuda")
    assert B.rmsnorm_quant_weight(w, ldw, c, K + pad, s, s.shape[1], N, K, dtype, pow2) == 0
    assert (c[:, K:] == 0x55).all() and (s[:, -1] == 7.0).all()
    return c[:, :K].view(F8), s[:, :-1]


def weight_blocks(w):
    """w [N, K] as [block rows, 128, block columns, 128], padded with zeros."""
    N, K = w.shape
    n, k = -(-N // 128), -(-K // 128)
    return torch.nn.functional.pad(w, (0, k * 128 - K, 0, n * 128 - N)).view(n, 128, k, 128)


def check_weight(w, c, s, pow2):
    N, K = w.shape
    # fp32 quotients, exactly rounded: in 64 bits first, which has more than twice the bits (torch
    # on the GPU divides by a number by multiplying by its inverse)
    want = (weight_blocks(w.double()).abs().amax((1, 3)) / 448.0).float().clamp_min(2.0 ** -126)
    if pow2:
        want = torch.exp2(torch.ceil(torch.log2(want.double()))).float()
    assert torch.equal(s, want)
    q = (w.double() / spread(s, N, K)).float()
    assert torch.equal(c.view(torch.uint8), q.to(F8).view(torch.uint8))
    # a code is off by at most half a step of e4m3, 2^-4 of the value, 2^-10 below 2^-6
    v = w.double() / spread(s, N, K)
    ref.assert_close(c.double(), v, v.abs() * (2.0 ** -4 + U) + 2.0 ** -10, "codes")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("layout", ["dense", "pitched", "shifted"])
@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (129, 127), (300, 1000), (5, 4099), (257, 640)])
def test_weight_shapes(N, K, layout, pow2, dtype):
    dt = ref.TYPES[dtype]
    pitch, start = {"dense": (K, 0), "pitched": (-(-K // 8) * 8 + 8, 0), "shifted": (K + 5, 3)}[layout]
    buf = torch.full((start + N * pitch + 8,), float("nan"), dtype=dt, device="cuda")
    w = buf[start:start + N * pitch].view(N, pitch)[:, :K]
    g = torch.Generator().manual_seed(N + K)
    w.copy_((torch.randn(N, K, generator=g) * torch.exp(2 * torch.randn(N, 1, generator=g))).to(dt))
    c, s = quant_weight(w, pitch, N, K, dtype, pow2, pad=8 if layout == "pitched" else 3)
    check_weight(w, c, s, pow2)


def test_weight_special_values():
    w = torch.ones(300, 400, device="cuda")
    w[0:128, 0:128] = 0.0
    w[5, 200] = float("nan")
    w[130, 10] = float("-inf")
    w[140, 300] = 1e-40
    w[256:, 256:384] = -1e-42
    c, s = quant_weight(w, 400, 300, 400, "float32", False)
    v = c.double()
    assert s[0, 0] == 2.0 ** -126 and (v[:128, :128] == 0).all()
    assert torch.isnan(s[0, 1]) and torch.isnan(v[:128, 128:256]).all()
    assert torch.isinf(s[1, 0]) and torch.isnan(v[130, 10]) and (v[131:256, :128] == 0).all()
    assert s[2, 2] == 2.0 ** -126
    assert torch.isfinite(v[128:, 128:]).all() and torch.isfinite(s[1:, 1:]).all()
