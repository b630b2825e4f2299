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


# --------------------------------------------------------------------------- #
# keys and values into a paged cache
# --------------------------------------------------------------------------- #
EPS = 1e-6


class Cache:
    """A paged cache [pages, size, heads, D] of one type in one of the orders that caches have, filled with
    a byte that tells what was written; ``t`` and ``s`` are the rows and their scales (or None)."""

    def __init__(self, pages, size, heads, D, dtype, bits8, order, seed=0):
        dt = F8 if bits8 else ref.TYPES[dtype]
        e = torch.empty(0, dtype=dt).element_size()
        gap = {"spaced": 3}.get(order, 0)
        width = D + gap
        if order in ("rows", "spaced"):
            strides = (size * heads * width, heads * width, width)
        elif order == "heads first":
            strides = (heads * size * width, width, size * width)
        elif order == "keys and values":                    # [pages, 2, size, heads, D]
            strides = (2 * size * heads * width, heads * width, width)
        self.buf = torch.full((pages * strides[0] * e + 64 * e,), 0x55, dtype=torch.uint8, device="cuda")
        typed = self.buf.view(dt)
        self.start = gap
        self.t = typed.as_strided((pages, size, heads, D), (*strides, 1), self.start)
        self.typed, self.strides, self.shape = typed, strides, (pages, size, heads, D)
        self.sbuf = torch.full((pages, size, heads + gap), 7.0, device="cuda") if bits8 else None
        self.s = self.sbuf[..., :heads] if bits8 else None

    def other(self):
        """The values' half of a cache of keys and values."""
        c = object.__new__(Cache)
        c.__dict__ = dict(self.__dict__)
        _, size, heads, D = self.shape
        c.start = size * heads * (self.strides[2])
        c.t = self.typed.as_strided(self.shape, (*self.strides, 1), c.start)
        if self.sbuf is not None:
            c.sbuf = torch.full_like(self.sbuf, 7.0)
            c.s = c.sbuf[..., :heads]
        return c

    def rows(self, slots):
        size = self.shape[1]
        return self.t[slots // size, slots % size], None if self.s is None else self.s[slots // size, slots % size]

    def untouched_but(self, slots, *more):
        """Every byte that is not a row of the given slots (of this cache and others in its buffer) is as it was."""
        mark = torch.zeros(self.typed.shape, dtype=torch.bool, device="cuda")
        for c in (self, *more):
            view = mark.as_strided(c.shape, (*c.strides, 1), c.start)
            view[slots // c.shape[1], slots % c.shape[1]] = True
        raw = self.buf.view(-1, self.typed.element_size())
        assert (raw[~mark] == 0x55).all(), "written outside the slots"
        for c in (self, *more):
            if c.sbuf is not None:
                m = torch.zeros(c.sbuf.shape, dtype=torch.bool, device="cuda")
                m[slots // c.shape[1], slots % c.shape[1], :c.shape[2]] = True
                assert (c.sbuf[~m] == 7.0).all()


def randn(*shape, dtype, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(ref.TYPES[dtype])


def freqs(R, base=10000.0):
    return torch.tensor([base ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64)


def spaced_heads(x, how):
    """x [T, H, D] on the GPU, as it lies in one of the layouts that a model has."""
    T, H, D = x.shape
    lead, tok, head = {"dense": (0, H * D, D), "fused": (2 * D, (H + 5) * D, D), "odd": (3, H * (D + 5) + 1, D + 5)}[how]
    buf = torch.full((lead + T * tok + D + 64,), 3.0).to(x.dtype).cuda()
    t = buf.as_strided((T, H, D), (tok, head, 1), lead)
    t.copy_(x)
    return t


def check_rows(got, scales, x, w, pos, R, inter, mscale, offset, dtype):
    """Rows of a cache against z: rotated keys, or the values as they are (w: "values")."""
    if isinstance(w, str):
        if scales is None:
            assert torch.equal(got.view(torch.uint8), x.cuda().view(torch.uint8))
            return
        z, err = x.double(), torch.zeros(x.shape, dtype=torch.float64)
    else:
        z, err = ref.rope_fwd(x, w, pos, freqs(R), inter, mscale, EPS, offset)
    if scales is None:
        ref.assert_close(got, z, err + ref.rounding(z.abs() + err, ref.TYPES[dtype]), "rows")
        return
    s = scales.double().cpu().unsqueeze(-1)
    amax = z.abs().amax(-1, keepdim=True)
    # the largest |z| is off by at most the largest error, the product with r / 448 by 3 u
    ref.assert_close(s, (amax / 448.0).clamp_min(2.0 ** -126), (err.amax(-1, keepdim=True) + 3 * U * amax) / 448.0, "scales")
    # the factors r / scale: 1 / scale off by a unit in the last place (2 u) and the products by u each
    off = err + 5 * U * z.abs()
    ref.assert_close(got.double().cpu() * s, z, off + torch.maximum((z.abs() + off) * 2.0 ** -4, s * 2.0 ** -10), "codes")


def run_append(T, Hq, Hk, D, R, dtype, size=16, bits8=(False, False), inter=False, offset=False, mscale=1.0, order="rows",
               how="dense", pos=None, slots=None, weights=True, with_q=True, with_v=True, seed=80, in_place=False):
    q, k, v = (randn(T, h, D, dtype=dtype, seed=seed + i, scale=1.5) for i, h in enumerate((Hq, Hk, Hk)))
    wq = wk = None
    if weights:
        wq, wk = (randn(D, dtype=dtype, seed=seed + 3 + i, scale=0.2) + (0 if offset else 1) for i in range(2))
    pages = -(-T // size) + 3
    if slots is None:
        slots = torch.randperm(pages * size, generator=torch.Generator().manual_seed(seed + 9))[:T]
    if pos is None:
        pos = torch.arange(T) * 37 + 5
    kc = Cache(pages, size, Hk, D, dtype, bits8[0], order)
    vc = kc.other() if order == "keys and values" else Cache(pages, size, Hk, D, dtype, bits8[1], order)
    qg, kg, vg = (spaced_heads(t, how) for t in (q, k, v))
    out = qg if in_place else torch.full((T, Hq, D), 5.0).to(qg.dtype).cuda()
    wg = [None if w is None else w.cuda() for w in (wq, wk)]
    sg, pg, fg = slots.cuda(), pos.cuda(), freqs(R).cuda()
    st = B.rmsnorm_rope_append(B.rope_heads([(qg, wg[0], out)]) if with_q else None, B.cache_heads(kg, wg[1], kc.t, kc.s),
                               B.cache_heads(vg, None, vc.t, vc.s) if with_v else None, sg, pages, size, pg, T, D, R, fg,
                               int(inter), mscale, EPS, dtype, int(offset))
    assert st == 0, B.rmsnorm_status_string(st)
    stored = (slots >= 0) & (slots < pages * size)
    at = slots[stored].cuda()
    if order == "keys and values":
        kc.untouched_but(at, vc)
    else:
        kc.untouched_but(at)
        vc.untouched_but(at if with_v else at[:0])
    check_rows(*kc.rows(at), k[stored], wk, pos[stored], R, inter, mscale, offset, dtype)
    if with_v:
        check_rows(*vc.rows(at), v[stored], "values", None, R, inter, mscale, offset, dtype)
    if with_q:
        want, err = ref.rope_fwd(q, wq, pos, freqs(R), inter, mscale, EPS, offset)
        ref.assert_close(out, want, err + ref.rounding(want.abs() + err, ref.TYPES[dtype]), "queries")
    return kc, vc, out


HEADS = [(1, 1, 1, 2, 2), (5, 3, 1, 8, 8), (3, 2, 2, 16, 16), (7, 4, 2, 64, 64), (6, 5, 1, 64, 32), (4, 8, 2, 80, 80),
         (4, 3, 3, 96, 48), (9, 7, 1, 128, 128), (3, 32, 8, 128, 128), (5, 2, 1, 128, 24), (3, 4, 4, 192, 128),
         (4, 3, 1, 256, 256), (2, 3, 1, 512, 512), (5, 2, 1, 33, 32), (3, 2, 1, 77, 6), (2, 2, 1, 511, 510), (2, 5, 3, 90, 90),
         (700, 5, 2, 64, 64), (3, 70, 9, 40, 16), (900, 12, 4, 80, 40), (300, 9, 3, 90, 44)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R", HEADS)
def test_append_shapes(T, Hq, Hk, D, R, bits8, inter, dtype):
    run_append(T, Hq, Hk, D, R, dtype, bits8=(bits8, bits8), inter=inter)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("how", ["fused", "odd"])
@pytest.mark.parametrize("order,bits8", [(o, (k, v)) for o in ("heads first", "spaced", "keys and values") for k in (False, True)
                                         for v in (False, True) if o != "keys and values" or k == v])  # one tensor has one type
def test_append_layouts(order, bits8, how, dtype):
    for T, Hq, Hk, D, R in ((6, 3, 2, 64, 32), (50, 4, 1, 128, 128), (40, 3, 3, 36, 20), (40, 4, 2, 72, 40)):
        for size in (1, 7, 64):
            run_append(T, Hq, Hk, D, R, dtype, size=size, bits8=bits8, offset=True, mscale=1.25, order=order, how=how)


@pytest.mark.parametrize("bits8", [False, True])
def test_append_without_weights_queries_or_values(bits8):
    for D, R in ((64, 64), (64, 24), (50, 30)):
        run_append(9, 4, 2, D, R, "bfloat16", bits8=(bits8, bits8), weights=False)
        run_append(9, 4, 2, D, R, "bfloat16", bits8=(bits8, bits8), with_q=False)
        run_append(9, 4, 2, D, R, "float16", bits8=(bits8, bits8), with_v=False)
        run_append(9, 4, 2, D, R, "float32", bits8=(bits8, bits8), with_q=False, with_v=False)
        run_append(9, 4, 2, D, R, "bfloat16", bits8=(bits8, bits8), in_place=True, how="fused")


@pytest.mark.parametrize("bits8", [False, True])
def test_append_padded_tokens_and_slots_behind_the_last(bits8):
    for D, R in ((64, 64), (64, 24), (50, 30)):
        slots = torch.randperm(96)[:60]
        slots[::3] = -1
        slots[7] = -(1 << 40)
        run_append(60, 4, 2, D, R, "bfloat16", bits8=(bits8, bits8), slots=slots)
        assert B.rmsnorm_device_error(clear=True) == 0
        slots[5] = 7 * 16                                   # the first behind seven pages of 16
        slots[8] = 1 << 62
        run_append(60, 4, 2, D, R, "bfloat16", bits8=(bits8, bits8), slots=slots)
        assert B.rmsnorm_device_error(clear=True) == 4


def test_append_to_a_cache_of_more_than_2_to_the_32_entries():
    # 8 GiB and more of codes: offsets past 32 bits, of which a few rows are read
    pages, size, H, D = 70000, 64, 8, 128
    kc = torch.empty(pages, size, H, D, dtype=F8, device="cuda")
    ks = torch.empty(pages, size, H, device="cuda")
    T = 5
    k, w = randn(T, H, D, dtype="bfloat16", seed=1), randn(D, dtype="bfloat16", seed=2) + 1
    slots = torch.tensor([0, pages * size - 1, (1 << 22) + 1, 3, pages * size // 2])
    pos = torch.arange(T)
    kg, wg, sg, pg, fg = k.cuda(), w.cuda(), slots.cuda(), pos.cuda(), freqs(D).cuda()
    heads = B.cache_heads(kg, wg, kc, ks)
    assert B.rmsnorm_rope_append(None, heads, None, sg, pages, size, pg, T, D, D, fg, 0, 1.0, EPS, "bfloat16", 0) == 0
    check_rows(kc[sg // size, sg % size], ks[sg // size, sg % size], k, w, pos, D, False, 1.0, False, "bfloat16")


def test_append_of_infinities_and_nan_keeps_them_in_their_rows():
    T, H, D, R = 6, 2, 64, 32
    for bits8 in (False, True):
        for inter in (False, True):
            k, v = randn(T, H, D, dtype="float32", seed=5), randn(T, H, D, dtype="float32", seed=6)
            k[1, 0, 50] = float("inf")                      # behind the rotated entries
            k[2, 1, 3] = float("nan")
            v[1, 1, 7] = float("-inf")
            v[3, 0, 9] = float("nan")
            v[4, 0] = 0.0
            v[4, 0, 5] = -0.0
            kc, vc = (Cache(1, 16, H, D, "float32", bits8, "rows") for _ in range(2))
            kg, vg, sg, pg, fg = k.cuda(), v.cuda(), torch.arange(T).cuda(), torch.arange(T).cuda(), freqs(R).cuda()
            args = (B.cache_heads(kg, None, kc.t, kc.s), B.cache_heads(vg, None, vc.t, vc.s))
            assert B.rmsnorm_rope_append(None, *args, sg, 1, 16, pg, T, D, R, fg, int(inter), 1.0, EPS, "float32", 0) == 0
            got_k, got_v = (c.t[0, :T].double().cpu() for c in (kc, vc))
            clean = torch.ones(T, H, dtype=torch.bool)
            clean[1, 0] = clean[2, 1] = False
            z, _ = ref.rope_fwd(k, None, torch.arange(T), freqs(R), inter, 1.0, EPS)
            if bits8:
                assert torch.isinf(kc.s[0, 1, 0]) and torch.isnan(kc.s[0, 2, 1]) and torch.isinf(vc.s[0, 1, 1])
                assert torch.isnan(got_k[1, 0, 50]) and (got_k[1, 0, :50] == 0).all()
                assert torch.isnan(vc.s[0, 3, 0]) and vc.s[0, 4, 0] == 2.0 ** -126 and (got_v[4, 0] == 0).all()
            else:
                # the infinity stays where it is
                assert torch.equal(torch.isfinite(got_k[1, 0]), torch.isfinite(k[1, 0]))
                assert torch.equal(vc.t[0, :T].cpu().view(torch.int32), v.view(torch.int32))
            assert torch.isfinite(got_k[clean]).all()


# --------------------------------------------------------------------------- #
# more of the products: every way of cutting them, special values, use
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K,layout", [(1300, 2000, 384, "dense"),     # pairs of blocks
                                          (5000, 4100, 256, "padded"),    # pairs, several tiles each
                                          (2500, 1300, 301, "dense"),     # 128 x 128, several tiles, rows off 16 bytes
                                          (150, 2600, 1024, "dense"),     # clusters that share K
                                          (70, 900, 2050, "shifted"), (20, 300, 16384, "dense"), (64, 20000, 256, "dense"),
                                          (40, 1, 700, "odd pitch"), (700, 1, 640, "dense"), (1, 5, 100000, "dense")])
def test_matmul_of_every_cut(M, N, K, layout, dtype):
    for group in (0, 128):
        a, lda, b, ldb, sa, sb = product_inputs(M, N, K, group, 7, layout)
        check_product(a, b, sa, sb, dtype, group, product(a, lda, b, ldb, sa, sb, dtype, group))


@pytest.mark.parametrize("M", [3, 100, 1400])
def test_matmul_output_of_any_alignment_and_scales_of_any_pitch(M):
    N, K = 1999, 260
    a, lda, b, ldb, sa, sb = product_inputs(M, N, K, 128, 21)
    wide_a, wide_b = torch.full((M, 7), float("nan"), device="cuda"), torch.full((sb.shape[0], 9), float("nan"), device="cuda")
    wide_a[:, 1:4], wide_b[:, 2:5] = sa, sb
    for dtype in DTYPES:
        for start, pitch in ((0, 2000), (1, 2001), (8, 2008)):
            buf = torch.full((start + M * pitch + 64,), 7.0, dtype=ref.TYPES[dtype], device="cuda")
            y = buf[start:start + M * pitch].view(M, pitch)
            assert B.rmsnorm_quant_matmul(a, lda, wide_a[:, 1:], 7, b, ldb, wide_b[:, 2:], 9, None, y, pitch, M, N, K, dtype,
                                          128) == 0
            check_product(a, b, sa, sb, dtype, 128, y)
            assert (buf[:start] == 7.0).all() and (buf[start + M * pitch:] == 7.0).all()


@pytest.mark.parametrize("M,K", [(5, 300), (5, 304), (90, 300), (90, 304), (1500, 384)])
def test_matmul_of_nan_and_infinite_scales_stays_in_their_rows_and_columns(M, K):
    N = 1400
    a, lda, b, ldb, sa, sb = product_inputs(M, N, K, 128, 31)
    sa[1, 1] = float("nan")                                 # a row
    sb[3, 0] = float("nan")                                 # 128 columns
    a.view(torch.uint8)[2, 7] = 0x7F                        # a NaN among the codes
    b.view(torch.uint8)[700, K - 1] = 0xFF
    sa[4] = 0.0
    y = product(a, lda, b, ldb, sa, sb, "float32", 128)[:, :N]
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[1] = bad[2] = True
    bad[:, 384:512] = True
    bad[:, 700] = True
    assert torch.equal(torch.isnan(y), bad)
    clean = ~bad
    assert (y[4][clean[4]] == 0).all()
    sb[3, 0], sa[1, 1] = 0.0, 0.0
    a.view(torch.uint8)[2, 7], b.view(torch.uint8)[700, K - 1] = 0, 0
    want, err = product_bound(a, b, sa, sb, 128)
    assert ((y.double() - want).abs() <= err + want.abs() * U)[clean].all()


def test_matmul_results_are_the_same_bits_every_time():
    for M, N, K in ((8, 4096, 4096), (150, 2600, 1024), (90, 512, 1031), (1300, 2000, 640)):
        a, lda, b, ldb, sa, sb = product_inputs(M, N, K, 128, 41)
        first = product(a, lda, b, ldb, sa, sb, "float32", 128)
        for _ in range(5):
            assert torch.equal(product(a, lda, b, ldb, sa, sb, "float32", 128), first)


def test_matmul_of_rows_past_32_bits():
    # codes 3 GiB apart, and an output of more than 2^32 bytes
    M, N, K, pitch = 40000, 300, 130, 80000
    buf = torch.zeros(M * pitch, dtype=torch.uint8, device="cuda")
    a = buf.view(F8).as_strided((M, K), (pitch, 1))
    rows = torch.tensor([0, 1, 26843, 26844, 39999])
    v, _ = codes(len(rows), K, 51)
    buf.view(M, pitch)[rows.cuda(), :K] = v.contiguous().view(torch.uint8)
    b, ldb = codes(N, K, 52)
    sa, sb = torch.ones(M, 2, device="cuda"), torch.ones(3, 2, device="cuda")
    y = torch.empty(M * 60000, dtype=torch.bfloat16, device="cuda")
    assert B.rmsnorm_quant_matmul(a, pitch, sa, 2, b, ldb, sb, 2, None, y, 60000, M, N, K, "bfloat16", 128) == 0
    got = y.view(M, 60000)[:, :N]
    want, err = product_bound(v, b, sa[:5], sb, 128)
    ref.assert_close(got[rows.cuda()], want, err + ref.rounding(want.abs() + err, torch.bfloat16), "y")
    assert (got[2:26843] == 0).all()


def everything(seed):
    """One call of each operator on inputs of a seed, as functions of the buffers; returns (calls, buffers)."""
    T, H, D = 33, 4, 64
    a, lda, b, ldb, sa, sb = product_inputs(T, 3 * H * D, 512, 128, seed)
    w = randn(300, 200, dtype="bfloat16", seed=seed).cuda()
    st = {"a": a, "sa": sa, "w": w, "y": torch.zeros(T, 3 * H * D, dtype=torch.bfloat16, device="cuda"),
          "wc": torch.zeros(300, 200, dtype=F8, device="cuda"), "ws": torch.zeros(3, 2, device="cuda"),
          "q": torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda"), "pos": torch.arange(T, device="cuda"),
          "slots": torch.arange(T, device="cuda") * 2 + 1, "kc": torch.zeros(5, 16, H, D, dtype=F8, device="cuda"),
          "vc": torch.zeros(5, 16, H, D, dtype=F8, device="cuda"), "ks": torch.zeros(5, 16, H, device="cuda"),
          "vs": torch.zeros(5, 16, H, device="cuda"), "f": freqs(D).cuda()}
    q, k, v = st["y"].view(T, 3, H, D).unbind(1)
    heads = (B.rope_heads([(q, None, st["q"])]), B.cache_heads(k, None, st["kc"], st["ks"]),
             B.cache_heads(v, None, st["vc"], st["vs"]))

    def calls(stream=None):
        assert B.rmsnorm_quant_weight(w, 200, st["wc"], 200, st["ws"], 2, 300, 200, "bfloat16", False, stream) == 0
        assert B.rmsnorm_quant_matmul(a, lda, sa, 4, b, ldb, sb, 4, None, st["y"], 3 * H * D, T, 3 * H * D, 512, "bfloat16",
                                      128, stream) == 0
        assert B.rmsnorm_rope_append(*heads, st["slots"], 5, 16, st["pos"], T, D, D, st["f"], 0, 1.0, EPS, "bfloat16", 0,
                                     stream) == 0
    return calls, st


OUTS = ("wc", "ws", "y", "q", "kc", "vc", "ks", "vs")


def same(st, want):
    return all(torch.equal(st[n].view(torch.uint8), want[n].view(torch.uint8)) for n in OUTS)


def test_captured_and_replayed_with_new_inputs():
    calls, st = everything(1)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        calls()
    for seed in (2, 3):
        eager, other = everything(seed)
        eager()
        st["a"].copy_(other["a"])
        st["sa"].copy_(other["sa"])
        st["w"].copy_(other["w"])
        # the weights of both are of different seeds: the product's stays that of seed 1
        for n in OUTS:
            st[n].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(st["wc"].view(torch.uint8), other["wc"].view(torch.uint8)) and torch.equal(st["ws"], other["ws"])
        _, _, b, _, _, sb = product_inputs(33, 768, 512, 128, 1)
        want, err = product_bound(st["a"], b, st["sa"], sb, 128)
        ref.assert_close(st["y"], want, err + ref.rounding(want.abs() + err, torch.bfloat16), "y")
        q, k, v = st["y"].cpu().view(33, 3, 4, 64).unbind(1)
        for rows, scales, heads, w in (("kc", "ks", k, None), ("vc", "vs", v, "values")):
            check_rows(st[rows].view(80, 4, 64)[st["slots"]], st[scales].view(80, 4)[st["slots"]], heads, w, st["pos"].cpu(), 64,
                       False, 1.0, False, "bfloat16")


def test_two_streams_at_once():
    made = [everything(s) for s in (5, 6)]
    for calls, _ in made:
        calls()
    torch.cuda.synchronize()
    want = [{n: st[n].clone() for n in OUTS} for _, st in made]
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(20):
        for (calls, st), s in zip(made, streams):
            with torch.cuda.stream(s):
                for n in OUTS:
                    st[n].zero_()
                calls()
    torch.cuda.synchronize()
    assert all(same(st, w) for (_, st), w in zip(made, want))


def test_calls_that_follow_each_other_see_each_others_results():
    # each kernel may start before the one before it has ended; the chain is the same as with waits
    calls, st = everything(9)
    calls()
    torch.cuda.synchronize()
    want = {n: st[n].clone() for n in OUTS}
    for _ in range(50):
        for n in OUTS:
            st[n].zero_()
        calls()
    torch.cuda.synchronize()
    assert same(st, want)


def test_append_of_more_values_than_keys():
    # heads of two kinds need not be as many
    T, Hk, Hv, D, size = 70, 2, 5, 64, 16
    k, v = randn(T, Hk, D, dtype="bfloat16", seed=3), randn(T, Hv, D, dtype="bfloat16", seed=4)
    pos, slots = torch.arange(T), torch.randperm(96, generator=torch.Generator().manual_seed(5))[:T]
    for bits8 in (False, True):
        kc, vc = Cache(6, size, Hk, D, "bfloat16", bits8, "rows"), Cache(6, size, Hv, D, "bfloat16", bits8, "heads first")
        kg, vg, sg, pg, fg = k.cuda(), v.cuda(), slots.cuda(), pos.cuda(), freqs(D).cuda()
        heads = B.cache_heads(kg, None, kc.t, kc.s), B.cache_heads(vg, None, vc.t, vc.s)
        assert B.rmsnorm_rope_append(None, *heads, sg, 6, size, pg, T, D, D, fg, 0, 1.0, EPS, "bfloat16", 0) == 0
        kc.untouched_but(sg)
        vc.untouched_but(sg)
        check_rows(*kc.rows(sg), k, None, pos, D, False, 1.0, False, "bfloat16")
        check_rows(*vc.rows(sg), v, "values", None, D, False, 1.0, False, "bfloat16")


@pytest.mark.parametrize("M,K", [(40, 512), (150, 515), (1300, 640)])
def test_matmul_of_rows_with_themselves(M, K):
    # one tensor on both sides, with scales of each kind
    a, lda = codes(M, K, 61)
    g = torch.Generator().manual_seed(62)
    n, k = -(-M // 128), -(-K // 128)
    sa, sb = torch.rand(M, k, generator=g).cuda() + 0.1, torch.rand(n, k, generator=g).cuda() + 0.1
    check_product(a, a, sa, sb, "float32", 128, product(a, lda, a, lda, sa, sb, "float32", 128))


def test_matmul_and_append_from_two_threads():
    import threading
    made = [everything(s) for s in (11, 12)]
    for calls, _ in made:
        calls()
    torch.cuda.synchronize()
    want = [{n: st[n].clone() for n in OUTS} for _, st in made]
    failed = []

    def work(calls, st):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    for n in OUTS:
                        st[n].zero_()
                    calls()
            stream.synchronize()
        except Exception as e:  # noqa: BLE001 -- reported by the assertion below
            failed.append(e)
    threads = [threading.Thread(target=work, args=m) for m in made]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and all(same(st, w) for (_, st), w in zip(made, want))


@pytest.mark.parametrize("M,N,side,pitch", [(130, 300, "a", (1 << 25) + 3), (20, 200, "b", (1 << 25) + 3),   # the loaders' rows
                                            (9, 130, "b", 1 << 25), (130, 300, "a", 1 << 25),                 # by TMA
                                            (1300, 2000, "a", 1 << 22)])                                      # pairs
def test_matmul_of_an_operand_of_more_than_2_to_the_32_bytes(M, N, side, pitch):
    K = 260
    a, lda, b, ldb, sa, sb = product_inputs(M, N, K, 128, 71, "padded")
    dense = a if side == "a" else b
    rows = dense.shape[0]
    assert (rows - 1) * pitch > 1 << 32
    far = torch.empty(rows * pitch, dtype=torch.uint8, device="cuda").as_strided((rows, K), (pitch, 1))
    far.copy_(dense.view(torch.uint8))
    far = far.view(F8)
    y = product(far, pitch, b, ldb, sa, sb, "float32", 128) if side == "a" \
        else product(a, lda, far, pitch, sa, sb, "float32", 128)
    check_product(a, b, sa, sb, "float32", 128, y)


@pytest.mark.parametrize("dtype", DTYPES)
def test_weight_scales_that_are_powers_of_two_stay(dtype):
    # largest entries of 7 * 2^k: 7 / 448 = 2^-6 exactly, and a step of the type above it the next power
    w = randn(5 * 128, 300, dtype=dtype, seed=95, scale=0.5).clamp(-1, 1)
    step = torch.finfo(w.dtype).eps * 4                     # between 4 and 8
    tops = [7.0, 7.0 + step, 3.5, 7.0 * 2.0 ** -3, 14.0 - 2 * step]
    for i, top in enumerate(tops):
        w[128 * i:128 * (i + 1)] *= 2.0 ** -3
        w[128 * i + 9, ::128] = -top
    c, s = quant_weight(w.cuda(), 300, *w.shape, dtype, True)
    want = torch.tensor([2.0 ** -6, 2.0 ** -5, 2.0 ** -7, 2.0 ** -9, 2.0 ** -5]).unsqueeze(1).expand(5, 3)
    assert torch.equal(s.cpu(), want)
    v = w.double() / spread(want, *w.shape)                 # exact: by powers of two
    assert torch.equal(c.cpu().view(torch.uint8), v.float().to(F8).view(torch.uint8))
