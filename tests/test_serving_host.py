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


def append(q=True, v=True, **kw):
    qs = dict(x=0x1000000, x_token=256, x_head=64, gamma=0x1100000, y=0x1200000, y_token=256, y_head=64, heads=4)
    ks = dict(x=0x2000000, x_token=128, x_head=64, gamma=0x2100000, rows=0x3000000, page=2048, row=128, head=64, scales=None,
              scale_page=0, scale_row=0, scale_head=0, heads=2)
    vs = dict(ks, x=0x4000000, gamma=None, rows=0x5000000)
    a = dict(slots=0x6000000, pages=10, page_size=16, positions=0x6100000, T=4, D=64, rotary_dim=64, inv_freq=0x6200000,
             interleaved=0, mscale=1.0, eps=1e-6, dtype=2, offset=0, stream=0)
    for name, value in kw.items():
        kind, _, field = name.partition("_")
        (qs if kind == "q" else ks if kind == "k" else vs if kind == "v" else a)[field if kind in "qkv" else name] = value
    keep = [(B.RopeHeads * 1)(B.RopeHeads(**qs)), (B.CacheHeads * 1)(B.CacheHeads(**ks)), (B.CacheHeads * 1)(B.CacheHeads(**vs))]
    return B.rmsnorm_rope_append(keep[0] if q else None, keep[1], keep[2] if v else None, **a)


SCALES = dict(k_scales=0x7000000, k_scale_page=32, k_scale_row=2, k_scale_head=1)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=4)), (ARG, dict(offset=2)), (SHAPE, dict(D=513)), (SHAPE, dict(rotary_dim=0)), (SHAPE, dict(rotary_dim=3)),
    (SHAPE, dict(rotary_dim=66)), (EPS, dict(eps=0.0)), (ARG, dict(interleaved=2)), (ARG, dict(mscale=float("inf"))),
    (SHAPE, dict(T=-1)), (SHAPE, dict(pages=0)), (SHAPE, dict(page_size=0)), (SHAPE, dict(page_size=1 << 31)),
    (SHAPE, dict(pages=1 << 45)), (SHAPE, dict(q_heads=0)), (SHAPE, dict(k_heads=0)), (SHAPE, dict(v_heads=65537)),
    (SHAPE, dict(q_x_token=63)), (SHAPE, dict(q_y_head=63)), (SHAPE, dict(k_x_head=-64)), (SHAPE, dict(k_row=127)),
    (SHAPE, dict(k_head=63)), (SHAPE, dict(k_page=2047)), (SHAPE, dict(v_page=0)), (SHAPE, dict(v_row=-128)),
    (SHAPE, dict(k_page=1 << 60)), (SHAPE, dict(SCALES, k_scale_row=1)), (SHAPE, dict(SCALES, k_scale_page=31)),
    (ARG, dict(v_gamma=0x7000000)), (OK, dict(T=0, q_x=None, k_x=None, k_rows=None, slots=None, positions=None)),
    (NULL, dict(q_x=None)), (NULL, dict(q_y=None)), (NULL, dict(k_x=None)), (NULL, dict(k_rows=None)), (NULL, dict(v_x=None)),
    (NULL, dict(slots=None)), (NULL, dict(positions=None)), (NULL, dict(inv_freq=None)), (ALIGN, dict(q_x=0x1000001)),
    (ALIGN, dict(k_rows=0x3000001)), (ALIGN, dict(SCALES, k_scales=0x7000002)), (ALIGN, dict(slots=0x6000004)),
    (ALIGN, dict(positions=0x6100004)), (ALIGN, dict(k_gamma=0x2100001)),
    (ARG, dict(k_rows=0x2000000)), (ARG, dict(k_rows=0x4000000 + 1022)), (ARG, dict(v_rows=0x3000000)),
    (ARG, dict(v_rows=0x3000000 + 64)), (ARG, dict(v_rows=0x3000000 + 2 * 2048 * 10 - 2)), (ARG, dict(k_rows=0x1200000)),
    (ARG, dict(k_rows=0x1100000)), (ARG, dict(k_rows=0x6000000)), (ARG, dict(SCALES, k_scales=0x3000000)),
    (ARG, dict(SCALES, k_scales=0x2000000)), (ARG, dict(q_y=0x2000000)), (ARG, dict(q_y=0x1000000, q_y_token=512)),
    (ARG, dict(q_y=0x1100000)), (ARG, dict(SCALES, v_scales=0x7000000, v_scale_page=32, v_scale_row=2, v_scale_head=1)),
    # the halves of one tensor must have its strides, and rows of the other must fit between
    (ARG, dict(v_rows=0x3000000 + 2 * 2048)), (ARG, dict(k_page=4096, v_page=2048, v_rows=0x3000000 + 2 * 2048)),
    (ARG, dict(k_page=4096, v_page=4096, v_rows=0x3000000 + 2 * 2048 - 2)),
])
def test_append_refusals(want, kw):
    assert append(**kw) == want


@pytest.mark.parametrize("y,strides", [(0x2000000 + 2, {}), (0x2000000 + 128, {}), (0x1000000 + 128, {}), (0x1000000 + 2, {}),
                                       (0x1000000 - 2, {}), (0x4000000 - 2, {}), (0x4000000 + 510, {}),
                                       (0x2000000 - 4 * 256 * 2 + 2, {}), (0x1000000 + 2, dict(T=1, q_heads=1))])
def test_append_refuses_queries_written_on_parts_of_heads(y, strides):
    assert append(q_y=y, **strides) == ARG


def test_append_takes_queries_written_between_the_heads_of_their_rows():
    # (all that is wrong with these calls is that there are no positions)
    base = 0x1000000

    def rows(token, head, at, **kw):
        """q, k and v at `at` elements of one tensor."""
        a = {f"{n}_{f}": x for n, first in zip("qkv", at)
             for f, x in (("x", base + 2 * first), ("x_token", token), ("x_head", head))}
        return append(**dict(a, q_y=base + 2 * at[0], q_y_token=token, q_y_head=head, positions=None, **kw))
    assert rows(512, 64, (0, 256, 384)) == NULL                                   # a fused projection's rows, in place
    assert rows(512 + 40, 64, (0, 256, 384)) == NULL
    assert rows(4 * 192, 192, (0, 64, 128), k_heads=4, v_heads=4, k_row=256, v_row=256, k_page=4096, v_page=4096) == NULL
    assert rows(4 * 192 + 24, 192, (0, 64, 128), k_heads=4, v_heads=4, k_row=256, v_row=256, k_page=4096, v_page=4096) == NULL
    assert rows(128, 4 * 128, (0, 64, 64 + 512)) == NULL                          # heads outside of tokens
    assert rows(512, 64, (0, 192, 384)) == ARG
    assert rows(4 * 192, 192, (0, 65, 128), k_heads=4, v_heads=4, k_row=256, v_row=256, k_page=4096, v_page=4096) == NULL
    assert rows(4 * 192, 192, (0, 63, 128), k_heads=4, v_heads=4, k_row=256, v_row=256, k_page=4096, v_page=4096) == ARG
    # the output in a gap of the queries' own rows, and behind the last row
    assert append(q_x=base, q_x_token=1024, q_y=base + 512, q_y_token=1024, positions=None) == NULL
    assert append(q_x=base, q_x_token=1024, q_y=base + 510, q_y_token=1024, positions=None) == ARG
    assert append(q_y=0x1000000 + 4 * 256 * 2, positions=None) == NULL
    assert append(q_y=0x1000000 + 4 * 256 * 2 - 2, positions=None) == ARG


def test_append_refuses_every_output_of_the_queries_that_meets_other_heads():
    import random
    rng, D, base = random.Random(5), 8, 0x1000000

    def lies(p, token, head, heads, T):
        return {p + 2 * (t * token + h * head + d) for t in range(T) for h in range(heads) for d in range(D)}
    met = 0
    for _ in range(4000):
        T, Hq, Hk = rng.randint(1, 5), rng.randint(1, 4), rng.randint(1, 3)
        tok = D * rng.randint(1, 14) + rng.choice([0, 0, 1, 4])

        def strides():
            return rng.choice([(tok, rng.choice([D, 2 * D, 3 * D, D + 1])), (rng.choice([D, 2 * D]), D * T * 2 + rng.choice([0, 3])),
                               (D * rng.randint(1, 14), rng.choice([D, 3 * D]))])
        sy = strides()
        sx, sk = (sy if rng.random() < 0.5 else strides() for _ in range(2))
        y = base
        x, k = (base + 2 * rng.choice([0, rng.randint(-150, 150), D * rng.randint(-20, 20)]) for _ in range(2))
        st = append(v=False, T=T, D=D, rotary_dim=D, q_x=x, q_x_token=sx[0], q_x_head=sx[1], q_heads=Hq, q_y=y, q_y_token=sy[0],
                    q_y_head=sy[1], k_x=k, k_x_token=sk[0], k_x_head=sk[1], k_heads=Hk, k_head=D, k_row=D * Hk,
                    k_page=D * Hk * 16, positions=None)
        if st == SHAPE:
            continue
        assert st in (ARG, NULL)
        out = lies(y, *sy, Hq, T)
        in_place = x == y and (T == 1 or sx[0] == sy[0]) and (Hq == 1 or sx[1] == sy[1])
        if (not in_place and out & lies(x, *sx, Hq, T)) or out & lies(k, *sk, Hk, T):
            met += 1
            assert st == ARG, (T, Hq, Hk, sy, sx, sk, x - y, k - y)
    assert met > 500


def test_only_debug_builds_let_a_product_give_up():
    assert B.rmsnorm_selftest_matmul_gives_up(0) == B.rmsnorm_selftest_matmul_gives_up(-1) == 7   # RMSNORM_ERR_UNSUPPORTED


def test_append_wants_keys():
    assert B.rmsnorm_rope_append(None, None, None, 0x1000, 1, 1, 0x2000, 1, 64, 64, 0x3000, 0, 1.0, 1e-6, 2, 0, 0) == NULL


def test_cache_heads_checks_its_tensors():
    import torch
    x, rows = torch.empty(2, 2, 8), torch.empty(3, 4, 2, 8)
    with pytest.raises(ValueError):
        B.cache_heads(x, None, rows[0])
    with pytest.raises(ValueError):
        B.cache_heads(x, None, rows.transpose(2, 3))
    with pytest.raises(ValueError):
        B.cache_heads(x, None, rows, torch.empty(3, 4))


# --------------------------------------------------------------------------- #
# the torch front end's checks, before the library is called
# --------------------------------------------------------------------------- #
def test_quant_weight_front_checks():
    import torch
    from rmsnorm_fwd_bwd_gb300 import serving
    for w in (torch.zeros(4), torch.zeros(2, 3, 4), torch.zeros(3, 0)):
        with pytest.raises(ValueError):
            serving.quant_weight(w)


def test_quant_matmul_front_checks():
    import torch
    from rmsnorm_fwd_bwd_gb300 import serving
    f8 = torch.float8_e4m3fn
    good = dict(codes=torch.zeros(3, 200).to(f8), scales=torch.ones(3, 2), weight=torch.zeros(130, 200).to(f8),
                weight_scales=torch.ones(2, 2), bias=torch.zeros(130, dtype=torch.bfloat16))
    for bad in (dict(codes=torch.zeros(3, 200)), dict(weight=torch.zeros(130, 200)), dict(scales=torch.ones(3, 2).double()),
                dict(weight_scales=torch.ones(2, 2).half()), dict(codes=torch.zeros(3, 199).to(f8)), dict(scales=torch.ones(3, 3)),
                dict(scales=torch.ones(2, 2)), dict(scales=torch.ones(2)), dict(weight_scales=torch.ones(2, 1)),
                dict(weight_scales=torch.ones(1, 2)), dict(bias=torch.zeros(130)), dict(bias=torch.zeros(129, dtype=torch.bfloat16)),
                dict(weight=torch.zeros(200).to(f8)), dict(scales=torch.ones(3, 2, device="meta"))):
        with pytest.raises(ValueError):
            serving.quant_matmul(**dict(good, **bad))


def test_quant_matmul_wants_no_gradient(monkeypatch):
    import torch
    from rmsnorm_fwd_bwd_gb300 import serving
    monkeypatch.setattr(serving, "_quant_matmul_run", lambda codes, scales, weight, *rest: torch.zeros(3, weight.shape[0]))
    f8 = torch.float8_e4m3fn
    good = dict(codes=torch.zeros(3, 200).to(f8), scales=torch.ones(3, 2), weight=torch.zeros(130, 200).to(f8),
                weight_scales=torch.ones(2, 2), bias=torch.zeros(130, dtype=torch.bfloat16))
    assert serving.quant_matmul(**good).shape == (3, 130)
    for name in good:
        bad = dict(good, **{name: good[name].clone().requires_grad_()})
        with pytest.raises(ValueError, match="not differentiable"):
            serving.quant_matmul(**bad)
        with torch.no_grad():
            assert not serving.quant_matmul(**bad).requires_grad


def test_rope_append_front_checks():
    import torch
    from rmsnorm_fwd_bwd_gb300 import serving
    f8 = torch.float8_e4m3fn
    pos = torch.arange(3)
    good = dict(q=torch.zeros(3, 4, 8), k=torch.zeros(3, 2, 8), v=torch.zeros(3, 2, 8), q_weight=torch.ones(8),
                k_weight=torch.ones(8), positions=pos, slots=pos, inv_freq=torch.ones(4, dtype=torch.float64),
                k_cache=torch.zeros(2, 5, 2, 8), v_cache=torch.zeros(2, 5, 2, 8), k_scales=None, v_scales=None)
    for bad in (dict(q=torch.zeros(2, 4, 8)), dict(q=torch.zeros(3, 4, 6)), dict(q=torch.zeros(3, 0, 8)), dict(q=torch.zeros(3, 4, 8).half()),
                dict(v=torch.zeros(3, 2, 6)), dict(v=torch.zeros(3, 2, 8).half()), dict(q_weight=torch.ones(7)),
                dict(k_weight=torch.ones(8).half()), dict(q=None), dict(v=None), dict(v_cache=None),
                dict(positions=pos.int()), dict(positions=pos[:2]), dict(slots=pos.int()), dict(slots=pos[:2]),
                dict(inv_freq=torch.ones(4)), dict(k_cache=torch.zeros(2, 5, 3, 8)), dict(k_cache=torch.zeros(2, 5, 2, 7)),
                dict(k_cache=torch.zeros(10, 2, 8)), dict(k_cache=torch.zeros(2, 5, 8, 2).transpose(2, 3)),
                dict(k_cache=torch.zeros(2, 5, 2, 8).half()), dict(k_cache=torch.zeros(0, 5, 2, 8)),
                dict(k_scales=torch.ones(2, 5, 2)), dict(v_cache=torch.zeros(3, 5, 2, 8)),
                dict(k_cache=torch.zeros(2, 5, 2, 8).to(f8)),
                dict(k_cache=torch.zeros(2, 5, 2, 8).to(f8), k_scales=torch.ones(2, 5, 2).half()),
                dict(k_cache=torch.zeros(2, 5, 2, 8).to(f8), k_scales=torch.ones(2, 5, 1)),
                dict(k=torch.zeros(3, 2, 8, requires_grad=True)), dict(k_weight=torch.ones(8, requires_grad=True)),
                dict(slots=torch.arange(3, device="meta"))):
        with pytest.raises(ValueError):
            serving.rms_norm_rope_append(**dict(good, **bad))


def test_quant_linear_keeps_codes_and_scales_through_changes_of_type():
    import torch
    from rmsnorm_fwd_bwd_gb300 import serving
    lin = serving.QuantLinear(200, 130, True, device="cpu")
    lin.weight.view(torch.uint8).copy_(torch.arange(130 * 200).remainder(120).view(130, 200))
    lin.weight_scales.copy_(torch.rand(2, 2))
    before = lin.weight.clone().view(torch.uint8), lin.weight_scales.clone()
    lin.half()
    assert lin.out_dtype == torch.float16 and lin.bias.dtype == torch.float16
    assert torch.equal(lin.weight.view(torch.uint8), before[0]) and torch.equal(lin.weight_scales, before[1])
    assert set(lin.state_dict()) == {"weight", "weight_scales", "bias"}
    with pytest.raises(ValueError):
        serving.RMSNormQuantLinear(torch.ones(200), lin, group=64)


@pytest.mark.parametrize("bias", [False, True])
def test_quant_linear_keeps_codes_and_scales_through_type(bias):
    # Module.type converts every tensor, whole numbers too
    import torch
    from rmsnorm_fwd_bwd_gb300 import serving
    for dtype in (torch.float16, torch.float32, torch.bfloat16):
        lin = serving.QuantLinear(201, 130, bias, device="cpu")
        lin.weight.view(torch.uint8).copy_(torch.arange(130 * 201).remainder(120).view(130, 201))
        lin.weight_scales.copy_(torch.rand(2, 2))
        before = lin.weight.clone().view(torch.uint8), lin.weight_scales.clone()
        lin.type(dtype)
        assert lin.weight.dtype == serving.CODES and lin.weight.shape == (130, 201)
        assert torch.equal(lin.weight.view(torch.uint8), before[0])
        assert lin.weight_scales.dtype == torch.float32 and torch.equal(lin.weight_scales, before[1])
        assert lin.out_dtype == dtype and (lin.bias is None or lin.bias.dtype == dtype)


def test_quant_linear_without_a_bias_changes_its_outputs_type():
    import torch
    from rmsnorm_fwd_bwd_gb300 import serving
    lin = torch.nn.Sequential(serving.QuantLinear(200, 130, device="cpu"))
    assert lin[0].out_dtype == torch.bfloat16
    for dtype in (torch.float16, torch.float32):
        assert lin.to(dtype)[0].out_dtype == dtype
        assert lin[0].weight_scales.dtype == torch.float32 and lin[0].weight.dtype == serving.CODES
    assert lin.to("meta")[0].out_dtype == torch.float32 and lin[0].weight.device.type == "meta"
    assert lin.to_empty(device="cpu").share_memory()[0].weight.device.type == "cpu"


def test_quant_linear_scales_are_float32_whatever_the_default_is():
    import torch
    from rmsnorm_fwd_bwd_gb300 import serving
    torch.set_default_dtype(torch.bfloat16)
    try:
        lin, cache = serving.QuantLinear(200, 130, device="cpu"), serving.PagedCache(3, 5, 2, 8, bits8=True, device="cpu")
    finally:
        torch.set_default_dtype(torch.float32)
    assert lin.weight_scales.dtype == torch.float32 and cache.k_scales.dtype == torch.float32


def test_paged_cache_shapes():
    import torch
    from rmsnorm_fwd_bwd_gb300 import serving
    for first in (False, True):
        c = serving.PagedCache(3, 5, 2, 8, bits8=True, heads_first=first, device="cpu")
        assert c.k.shape == c.v.shape == (3, 5, 2, 8) and c.k_scales.shape == c.v_scales.shape == (3, 5, 2)
        assert c.k.stride() == ((80, 8, 40, 1) if first else (80, 16, 8, 1))
        c.k.view(torch.uint8)[1, 2] = 0x38                  # 1.0
        c.k_scales[1, 2] = 3.0
        k, v = c.rows(torch.tensor([7, 0]))
        assert (k[0] == 3.0).all() and (k[1] == 0.0).all() and (v == 0.0).all()
    c = serving.PagedCache(3, 5, 2, 8, dtype=torch.float16, device="cpu")
    assert c.k.dtype == torch.float16 and c.k_scales is None


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("first", [False, True])
def test_paged_cache_rows_of_slots_without_one_are_zeros(bits8, first):
    import torch
    from rmsnorm_fwd_bwd_gb300 import serving
    c = serving.PagedCache(3, 5, 2, 8, dtype=torch.float32, bits8=bits8, heads_first=first, device="cpu")
    for cache, scales, value in ((c.k, c.k_scales, 1.0), (c.v, c.v_scales, 2.0)):
        if bits8:
            cache.view(torch.uint8).fill_(0x38)             # 1.0
            scales.fill_(value)
            scales[2, 4] = float("nan")
        else:
            cache.fill_(value)
            cache[2, 4] = float("nan")
    slots = torch.tensor([[0, -1, 13], [15, -(1 << 40), 1 << 40]])
    for rows, value in zip(c.rows(slots), (1.0, 2.0)):
        assert rows.shape == (2, 3, 2, 8)
        assert (rows[0, 0] == value).all() and (rows[0, 2] == value).all()
        assert (rows[0, 1] == 0.0).all() and (rows[1] == 0.0).all()
    k, _ = c.rows(torch.tensor(-1))
    assert k.shape == (2, 8) and (k == 0.0).all()
    assert torch.isnan(c.rows(torch.tensor([14]))[0]).all() and c.rows(torch.zeros(0, dtype=torch.int64))[0].shape == (0, 2, 8)
