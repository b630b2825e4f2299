"""The torch front end of the serving operators on the GPU: views, opcheck, modules, a captured
step, and the way from the residual stream to a paged cache and back."""
import pytest
import torch

from rmsnorm_fwd_bwd_gb300 import binding as B
from rmsnorm_fwd_bwd_gb300 import fused, serving
from rmsnorm_fwd_bwd_gb300.autograd import DeviceError, check_device_error
from tests import fused_ref as ref
from tests.test_serving_gpu import check_product, check_rows, check_weight, freqs, product_inputs, randn

pytestmark = pytest.mark.gpu
EPS = 1e-6
U = ref.U


@pytest.fixture(autouse=True)
def _clean():
    B.rmsnorm_device_error(clear=True)
    yield
    assert B.rmsnorm_device_error(clear=True) == 0


def test_quant_weight_of_views():
    big = randn(260, 400, dtype="bfloat16", seed=1).cuda()
    for w in (big, big[:, 3:300], big.t(), big[::2], big[:0]):
        c, s = serving.quant_weight(w)
        if w.shape[0]:
            check_weight(w.contiguous(), c, s, False)
    assert c.shape == (0, 400) and s.shape == (0, 4)


@pytest.mark.parametrize("group", [0, 128])
def test_quant_matmul_of_views_and_leading_dimensions(group):
    a, _, b, _, sa, sb = product_inputs(24, 130, 384, group, 2)
    for codes, scales in ((a.view(4, 6, 384), sa.view(4, 6, -1)), (a[:0], sa[:0]), (a[5], sa[5]),
                          (a.view(4, 6, 384).transpose(0, 1), sa.view(4, 6, -1).transpose(0, 1))):
        y = serving.quant_matmul(codes, scales, b, sb, dtype=torch.float32)
        assert y.shape == (*codes.shape[:-1], 130)
        if codes.numel():
            y7 = torch.nn.functional.pad(y.reshape(-1, 130), (0, 1), value=7.0)
            check_product(codes.reshape(-1, 384), b, scales.reshape(-1, scales.shape[-1]), sb, "float32", group, y7)
    bias = randn(130, dtype="float16", seed=3).cuda()
    y = serving.quant_matmul(a, sa, b, sb, bias, torch.float16)
    check_product(a, b, sa, sb, "float16", group, torch.nn.functional.pad(y, (0, 1), value=7.0), bias)


def step_inputs(lead=(3, 7), Hq=6, Hk=2, D=64, dtype="bfloat16", seed=10):
    T = 1
    for n in lead:
        T *= n
    q, k, v = (randn(T, h, D, dtype=dtype, seed=seed + i) for i, h in enumerate((Hq, Hk, Hk)))
    return T, q, k, v


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("heads_first", [False, True])
def test_append_through_a_module_and_its_cache(bits8, heads_first):
    T, q, k, v = step_inputs()
    rope = fused.RMSNormRope(64, 32, dtype=torch.bfloat16, device="cuda")
    cache = serving.PagedCache(4, 10, 2, 64, bits8=bits8, heads_first=heads_first)
    slots, pos = torch.randperm(40)[:T].view(3, 7), torch.arange(T).view(3, 7) * 11
    before = cache.k._version
    with torch.no_grad():
        out = rope.append(*(t.cuda().view(3, 7, *t.shape[1:]) for t in (q, k, v)), pos.cuda(), slots.cuda(), cache)
    assert cache.k._version > before
    ones = torch.ones(64, dtype=torch.bfloat16)
    want, err = ref.rope_fwd(q, ones, pos.flatten(), freqs(32), False, 1.0, EPS)
    ref.assert_close(out.flatten(0, 1), want, err + ref.rounding(want.abs() + err, torch.bfloat16), "queries")
    at = slots.flatten().cuda()
    raw = lambda t: None if t is None else t[at // 10, at % 10]
    codes = lambda t: t.view(torch.uint8)[at // 10, at % 10].view(t.dtype) if bits8 else t[at // 10, at % 10]
    check_rows(codes(cache.k), raw(cache.k_scales), k, ones, pos.flatten(), 32, False, 1.0, False, "bfloat16")
    check_rows(codes(cache.v), raw(cache.v_scales), v, "values", None, 32, False, 1.0, False, "bfloat16")
    rk, rv = cache.rows(slots.cuda())
    assert rk.shape == rv.shape == (3, 7, 2, 64) and torch.isfinite(rk.float()).all()
    if not bits8:
        assert torch.equal(rv.flatten(0, 1).cpu(), v)


def test_append_of_nothing_and_without_queries():
    T, q, k, v = step_inputs()
    cache = serving.PagedCache(4, 10, 2, 64)
    inv = freqs(64).cuda()
    none = lambda t: t[:0].cuda()
    pos = torch.arange(T).cuda()
    out = serving.rms_norm_rope_append(none(q), none(k), none(v), None, None, pos[:0], pos[:0], inv, cache.k, cache.v)
    assert out.shape == (0, 6, 64) and (cache.k == 0).all()
    assert serving.rms_norm_rope_append(None, k.cuda(), None, None, None, pos, pos, inv, cache.k) is None
    assert (cache.v == 0).all() and (cache.k.view(40, 2, 64)[:T] != 0).any()


def test_a_slot_behind_the_last_is_reported():
    T, q, k, v = step_inputs()
    cache = serving.PagedCache(2, 10, 2, 64)
    pos = torch.arange(T).cuda()
    serving.rms_norm_rope_append(None, k.cuda(), v.cuda(), None, None, pos, pos, freqs(64).cuda(), cache.k, cache.v)
    with pytest.raises(DeviceError):
        check_device_error()


def test_append_wants_no_gradient():
    T, q, k, v = step_inputs()
    cache = serving.PagedCache(4, 10, 2, 64)
    rope = fused.RMSNormRope(64, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(T).cuda()
    with pytest.raises(ValueError, match="not differentiable"):
        rope.append(q.cuda(), k.cuda(), v.cuda(), pos, pos, cache)


def test_ops_pass_opcheck_and_compile_traces_them():
    tests = ("test_schema", "test_faketensor")
    w = randn(130, 200, dtype="float32", seed=4).cuda()
    torch.library.opcheck(torch.ops.rmsnorm_gb300.quant_weight, (w, False), test_utils=tests)
    a, _, b, _, sa, sb = product_inputs(5, 130, 200, 128, 5)
    y = torch.ops.rmsnorm_gb300.quant_matmul(a, sa, b, sb, None, torch.bfloat16)
    assert torch.equal(y, serving.quant_matmul(a, sa, b, sb))
    T, q, k, v = step_inputs()
    pos, inv = torch.arange(T).cuda(), freqs(64).cuda()
    caches = [serving.PagedCache(4, 10, 2, 64) for _ in range(2)]
    args = (q.cuda(), k.cuda(), v.cuda(), None, None, pos, pos, inv)
    torch.library.opcheck(torch.ops.rmsnorm_gb300.rope_append,
                          (*args, caches[0].k, caches[0].v, None, None, False, 1.0, EPS, False), test_utils=tests)
    one = torch.ops.rmsnorm_gb300.rope_append(*args, caches[0].k, caches[0].v, None, None, False, 1.0, EPS, False)
    two = serving.rms_norm_rope_append(*args, caches[1].k, caches[1].v)
    assert torch.equal(one, two) and torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)


def test_quant_linear_from_linear_moves_and_saves():
    lin = torch.nn.Linear(300, 130, device="cuda", dtype=torch.bfloat16)
    q = serving.QuantLinear.from_linear(lin)
    x = randn(9, 300, dtype="bfloat16", seed=6).cuda()
    codes, scales, _ = fused.rms_norm_quant(x, torch.ones(300, dtype=torch.bfloat16, device="cuda"), group=128)
    y = q(codes, scales)
    other = serving.QuantLinear(300, 130, True, device="cuda")
    other.load_state_dict(q.state_dict())
    assert torch.equal(other(codes, scales), y) and y.dtype == torch.bfloat16
    moved = other.cpu().cuda().half()
    assert moved.weight.dtype == torch.float8_e4m3fn and moved.weight_scales.dtype == torch.float32
    assert torch.equal(moved.weight_scales, q.weight_scales)
    half = moved(codes, scales)
    assert half.dtype == torch.float16
    # the bias in half, and one rounding each
    assert (half.float() - y.float()).abs().max() <= y.float().abs().max() * 2.0 ** -7


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("bits8", [False, True])
def test_from_the_residual_stream_to_the_cache_and_an_attention(group, bits8):
    """A prompt and three decoding steps of one layer's way into attention: norm with an 8-bit output,
    the projection, head norm, rotation and cache, captured for the steps, against 64 bits."""
    N, Hq, Hk, D, size = 512, 6, 2, 64, 5
    width = (Hq + 2 * Hk) * D
    torch.manual_seed(3)
    lin = torch.nn.Linear(N, width, bias=True, device="cuda", dtype=torch.bfloat16)
    norm_w = (1 + 0.1 * torch.randn(N)).to(torch.bfloat16).cuda()
    layer = serving.RMSNormQuantLinear(norm_w, serving.QuantLinear.from_linear(lin), EPS, group=group)
    rope = fused.RMSNormRope(D, dtype=torch.bfloat16, device="cuda")
    cache = serving.PagedCache(8, size, Hk, D, bits8=bits8)
    order = torch.randperm(8)

    def step(x, res, pos, slots):
        with torch.no_grad():
            y, h = layer(x, res)
            q, k, v = y.split([Hq * D, Hk * D, Hk * D], dim=-1)
            heads = [t.unflatten(-1, (-1, D)) for t in (q, k, v)]
            return rope.append(*heads, pos, slots, cache), h, y

    total = 30
    x, res = randn(total, N, dtype="bfloat16", seed=7).cuda(), randn(total, N, dtype="bfloat16", seed=8).cuda()
    pos = torch.arange(total)
    slots = (order[pos // size] * size + pos % size).cuda()
    prompt = total - 3
    queries, hs, ys = ([t] for t in step(x[:prompt], res[:prompt], pos[:prompt].cuda(), slots[:prompt]))
    # one decoding step, captured, and replayed for the three tokens
    bx, bres = x[:1].clone(), res[:1].clone()
    bpos, bslot = (torch.full((1,), n, dtype=torch.int64, device="cuda") for n in (0, -1))
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(bx, bres, bpos, bslot)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = step(bx, bres, bpos, bslot)
    for t in range(prompt, total):
        bx.copy_(x[t:t + 1])
        bres.copy_(res[t:t + 1])
        bpos.fill_(t)
        bslot.copy_(slots[t:t + 1])
        graph.replay()
        for kept, got in zip((queries, hs, ys), out):
            kept.append(got.clone())
    queries, h, y = (torch.cat(t) for t in (queries, hs, ys))

    # the projection of the codes in 64 bits
    codes, scales, h2 = fused.rms_norm_quant(x, norm_w, EPS, residual=res, group=group)
    assert torch.equal(h, h2)
    check_product(codes, layer.linear.weight, scales, layer.linear.weight_scales, "bfloat16", group,
                  torch.nn.functional.pad(y, (0, 1), value=7.0), layer.linear.bias)
    # the cache's rows from those projections
    q, k, v = (t.unflatten(-1, (-1, D)).cpu() for t in y.split([Hq * D, Hk * D, Hk * D], dim=-1))
    ones = torch.ones(D, dtype=torch.bfloat16)
    want, err = ref.rope_fwd(q, ones, pos, freqs(D), False, 1.0, EPS)
    ref.assert_close(queries, want, err + ref.rounding(want.abs() + err, torch.bfloat16), "queries")
    page, row = slots // size, slots % size
    take = lambda t: t.view(torch.uint8)[page, row].view(t.dtype) if bits8 else t[page, row]
    for rows, s, heads, w in ((cache.k, cache.k_scales, k, ones), (cache.v, cache.v_scales, v, "values")):
        check_rows(take(rows), None if s is None else s[page, row], heads, w, pos, D, False, 1.0, False, "bfloat16")
    # and an attention reads them
    rk, rv = (t.double().repeat_interleave(Hq // Hk, 1) for t in cache.rows(slots))
    att = torch.einsum("qhd,khd->hqk", queries.double(), rk) * D ** -0.5
    att = att.masked_fill(torch.ones(total, total, device="cuda").triu(1).bool(), float("-inf")).softmax(-1)
    assert torch.isfinite(torch.einsum("hqk,khd->qhd", att, rv)).all()


@pytest.mark.parametrize("group", [0, 128])
def test_the_product_passes_opcheck_and_compiles_without_breaks(group):
    a, _, b, _, sa, sb = product_inputs(24, 130, 384, group, 90)
    a, b = a.contiguous(), b.contiguous()
    bias = randn(130, dtype="bfloat16", seed=91).cuda()
    before = [t.view(torch.uint8).clone() for t in (a, sa, b, sb, bias)]
    for extra in (None, bias):
        # (the check of the schema multiplies its tensors, which torch does not do in e4m3: by hand below)
        torch.library.opcheck(torch.ops.rmsnorm_gb300.quant_matmul, (a, sa, b, sb, extra, torch.bfloat16),
                              test_utils=("test_faketensor",))
    assert all(torch.equal(t.view(torch.uint8), u) for t, u in zip((a, sa, b, sb, bias), before))

    def f(codes, scales):
        return serving.quant_matmul(codes, scales, b, sb, bias) + 1
    compiled = torch.compile(f, backend="aot_eager", fullgraph=True)
    assert torch.equal(compiled(a, sa), f(a, sa))
    lead = a.view(4, 6, 384), sa.view(4, 6, -1)
    assert torch.equal(compiled(*lead), f(*lead))


def test_a_weight_compiles_without_breaks():
    w = randn(130, 200, dtype="bfloat16", seed=92).cuda()

    def f(w):
        codes, scales = serving.quant_weight(w * 2)
        return codes.view(torch.uint8), scales + 1
    for got, want in zip(torch.compile(f, backend="aot_eager", fullgraph=True)(w), f(w)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("heads_first", [False, True])
def test_an_append_through_modules_compiles_without_breaks(bits8, heads_first):
    N, Hq, Hk, D = 256, 4, 2, 64
    torch.manual_seed(4)
    lin = serving.QuantLinear.from_linear(torch.nn.Linear(N, (Hq + 2 * Hk) * D, device="cuda", dtype=torch.bfloat16))
    layer = serving.RMSNormQuantLinear(torch.ones(N, dtype=torch.bfloat16, device="cuda"), lin)
    rope = fused.RMSNormRope(D, 32, dtype=torch.bfloat16, device="cuda")
    caches = [serving.PagedCache(4, 10, Hk, D, bits8=bits8, heads_first=heads_first) for _ in range(2)]

    def step(x, pos, slots, cache):
        y, h = layer(x)
        q, k, v = (t.unflatten(-1, (-1, D)) for t in y.split([Hq * D, Hk * D, Hk * D], dim=-1))
        return rope.append(q, k, v, pos, slots, cache) + 1, h
    compiled = torch.compile(step, backend="aot_eager", fullgraph=True)
    x, pos = randn(7, N, dtype="bfloat16", seed=93).cuda(), torch.arange(7).cuda() * 3
    with torch.no_grad():
        for shift in (0, 9):                                # the second call into what the first has left
            slots = torch.tensor([3, -1, 39, 12, 0, 11, 25]).cuda()
            slots = torch.where(slots < 0, slots, (slots + shift) % 40)
            want, got = (f(x + shift, pos, slots, c) for f, c in ((step, caches[0]), (compiled, caches[1])))
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    one, two = caches
    bits = lambda t: t.view(torch.uint8) if bits8 else t
    assert torch.equal(bits(one.k), bits(two.k)) and torch.equal(bits(one.v), bits(two.v))
    assert (bits(one.k) != 0).any()
    if bits8:
        assert torch.equal(one.k_scales, two.k_scales) and torch.equal(one.v_scales, two.v_scales)


def test_rows_of_slots_without_one_are_zeros_on_the_gpu():
    T, q, k, v = step_inputs()
    cache = serving.PagedCache(4, 10, 2, 64)
    pos = torch.arange(T).cuda()
    slots = torch.where(pos % 3 == 1, -1, pos + 40 - T)     # the last row holds a token
    serving.rms_norm_rope_append(None, k.cuda(), v.cuda(), None, None, pos, slots, freqs(64).cuda(), cache.k, cache.v)
    rk, rv = cache.rows(torch.cat([slots, torch.tensor([40, 1 << 40]).cuda()]))
    stored = torch.cat([slots >= 0, torch.zeros(2, dtype=torch.bool, device="cuda")])
    assert torch.equal(rv[stored].cpu(), v[(slots >= 0).cpu()]) and (rk[~stored] == 0).all() and (rv[~stored] == 0).all()
