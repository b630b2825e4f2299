"""The torch front end of the fused operators on the GPU: gradients through autograd,
views, opcheck and tracing, modules, and a transformer block that runs them together."""
import pytest
import torch

from rmsnorm_fwd_bwd_gb300 import fused
from rmsnorm_fwd_bwd_gb300.autograd import rms_norm
from tests import fused_ref as ref
from tests.test_fused_gpu import (check_add_bwd, check_add_fwd, check_quant, check_rope, check_rope_bwd, freqs, randn,
                                  weight)

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def leaf(t):
    return t.cuda().requires_grad_(True)


@pytest.mark.parametrize("dtype,p,offset", [("bfloat16", 0.0, False), ("float16", 0.2, True), ("float32", 0.2, False)])
def test_rms_norm_add_gradients(dtype, p, offset):
    B, S, N = 3, 20, 320
    x, res, w = randn(B * S, N, dtype=dtype, seed=1), randn(B * S, N, dtype=dtype, seed=2), weight(N, dtype, offset)
    dy, dh = randn(B * S, N, dtype=dtype, seed=3), randn(B * S, N, dtype=dtype, seed=4)
    xt, rt, wt = leaf(x.view(B, S, N)), leaf(res.view(B, S, N)), leaf(w)
    rng = fused.dropout_state(123, 5)
    before = dict(fused.CALLS)
    y, h = fused.rms_norm_add(xt, rt, wt, EPS, offset, p, rng if p else None)
    rng[1] += 1                                         # the backward still drops what the forward dropped
    torch.autograd.backward([y, h], [dy.view(B, S, N).cuda(), dh.view(B, S, N).cuda()])
    assert fused.CALLS["add_forward"] == before["add_forward"] + 1
    assert fused.CALLS["add_backward"] == before["add_backward"] + 1
    keep = ref.kept(123, 5, B * S, N, p) if p else None
    hc = h.detach().cpu().view(B * S, N)
    r = ref.norm(hc, w, EPS)[1].squeeze(-1).float()
    check_add_fwd(x, res, w, dtype, y.detach().cpu().view(B * S, N), hc, r, offset, p, 123, 5)
    # the kernel's own r differs from the nearest fp32 by R_REL: held within the bound's slack by comparing
    # with that r instead
    check_add_bwd(dy, dh, hc, r, w, dtype, rt.grad.cpu().view(B * S, N), xt.grad.cpu().view(B * S, N), wt.grad.cpu(), offset,
                  keep, p)


def test_rms_norm_add_unused_outputs_views_and_no_residual():
    N = 256
    x, w = randn(12, N, dtype="float32", seed=5), weight(N, "float32", False)
    big = leaf(randn(12, 2 * N, dtype="float32", seed=6))
    wt = leaf(w)
    # x a view with spaced rows; only y used; the cotangent an expanded scalar
    y, _ = fused.rms_norm_add(big[:, :N], big[:, N:], wt)
    y.sum().backward()
    h = (big[:, :N] + big[:, N:]).detach().cpu()
    r = ref.norm(h, w, EPS)[1].squeeze(-1).float()
    one = torch.ones(12, N)
    check_add_bwd(one, None, h, r, w, "float32", big.grad[:, N:].cpu(), big.grad[:, :N].cpu(), wt.grad.cpu())
    # only h used: the gradient is h's own
    xt = leaf(x)
    _, h = fused.rms_norm_add(xt, None, wt)
    h.backward(one.cuda())
    assert torch.equal(xt.grad.cpu(), one)
    # no gradient asked for x
    y, _ = fused.rms_norm_add(x.cuda(), None, wt)
    y.sum().backward()
    # no rows
    y, h = fused.rms_norm_add(torch.empty(0, N, device="cuda"), None, w.cuda())
    assert y.shape == h.shape == (0, N)
    # the second order is refused, not wrong
    xt = leaf(x)
    y, _ = fused.rms_norm_add(xt, None, wt)
    (g,) = torch.autograd.grad(y.sum(), xt, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    q = leaf(randn(4, 2, 16, dtype="float32", seed=27))
    out, _ = fused.rms_norm_rope(q, None, leaf(weight(16, "float32", False)), None, torch.arange(4, device="cuda"),
                                 freqs(16).cuda())
    (g,) = torch.autograd.grad(out.sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_rms_norm_add_in_place():
    for shape in ((5, 7, 384), (9, 4099)):
        N = shape[-1]
        x, res, w = randn(*shape, dtype="bfloat16", seed=7).cuda(), randn(*shape, dtype="bfloat16", seed=8).cuda(), \
            weight(N, "bfloat16", False).cuda()
        y, h = fused.rms_norm_add(x, res, w)
        a, b = fused.rms_norm_add_(x, res, w)
        assert a is x and b is res and torch.equal(x, y) and torch.equal(res, h)
    with pytest.raises(ValueError):
        fused.rms_norm_add_(x, x, w)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("offset", [False, True])
@pytest.mark.parametrize("N", [64, 200, 1001, 4096, 4099, 5120, 16384])
def test_rms_norm_add_is_the_norm_of_the_sum_bit_by_bit(N, offset, dtype):
    # small whole numbers: sums of squares are exact in any order, so nothing else may differ
    g = torch.Generator().manual_seed(N)
    x, res = (torch.randint(-5, 6, (40, N), generator=g).to(ref.TYPES[dtype]).cuda() for _ in range(2))
    w = weight(N, dtype, offset).cuda()
    y, h = fused.rms_norm_add(x, res, w, EPS, offset)
    assert torch.equal(h, x + res)
    assert torch.equal(y, rms_norm(h, w, EPS, offset))
    # r, which the backward gets, too
    r = torch.ops.rmsnorm_gb300.fwd(h, w, EPS, offset)[1]
    assert torch.equal(torch.ops.rmsnorm_gb300.add_fwd(x, res, w, EPS, offset, 0.0, None)[2], r)


@pytest.mark.parametrize("group,pow2", [(0, False), (128, True)])
def test_rms_norm_quant(group, pow2):
    x, res, w = randn(6, 640, dtype="bfloat16", seed=9), randn(6, 640, dtype="bfloat16", seed=10), weight(640, "bfloat16", False)
    codes, scales, h = fused.rms_norm_quant(x.cuda().view(2, 3, 640), w.cuda(), residual=res.cuda().view(2, 3, 640),
                                            group=group, pow2=pow2)
    assert codes.dtype == torch.float8_e4m3fn and codes.shape == (2, 3, 640) and scales.shape == (2, 3, 5 if group else 1)
    check_quant(x, res, w, "bfloat16", codes.view(6, 640).cpu(), scales.view(6, -1).cpu(), h.view(6, 640).cpu(), group, pow2)
    xt = x.cuda()
    assert fused.rms_norm_quant(xt, w.cuda())[2] is xt


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_rms_norm_rope_gradients_from_a_fused_projection(dtype):
    B, S, Hq, Hk, D, R = 2, 9, 6, 2, 64, 32
    qkv = randn(B * S, (Hq + 2 * Hk) * D, dtype=dtype, seed=11)
    wq, wk = weight(D, dtype, False), weight(D, dtype, False, 8)
    t = leaf(qkv.view(B, S, -1))
    q, k, _ = t.split([Hq * D, Hk * D, Hk * D], dim=-1)
    pos = torch.arange(S, device="cuda").repeat(B, 1) + 70000
    wqt, wkt = leaf(wq), leaf(wk)
    inv, m = fused.rope_frequencies(R)
    qo, ko = fused.rms_norm_rope(q.unflatten(-1, (Hq, D)), k.unflatten(-1, (Hk, D)), wqt, wkt, pos, inv, True, m)
    dq, dk = randn(B * S, Hq, D, dtype=dtype, seed=12), randn(B * S, Hk, D, dtype=dtype, seed=13)
    torch.autograd.backward([qo, ko], [dq.cuda().view_as(qo), dk.cuda().view_as(ko)])
    xs = [qkv[:, :Hq * D].unflatten(1, (Hq, D)), qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))]
    p = pos.cpu().view(-1)
    check_rope(xs, [wq, wk], p, R, dtype, True, [qo.detach().cpu().view(B * S, Hq, D), ko.detach().cpu().view(B * S, Hk, D)])
    g = t.grad.cpu().view(B * S, -1)
    check_rope_bwd([dq, dk], xs, [wq, wk], p, R, dtype, True,
                   [g[:, :Hq * D].unflatten(1, (Hq, D)), g[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))],
                   [wqt.grad.cpu(), wkt.grad.cpu()])
    assert torch.all(g[:, (Hq + Hk) * D:] == 0)


def test_rms_norm_rope_layouts_of_torch():
    T, H, D = 7, 4, 32
    q = randn(T, H, D, dtype="float32", seed=14)
    pos, inv = torch.arange(T, device="cuda"), freqs(D).cuda()
    w = weight(D, "float32", False).cuda()
    want, none = fused.rms_norm_rope(q.cuda(), None, w, None, pos, inv)
    assert none is None
    heads_first = q.transpose(0, 1).contiguous().cuda().transpose(0, 1)         # [H, T, D] in memory
    assert torch.equal(fused.rms_norm_rope(heads_first, None, w, None, pos, inv)[0], want)
    spaced = torch.zeros(T, H, 2 * D, device="cuda")
    spaced[..., ::2] = q.cuda()                                                 # no unit stride in D
    assert torch.equal(fused.rms_norm_rope(spaced[..., ::2], None, w, None, pos, inv)[0], want)
    same = q[:, :1].cuda().expand(T, H, D)                                      # one head repeated
    got = fused.rms_norm_rope(same, None, w, None, pos, inv)[0]
    assert torch.equal(got, want[:, :1].expand(T, H, D))
    one = leaf(q[:, :1])                                                        # its gradient sums over the repeats
    dy = randn(T, H, D, dtype="float32", seed=15)
    out, _ = fused.rms_norm_rope(one.expand(T, H, D), None, w, None, pos, inv)
    out.backward(dy.cuda())
    (d64, _), (e, _) = ref.rope_bwd(dy, q[:, :1].expand(T, H, D), w.cpu(), pos.cpu(), freqs(D), False, 1.0, EPS)
    ref.assert_close(one.grad, d64.sum(1, keepdim=True), (e + 4 * ref.U * d64.abs()).sum(1, keepdim=True), "shared head")
    # batch and sequence that are not one stride apart
    b = randn(3, 5, H, D, dtype="float32", seed=16).cuda()
    cut = b[:, 1:4]
    p2 = torch.arange(9, device="cuda").view(3, 3)
    got, _ = fused.rms_norm_rope(cut, None, w, None, p2, inv)
    assert torch.equal(got, fused.rms_norm_rope(cut.contiguous(), None, w, None, p2, inv)[0])
    # no tokens
    e, f = fused.rms_norm_rope(q[:0].cuda(), q[:0].cuda(), w, w, pos[:0], inv)
    assert e.shape == f.shape == (0, H, D)


def test_opcheck():
    ops = torch.ops.rmsnorm_gb300
    x, res, w = (leaf(randn(6, 64, dtype="float32", seed=17)), leaf(randn(6, 64, dtype="float32", seed=18)),
                 leaf(weight(64, "float32", False)))
    rng = fused.dropout_state(3)
    tests = ("test_schema", "test_autograd_registration", "test_faketensor", "test_aot_dispatch_dynamic")
    torch.library.opcheck(ops.add_fwd.default, (x, res, w, EPS, False, 0.5, rng), test_utils=tests)
    torch.library.opcheck(ops.add_fwd.default, (x, None, w, EPS, True, 0.0, None), test_utils=tests)
    torch.library.opcheck(ops.quant_fwd.default, (x.detach(), res.detach(), w.detach(), EPS, False, 32, False),
                          test_utils=("test_schema", "test_faketensor"))
    q, k = leaf(randn(6, 3, 32, dtype="float32", seed=19)), leaf(randn(6, 1, 32, dtype="float32", seed=20))
    wq = leaf(weight(32, "float32", False))
    pos, inv = torch.arange(6, device="cuda"), freqs(16).cuda()
    torch.library.opcheck(ops.rope_fwd.default, (q, k, wq, None, pos, inv, False, 1.0, EPS, False), test_utils=tests)
    torch.library.opcheck(ops.add_fwd_.default, (x.detach().clone(), res.detach().clone(), w.detach(), EPS, False),
                          test_utils=("test_schema", "test_faketensor"))


class Block(torch.nn.Module):
    """A pre-norm block: attention with head norms and rotary positions, then a
    two-layer feed-forward, both added to the residual stream through RMSNormAdd."""

    def __init__(self, N, H, Hk, D, ours):
        super().__init__()
        self.H, self.Hk, self.D, self.ours = H, Hk, D, ours
        self.qkv = torch.nn.Linear(N, (H + 2 * Hk) * D, bias=False)
        self.out = torch.nn.Linear(H * D, N, bias=False)
        self.up, self.down = torch.nn.Linear(N, 2 * N, bias=False), torch.nn.Linear(2 * N, N, bias=False)
        self.norm1, self.norm2 = fused.RMSNormAdd(N, p=0.1), fused.RMSNormAdd(N, p=0.1)
        self.rope = fused.RMSNormRope(D, D // 2, base=1000.0, device="cpu")

    def add(self, m, x, res, keep):
        """keep: the elements that dropout keeps, as the oracle draws them."""
        if self.ours:
            return m(x, res, keep[0])
        p, mask = keep[1], keep[2]
        h = torch.where(mask, x * ref.drop_scale(p), torch.zeros((), dtype=x.dtype, device=x.device)) if p else x
        h = h if res is None else h + res
        return ref_norm(h, m.weight), h

    def heads(self, q, k, pos):
        if self.ours:
            return self.rope(q, k, pos)
        z = [ref_norm(t, w) for t, w in ((q, self.rope.q_weight), (k, self.rope.k_weight))]
        return [rotate_half(t, pos, self.rope.inv_freq.to(t.dtype)) for t in z]

    def forward(self, x, res, pos, keeps):
        S = x.shape[0]
        y, h = self.add(self.norm1, x, res, keeps[0])
        q, k, v = self.qkv(y).split([self.H * self.D, self.Hk * self.D, self.Hk * self.D], dim=-1)
        q, k = self.heads(q.unflatten(-1, (self.H, self.D)), k.unflatten(-1, (self.Hk, self.D)), pos)
        v = v.unflatten(-1, (self.Hk, self.D))
        k, v = (t.repeat_interleave(self.H // self.Hk, dim=1) for t in (k, v))
        s = torch.einsum("ihd,jhd->hij", q, k) / self.D ** 0.5
        s = s.masked_fill(torch.ones(S, S, dtype=torch.bool, device=x.device).triu(1), -float("inf"))
        a = self.out(torch.einsum("hij,jhd->ihd", s.softmax(-1), v).reshape(S, -1))
        y, h = self.add(self.norm2, a, h, keeps[1])
        return self.down(torch.nn.functional.silu(self.up(y))), h


def ref_norm(h, w):
    return h * (h.square().mean(-1, keepdim=True) + EPS).rsqrt() * w


def rotate_half(t, pos, inv):
    R = 2 * inv.numel()
    ang = pos.to(inv.dtype).unsqueeze(-1) * inv
    c, s = ang.cos().unsqueeze(1), ang.sin().unsqueeze(1)
    a, b = t[..., :R // 2], t[..., R // 2:R]
    return torch.cat([a * c - b * s, b * c + a * s, t[..., R:]], dim=-1)


def test_a_block_of_them_together():
    """Forward and gradients of a block in fp32 against the same block in 64 bits with
    elementary operations and the oracle's dropout. fp32's products of up to 256 terms are
    off by 256 * 2^-24 of their terms' magnitudes, over six products one after the
    other; 1e-4 of each gradient's norm leaves them that much."""
    N, H, Hk, D, S = 128, 4, 2, 32, 50
    torch.manual_seed(0)
    ours = Block(N, H, Hk, D, True)
    gold = Block(N, H, Hk, D, False)
    gold.load_state_dict(ours.state_dict())
    ours, gold = ours.cuda(), gold.double().cuda()
    x, res = randn(S, N, dtype="float32", seed=21), randn(S, N, dtype="float32", seed=22)
    pos = torch.arange(S, device="cuda") + 300
    ours_in = [leaf(x), leaf(res)]
    gold_in = [leaf(x.double()), leaf(res.double())]
    seeds = [(41, 0), (42, 0)]
    ko = [(fused.dropout_state(*s),) for s in seeds]
    kg = [(None, 0.1, ref.kept(*s, S, N, 0.1).cuda()) for s in seeds]
    torch.backends.cuda.matmul.allow_tf32 = False
    a, b = ours(*ours_in, pos, ko), gold(*gold_in, pos, kg)
    dy, dh = randn(S, N, dtype="float32", seed=23).cuda(), randn(S, N, dtype="float32", seed=24).cuda()
    torch.autograd.backward(list(a), [dy, dh])
    torch.autograd.backward(list(b), [dy.double(), dh.double()])

    def near(p, q, what):
        assert (p.double() - q).norm() <= 1e-4 * q.norm(), what
    near(a[0], b[0], "output")
    near(a[1], b[1], "residual stream")
    near(ours_in[0].grad, gold_in[0].grad, "dx")
    near(ours_in[1].grad, gold_in[1].grad, "dresidual")
    for (n, p), (_, q) in zip(ours.named_parameters(), gold.named_parameters()):
        near(p.grad, q.grad, n)
    # serving: no dropout, and the same stream in place
    ours.eval()
    with torch.no_grad():
        y, h = ours(x.cuda(), res.cuda(), pos, [(None,)] * 2)
        t, r = x.cuda(), res.cuda()
        fused.rms_norm_add_(t, r, ours.norm1.weight)
        y1, h1 = ours.norm1(x.cuda(), res.cuda())
        assert torch.equal(t, y1) and torch.equal(r, h1)
        codes, scales, h2 = fused.rms_norm_quant(x.cuda(), ours.norm1.weight, residual=res.cuda(), group=32)
        assert torch.equal(h2, h1)
        back = codes.float() * scales.repeat_interleave(32, dim=1)
        # e4m3 rounds by 2^-4 of a value, or by 2^-10 scales below its least normal number
        ref.assert_close(back, y1, y1.abs().cpu().double() * 2.0 ** -4 * (1 + 2.0 ** -16)
                         + scales.repeat_interleave(32, dim=1).cpu().double() * 2.0 ** -10, "8-bit output")


def test_a_compiled_graph_has_no_breaks():
    w = weight(64, "float32", False).cuda()

    def f(x, res):
        y, h = fused.rms_norm_add(x, res, w)
        return y * 2, h
    x, res = randn(6, 64, dtype="float32", seed=25).cuda(), randn(6, 64, dtype="float32", seed=26).cuda()
    out = torch.compile(f, backend="eager", fullgraph=True)(x, res)
    want = f(x, res)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_the_in_place_addition_compiles_without_breaks():
    w = weight(64, "float32", False).cuda()

    def f(x, res):
        y, h = fused.rms_norm_add_(x, res, w)
        return y * 2, h + 1
    (x, res), (xc, rc) = ([randn(6, 64, dtype="float32", seed=s).cuda() for s in (25, 26)] for _ in range(2))
    want, out = f(x, res), torch.compile(f, backend="aot_eager", fullgraph=True)(xc, rc)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert torch.equal(xc, x) and torch.equal(rc, res)
    with pytest.raises(ValueError, match="memory"):     # the addresses are looked at when the op runs
        torch.ops.rmsnorm_gb300.add_fwd_(x, x, w, EPS, False)


def test_a_captured_training_step_draws_and_differentiates_anew():
    N, p = 1032, 0.25
    w, rng = leaf(weight(N, "bfloat16", False)), fused.dropout_state(3)
    x, res, dy = (randn(1100, N, dtype="bfloat16", seed=s).cuda() for s in (95, 96, 97))
    x.requires_grad_()
    q, wq = leaf(randn(64, 3, 64, dtype="bfloat16", seed=98)), leaf(weight(64, "bfloat16", False))
    pos, inv = torch.arange(64, device="cuda"), freqs(64).cuda()

    def step():
        y, h = fused.rms_norm_add(x, res, w, EPS, False, p, rng)
        a, _ = fused.rms_norm_rope(q, None, wq, None, pos, inv)
        out = (y, h, a) + torch.autograd.grad((y, a), (x, w, q, wq), (dy, a.detach()))
        rng[1] += 1
        return [t.detach() for t in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (11, 12):
        for offset in (5, 1 << 40):
            with torch.no_grad():
                x.copy_(randn(1100, N, dtype="bfloat16", seed=seed))
            rng.copy_(torch.tensor([seed, offset]))
            graph.replay()
            replayed = [t.clone() for t in got]
            assert rng.tolist() == [seed, offset + 1]
            rng.copy_(torch.tensor([seed, offset]))
            for a, b in zip(replayed, step()):
                assert torch.equal(a, b)


def test_a_rotation_without_weights_keeps_no_heads():
    T, H, D, R = 9, 4, 64, 32
    pos, inv = torch.arange(T, device="cuda") * 5, freqs(R).cuda()
    w = weight(D, "float32", False)
    dq, dk = randn(T, H, D, dtype="float32", seed=30), randn(T, 2, D, dtype="float32", seed=31)
    for wq, wk in ((None, None), (w, None), (None, w)):
        x = [randn(T, H, D, dtype="float32", seed=32), randn(T, 2, D, dtype="float32", seed=33)]
        for through in (fused.rms_norm_rope, lambda *a: torch.ops.rmsnorm_gb300.rope_fwd(*a, False, 1.0, EPS, False)):
            q, k = (leaf(t) for t in x)
            wt = [None if v is None else leaf(v) for v in (wq, wk)]
            held = []
            with torch.autograd.graph.saved_tensors_hooks(lambda t: held.append(t.shape) or t, lambda t: t):
                qo, ko = through(q * 1.0, k * 1.0, *wt, pos, inv)
            assert (q.shape in held, k.shape in held) == (wq is not None, wk is not None)
            torch.autograd.backward([qo, ko], [dq.cuda(), dk.cuda()])
            check_rope_bwd([dq, dk], x, [wq, wk], pos.cpu(), R, "float32", False, [q.grad.cpu(), k.grad.cpu()],
                           [None if v is None else v.grad.cpu() for v in wt])
            # one output unused: no gradient there but zeros
            q, k = (leaf(t) for t in x)
            qo, _ = through(q, k, *wt, pos, inv)
            qo.backward(dq.cuda())
            assert torch.all(k.grad == 0)
            if wq is None:
                check_rope_bwd([dq], x[:1], [None], pos.cpu(), R, "float32", False, [q.grad.cpu()], [None])
