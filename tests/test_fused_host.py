"""The operators of include/rmsnorm_fused.h without a GPU: refusals (all before the
library touches CUDA), the formulas of the 64-bit oracle, Philox, the rotation's
frequencies, and the checks of the torch front end."""
import os
import re

import numpy as np
import pytest
import torch

from rmsnorm_fwd_bwd_gb300 import binding as B
from rmsnorm_fwd_bwd_gb300 import build as build_mod
from rmsnorm_fwd_bwd_gb300 import fused
from tests import fused_ref as ref

OK, NULL, SHAPE, DTYPE, EPS, ALIGN, WORKSPACE, ARG = 0, 1, 2, 3, 4, 5, 6, 9


@pytest.fixture(scope="module", autouse=True)
def library():
    build_mod.build()


def add_fwd(**kw):
    a = dict(x=0x1000, ldx=8, residual=0x2000, ldres=8, gamma=0x3000, h=0x4000, ldh=8, y=0x5000, ldy=8, rstd=0x6000,
             M=4, N=8, eps=1e-6, dtype=2, offset=0, dropout_p=0.0, rng=None, rng_used=None, stream=0)
    a.update(kw)
    return B.rmsnorm_add_fwd(**a)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=3)), (ARG, dict(offset=2)), (SHAPE, dict(M=-1)), (SHAPE, dict(N=0)), (SHAPE, dict(N=16385)),
    (EPS, dict(eps=0.0)), (EPS, dict(eps=float("nan"))), (SHAPE, dict(ldx=7)), (SHAPE, dict(ldres=7)),
    (SHAPE, dict(ldh=7)), (SHAPE, dict(ldy=7)), (ARG, dict(dropout_p=-0.1)), (ARG, dict(dropout_p=1.5)),
    (ARG, dict(dropout_p=float("nan"))), (OK, dict(M=0, x=None, y=None)), (NULL, dict(x=None)), (NULL, dict(gamma=None)),
    (NULL, dict(y=None)), (ALIGN, dict(x=0x1001)), (ALIGN, dict(residual=0x2001)), (ALIGN, dict(h=0x4001)),
    (ALIGN, dict(rstd=0x6002)), (NULL, dict(dropout_p=0.5)), (ALIGN, dict(dropout_p=0.5, rng=0x7004)),
    (ALIGN, dict(dropout_p=0.5, rng=0x7000, rng_used=0x7014)), (ARG, dict(h=0x5000)),
])
def test_add_fwd_refusals(want, kw):
    assert add_fwd(**kw) == want


def add_bwd(**kw):
    a = dict(dy=0x1000, lddy=8, dh=0x2000, lddh=8, h=0x3000, ldh=8, gamma=0x4000, rstd=0x5000, dx=0x6000, lddx=8,
             dresidual=0x7000, lddres=8, dgamma=0x8000, M=4, N=8, dtype=2, offset=0, dropout_p=0.0, rng=None,
             workspace=0x9000, workspace_bytes=1 << 20, stream=0)
    a.update(kw)
    return B.rmsnorm_add_bwd(**a)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=-1)), (ARG, dict(offset=-1)), (SHAPE, dict(N=16385)), (SHAPE, dict(lddy=7)), (SHAPE, dict(lddh=7)),
    (SHAPE, dict(ldh=7)), (SHAPE, dict(lddx=7)), (SHAPE, dict(lddres=7)), (ARG, dict(dropout_p=2.0)),
    (NULL, dict(dgamma=None)), (ALIGN, dict(dgamma=0x8001)), (NULL, dict(dy=None)), (NULL, dict(h=None)),
    (NULL, dict(gamma=None)), (NULL, dict(rstd=None)), (NULL, dict(workspace=None)), (ALIGN, dict(workspace=0x9008)),
    (ALIGN, dict(dx=0x6001)), (NULL, dict(dropout_p=0.5)), (ARG, dict(dropout_p=0.5, rng=0x100, dx=0x7000)),
])
def test_add_bwd_refusals(want, kw):
    assert add_bwd(**kw) == want


def quant(**kw):
    a = dict(x=0x1000, ldx=64, residual=0x2000, ldres=64, gamma=0x3000, h=0x4000, ldh=64, codes=0x5000, ldcodes=64,
             scales=0x6000, ldscales=2, M=4, N=64, eps=1e-6, dtype=1, offset=0, group=32, pow2=0, stream=0)
    a.update(kw)
    return B.rmsnorm_quant_fwd(**a)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=7)), (ARG, dict(offset=3)), (EPS, dict(eps=-1.0)), (ARG, dict(group=16)), (ARG, dict(group=-32)),
    (ARG, dict(pow2=2)), (SHAPE, dict(ldcodes=63)), (SHAPE, dict(ldscales=1)), (SHAPE, dict(ldh=63)),
    (OK, dict(M=0, x=None)), (NULL, dict(x=None)), (NULL, dict(codes=None)), (NULL, dict(scales=None)),
    (ALIGN, dict(scales=0x6002)), (ALIGN, dict(x=0x1001)),
])
def test_quant_refusals(want, kw):
    assert quant(**kw) == want


def rope(bwd=False, drop=(), **kw):
    s = dict(x=0x1000, x_token=128, x_head=64, gamma=0x2000, y=0x3000, y_token=128, y_head=64, heads=2)
    if bwd:
        s = dict(dy=0x1000, dy_token=128, dy_head=64, x=0x2000, x_token=128, x_head=64, gamma=0x3000, dx=0x4000,
                 dx_token=128, dx_head=64, dgamma=0x5000, heads=2)
    a = dict(sets=1, positions=0x6000, T=4, D=64, rotary_dim=64, inv_freq=0x7000, interleaved=0, mscale=1.0, eps=1e-6,
             dtype=2, offset=0, stream=0)
    if bwd:
        a.update(workspace=0x9000, workspace_bytes=1 << 24)
    for k, v in kw.items():
        (s if k in s and k not in ("heads_total",) else a)[k] = v
    cls = B.RopeHeadsBwd if bwd else B.RopeHeads
    n = a.pop("sets")
    sets = (cls * n)(*[cls(**s) for _ in range(n)]) if n else None
    return (B.rmsnorm_rope_bwd if bwd else B.rmsnorm_rope_fwd)(sets, **a)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=4)), (ARG, dict(offset=2)), (SHAPE, dict(D=513)), (SHAPE, dict(D=0)), (SHAPE, dict(rotary_dim=0)),
    (SHAPE, dict(rotary_dim=3)), (SHAPE, dict(rotary_dim=66)), (EPS, dict(eps=0.0)), (ARG, dict(interleaved=2)),
    (ARG, dict(mscale=float("inf"))), (ARG, dict(sets=0)), (ARG, dict(sets=3)), (SHAPE, dict(heads=0)),
    (SHAPE, dict(heads=65537, x_token=1 << 30)), (SHAPE, dict(x_token=63)), (SHAPE, dict(x_head=63)), (SHAPE, dict(x_token=-64)),
    (SHAPE, dict(sets=2, heads=40000)), (NULL, dict(positions=None)), (NULL, dict(inv_freq=None)),
    (ALIGN, dict(positions=0x6004)), (ALIGN, dict(inv_freq=0x7004)), (ALIGN, dict(gamma=0x2001)),
])
def test_rope_refusals(want, kw):
    assert rope(**kw) == want
    if "y" not in kw:
        kw = {{"x_token": "dy_token", "x_head": "dy_head"}.get(k, k): v for k, v in kw.items()}
        assert rope(bwd=True, **kw) == want


def test_rope_refusals_of_each_direction():
    assert rope(x=None) == NULL
    assert rope(y=None) == NULL
    assert rope(x=0x1001) == ALIGN
    assert rope(y_head=1) == SHAPE
    assert rope(T=0, positions=None, inv_freq=None, x=None, y=None) == OK
    assert rope(bwd=True, dy=None) == NULL
    assert rope(bwd=True, x=None) == NULL
    assert rope(bwd=True, dx=None) == NULL
    assert rope(bwd=True, dgamma=None) == NULL
    assert rope(bwd=True, workspace=None) == NULL
    assert rope(bwd=True, workspace=0x9008) == ALIGN
    assert rope(bwd=True, x_token=1) == SHAPE


def test_workspace_sizes_of_invalid_arguments():
    assert B.rmsnorm_add_bwd_workspace_size(0, 8, 0) == 0
    assert B.rmsnorm_add_bwd_workspace_size(4, 0, 0) == 0
    assert B.rmsnorm_add_bwd_workspace_size(4, 8, 9) == 0
    assert B.rmsnorm_rope_bwd_workspace_size(0, 1, 64, 0) == 0
    assert B.rmsnorm_rope_bwd_workspace_size(4, 0, 64, 0) == 0
    assert B.rmsnorm_rope_bwd_workspace_size(4, 1, 513, 0) == 0
    assert B.rmsnorm_rope_bwd_workspace_size(4, 1, 64, 5) == 0


def test_no_kernels_that_no_call_reaches():
    # rows of one offset are given to 32 lanes up to 64 octets: two octets a lane, never four
    root = os.path.join(os.path.dirname(build_mod.__file__), "_build")
    for name, kernels in (("add", "add_fwd_rows"), ("add_bwd", "add_bwd_rows"), ("quant", "quant_rows")):
        with open(os.path.join(root, name + ".ptxas.txt")) as f:
            seen = set(re.findall(kernels + r"ILi(\d)ELi(\d)ELi(n?\d+)ELi(\d)E", f.read()))
        assert len(seen) >= 30, name                    # (dtype, mode, lanes, octets)
        assert not [s for s in seen if s[1:] == ("2", "32", "4")], name


# --------------------------------------------------------------------------- #
# the oracle
# --------------------------------------------------------------------------- #
def test_philox_known_answers():
    # the test vectors of Philox4x32-10 that its authors give
    for ctr, key, out in (
            ([0] * 4, (0, 0), [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
            ([0xFFFFFFFF] * 4, (0xFFFFFFFF, 0xFFFFFFFF), [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
            ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], (0xA4093822, 0x299F31D0),
             [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])):
        assert ref.philox(np.array([ctr], dtype=np.uint32), key).tolist() == [out]


def test_dropout_share_and_streams():
    a = ref.kept(5, 7, 64, 512, 0.25)
    n = a.numel()
    assert abs(a.double().mean().item() - 0.75) < 5 * (0.75 * 0.25 / n) ** 0.5
    for other in (ref.kept(6, 7, 64, 512, 0.25), ref.kept(5, 8, 64, 512, 0.25), ref.kept(5, 7 + (1 << 32), 64, 512, 0.25)):
        # independent streams agree on 0.75^2 + 0.25^2 of the elements
        assert abs((a == other).double().mean().item() - 0.625) < 5 * (0.625 * 0.375 / n) ** 0.5
    # a row's numbers do not depend on the matrix around it
    assert torch.equal(ref.kept(5, 7, 3, 21, 0.25), a[:3, :21])


def _difference(f, v, t, step=1e-5):
    return (f(v + step * t) - f(v - step * t)) / (2 * step)


@pytest.mark.parametrize("offset", [False, True])
def test_add_bwd_formula_against_differences(offset):
    g = torch.Generator().manual_seed(3)
    M, N, p = 5, 23, 0.3
    x, res, dy, dh = (torch.randn(M, N, generator=g, dtype=torch.float64) for _ in range(4))
    w = torch.randn(N, generator=g, dtype=torch.float64)
    keep = ref.kept(11, 2, M, N, p)

    def loss(x, res, w):
        h = ref.add_sum(x, res, p, 11, 2)[0]
        return ((ref.norm(h, w, 1e-6, offset)[0] * dy).sum() + (h * dh).sum()).item()
    h = ref.add_sum(x, res, p, 11, 2)[0]
    r = ref.norm(h, w, 1e-6, offset)[1].squeeze(-1)
    (dres, dx, dw), _ = ref.add_bwd(dy, dh, h, r, w, offset, keep, p)
    for k in range(3):
        t, tw = torch.randn(M, N, generator=g, dtype=torch.float64), torch.randn(N, generator=g, dtype=torch.float64)
        # central differences: truncation step^2 and rounding 2^-53 / step, both near 1e-10 of the loss
        assert _difference(lambda v: loss(v, res, w), x, t) == pytest.approx((dx * t).sum().item(), rel=1e-6, abs=1e-7)
        assert _difference(lambda v: loss(x, v, w), res, t) == pytest.approx((dres * t).sum().item(), rel=1e-6, abs=1e-7)
        assert _difference(lambda v: loss(x, res, v), w, tw) == pytest.approx((dw * tw).sum().item(), rel=1e-6, abs=1e-7)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weight", [False, True])
def test_rope_bwd_formula_against_differences(interleaved, weight):
    g = torch.Generator().manual_seed(4)
    T, H, D, R = 3, 2, 14, 10
    x, dy, t = (torch.randn(T, H, D, generator=g, dtype=torch.float64) for _ in range(3))
    w, tw = (torch.randn(D, generator=g, dtype=torch.float64) for _ in range(2))
    w = w if weight else None
    pos, freq = torch.tensor([0, 5, 1000]), torch.rand(R // 2, generator=g, dtype=torch.float64)

    def loss(x, w):
        return (ref.rope_fwd(x, w, pos, freq, interleaved, 1.1, 1e-6)[0] * dy).sum().item()
    (dx, dw), _ = ref.rope_bwd(dy, x, w, pos, freq, interleaved, 1.1, 1e-6)
    assert _difference(lambda v: loss(v, w), x, t) == pytest.approx((dx * t).sum().item(), rel=1e-6, abs=1e-7)
    if weight:
        assert _difference(lambda v: loss(x, v), w, tw) == pytest.approx((dw * tw).sum().item(), rel=1e-6, abs=1e-7)


# --------------------------------------------------------------------------- #
# frequencies
# --------------------------------------------------------------------------- #
def test_rope_frequencies():
    f, m = fused.rope_frequencies(8, device="cpu")
    assert m == 1.0 and f.dtype == torch.float64
    assert f.tolist() == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15)
    lin, _ = fused.rope_frequencies(8, scaling="linear", factor=4.0, device="cpu")
    assert lin.tolist() == pytest.approx([v / 4.0 for v in f.tolist()], rel=1e-15)
    ntk, _ = fused.rope_frequencies(8, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0].item() == 1.0 and ntk[-1].item() == pytest.approx(f[-1].item() / 4.0, rel=1e-14)
    y, m = fused.rope_frequencies(128, scaling="yarn", factor=4.0, original_length=4096, device="cpu")
    f, _ = fused.rope_frequencies(128, device="cpu")
    assert m == pytest.approx(0.1 * np.log(4.0) + 1.0)
    turns = 4096 * f / (2 * np.pi)
    ratio = f / y
    assert torch.all(ratio[turns > 64] == 1.0)
    # below one turn, but for the pair that the rounding of the band's end takes in
    assert ratio[turns < 0.8].min().item() == pytest.approx(4.0, rel=1e-12)
    assert torch.all(ratio.diff() >= -1e-12) and ratio.min() >= 1.0
    one, _ = fused.rope_frequencies(2, scaling="ntk", factor=8.0, device="cpu")
    assert one.tolist() == [1.0]


@pytest.mark.parametrize("args,kw", [((7,), {}), ((0,), {}), ((8,), dict(base=0.0)), ((8,), dict(factor=0.5)),
                                     ((8,), dict(scaling="other")), ((8,), dict(scaling="yarn", factor=2.0))])
def test_rope_frequencies_refusals(args, kw):
    with pytest.raises(ValueError):
        fused.rope_frequencies(*args, device="cpu", **kw)


@pytest.mark.parametrize("R,base,length,factor", [(128, 1e4, 131072, 4.0), (128, 1e4, 65536, 4.0), (64, 1e4, 131072, 4.0),
                                                  (64, 1e4, 1 << 20, 32.0), (128, 1e4, 4096, 4.0), (128, 1e6, 32768, 4.0),
                                                  (2, 1e4, 4096, 2.0), (8, 10.0, 1 << 20, 4.0), (8, 300.0, 1 << 14, 4.0)])
def test_yarn_frequencies_where_the_band_ends_behind_the_last_pair(R, base, length, factor):
    # the published ramp over the pairs' index i, written with the turns that a pair makes: i is
    # pair(n) for n turns where length * base^(-2 i / R) = 2 pi n
    y, _ = fused.rope_frequencies(R, base, "yarn", factor, length, device="cpu")
    i = np.arange(R // 2)
    f = base ** (-2.0 * i / R)

    def pair(n):
        return R / 2 * np.log(length / (2 * np.pi * n)) / np.log(base)
    low, high = max(np.floor(pair(32.0)), 0), min(np.ceil(pair(1.0)), R - 1)
    slow = np.clip((i - low) / max(high - low, 0.001), 0, 1)
    assert y.tolist() == pytest.approx((f * (1 - slow) + f / factor * slow).tolist(), rel=1e-12)
    if pair(1.0) > R // 2:
        # every pair makes more than a turn: none is slowed by the whole factor
        assert length * f[-1] / (2 * np.pi) > 1.0 and (f / y.numpy()).max() < factor


@pytest.mark.parametrize("fast,slow", [(32.0, 0.0), (0.0, 0.0), (32.0, -1.0), (1.0, 2.0), (float("inf"), 1.0),
                                       (float("nan"), 1.0), (32.0, float("nan"))])
def test_yarn_refuses_turns_that_give_no_band(fast, slow):
    with pytest.raises(ValueError, match="turns"):
        fused.rope_frequencies(64, 1e4, "yarn", 4.0, 4096, fast, slow, device="cpu")


# --------------------------------------------------------------------------- #
# the torch front end's checks (before any call)
# --------------------------------------------------------------------------- #
def test_front_end_refusals():
    x, w = torch.zeros(4, 8), torch.ones(8)
    h = torch.zeros(4, 2, 8)
    pos, freq = torch.zeros(4, dtype=torch.int64), torch.ones(4, dtype=torch.float64)
    for call in (
            lambda: fused.rms_norm_add(x, torch.zeros(4, 7), w),
            lambda: fused.rms_norm_add(x, x, torch.ones(7)),
            lambda: fused.rms_norm_add(x, x, w.half()),
            lambda: fused.rms_norm_add(x, x.half(), w),
            lambda: fused.rms_norm_add(x, x, w, p=1.5),
            lambda: fused.rms_norm_add(x, x, w, p=0.1),
            lambda: fused.rms_norm_add(x, x, w, p=0.1, rng=torch.zeros(2)),
            lambda: fused.rms_norm_add(x, x, w, p=0.1, rng=torch.zeros(3, dtype=torch.int64)),
            lambda: fused.rms_norm_add_(x, torch.zeros(8, 4).t(), w),
            lambda: fused.rms_norm_add_(x, x, w),
            lambda: fused.rms_norm_add_(x, torch.zeros(4, 8, requires_grad=True), w),
            lambda: fused.rms_norm_quant(x, w, group=48),
            lambda: fused.rms_norm_quant(x, torch.ones(4, 8)),
            lambda: fused.rms_norm_rope(h, torch.zeros(3, 2, 8), w, w, pos, freq),
            lambda: fused.rms_norm_rope(h, torch.zeros(4, 2, 6), w, w, pos, freq),
            lambda: fused.rms_norm_rope(h, h, torch.ones(7), w, pos, freq),
            lambda: fused.rms_norm_rope(h, h, w, w, pos.int(), freq),
            lambda: fused.rms_norm_rope(h, h, w, w, pos[:3], freq),
            lambda: fused.rms_norm_rope(h, h, w, w, pos, freq.float()),
            lambda: fused.rms_norm_rope(h, None, w, w, pos, freq),
            lambda: fused.rms_norm_rope(torch.zeros(4, 0, 8), None, w, None, pos, freq)):
        with pytest.raises(ValueError):
            call()


def test_dropout_state_holds_64_bits():
    s = fused.dropout_state((1 << 64) - 1, 1 << 63, device="cpu")
    assert s.tolist() == [-1, -(1 << 63)]


def test_rope_module_keeps_its_frequencies_in_64_bits():
    m = fused.RMSNormRope(16, 8, base=500.0).to(torch.bfloat16) if torch.cuda.is_available() else \
        fused.RMSNormRope(16, 8, base=500.0, device="cpu").to(torch.bfloat16)
    assert m.inv_freq.dtype == torch.float64 and m.q_weight.dtype == torch.bfloat16
    assert m.inv_freq.cpu().tolist() == fused.rope_frequencies(8, 500.0, device="cpu")[0].tolist()


# --------------------------------------------------------------------------- #
# calls that would overwrite themselves, lose a derivative or a trace
# --------------------------------------------------------------------------- #
def test_outputs_at_one_address_are_refused():
    assert add_fwd(rstd=0x5000) == ARG
    assert add_bwd(dgamma=0x6000) == ARG
    assert add_bwd(dgamma=0x7000) == ARG
    assert add_bwd(workspace=0x7000) == ARG
    assert quant(h=0x5000) == ARG
    assert quant(scales=0x5000) == ARG
    assert quant(scales=0x4000) == ARG
    # two sets at one address
    assert rope(sets=2) == ARG
    assert rope(bwd=True, sets=2) == ARG
    sets = (B.RopeHeadsBwd * 2)(*[B.RopeHeadsBwd(0x1000, 128, 64, 0x2000, 128, 64, 0x3000, y, 128, 64, 0x5000, 2)
                                  for y in (0x4000, 0x8000)])
    assert B.rmsnorm_rope_bwd(sets, 0x6000, 4, 64, 64, 0x7000, 0, 1.0, 1e-6, 2, 0, 0x9000, 1 << 24) == ARG


def test_output_rows_that_overlap_are_refused():
    # two heads of a token and two tokens of a head at one place
    assert rope(y_token=64, y_head=64) == SHAPE
    assert rope(y_token=64, y_head=128, T=2, heads=3, positions=None) == NULL
    assert rope(y_token=64, y_head=255, positions=None) == SHAPE
    assert rope(y_token=64, y_head=256, positions=None) == NULL  # heads outside tokens: accepted so far
    assert rope(bwd=True, dx_token=64, dx_head=64) == SHAPE
    # inputs may
    assert rope(x_token=64, x_head=64, positions=None) == NULL


def test_outputs_on_inputs_of_other_rows_are_refused():
    # an output may lie on an input where its rows are the same; rows of another pitch, the weight,
    # or another set's heads would be overwritten before they are read. (NULL: accepted so far;
    # what follows is refused for another reason.)
    for kw in (dict(h=0x1000), dict(h=0x2000), dict(y=0x1000), dict(y=0x2000)):
        for ld in ("ldh", "ldy", "ldx", "ldres"):
            hit = {"h": ("ldh",), "y": ("ldy",)}[next(iter(kw))] + ({0x1000: ("ldx",), 0x2000: ("ldres",)}[next(iter(kw.values()))])
            assert add_fwd(**kw, **{ld: 16}, dropout_p=0.5) == (ARG if ld in hit else NULL), (kw, ld)
        assert add_fwd(**kw, ldh=16, ldy=16, ldx=16, ldres=16, dropout_p=0.5) == NULL
        assert add_fwd(**kw, M=1, ldh=16, ldy=24, dropout_p=0.5) == NULL
    assert add_fwd(h=0x3000, dropout_p=0.5) == ARG and add_fwd(y=0x3000, dropout_p=0.5) == ARG
    for out, ld in (("dx", "lddx"), ("dresidual", "lddres")):
        for at in (0x1000, 0x2000, 0x3000):
            assert add_bwd(**{out: at, ld: 16}) == ARG
        assert add_bwd(**{out: 0x4000}) == ARG
    assert add_bwd(dx=0x7000, lddx=16) == ARG
    assert quant(h=0x1000, ldh=72) == ARG and quant(h=0x2000, ldres=72) == ARG and quant(h=0x3000) == ARG
    for at in (0x1000, 0x2000, 0x3000):
        assert quant(codes=at) == ARG and quant(scales=at) == ARG
    assert rope(y=0x1000, positions=None) == NULL
    assert rope(y=0x1000, y_token=256) == ARG and rope(y=0x1000, x_head=72) == ARG and rope(y=0x2000) == ARG
    assert rope(y=0x1000, y_token=256, T=1, positions=None) == NULL
    assert rope(bwd=True, dx=0x1000, dx_token=256) == ARG and rope(bwd=True, dx=0x2000, x_head=72) == ARG
    assert rope(bwd=True, dx=0x3000) == ARG and rope(bwd=True, dx=0x1000, positions=None) == NULL
    # one set's output on the other's heads
    for y0, y1 in ((0x2000, 0x1000), (0x1000, 0x3000), (0x2000, 0x8000)):
        sets = (B.RopeHeads * 2)(B.RopeHeads(0x1000, 128, 64, 0x3000, y0, 128, 64, 2),
                                 B.RopeHeads(0x2000, 128, 64, 0x3800, y1, 128, 64, 2))
        assert B.rmsnorm_rope_fwd(sets, 0x6000, 4, 64, 64, 0x7000, 0, 1.0, 1e-6, 2, 0) == ARG
    sets = (B.RopeHeads * 2)(B.RopeHeads(0x1000, 128, 64, 0x3000, 0x1000, 128, 64, 2),
                             B.RopeHeads(0x2000, 128, 64, 0x3000, 0x2000, 128, 64, 2))
    assert B.rmsnorm_rope_fwd(sets, None, 4, 64, 64, 0x7000, 0, 1.0, 1e-6, 2, 0) == NULL


def test_in_place_addition_refuses_shared_rows():
    buf = torch.zeros(8, 40)
    w = torch.ones(16)
    for a, b in ((buf[:, :16], buf[:, 8:24]), (buf[:4, :16], buf[2:6, :16]), (buf[:, :16], buf[:, :16]),
                 (buf[:4, 16:32], buf[1:5, 8:24]), (buf.view(-1)[:64].view(4, 16), buf.view(-1)[48:112].view(4, 16))):
        assert fused._share_rows(a, b) and fused._share_rows(b, a)
        with pytest.raises(ValueError):
            fused.rms_norm_add_(a, b, w)
    for a, b in ((buf[:, :16], buf[:, 16:32]), (buf[:, 24:40], buf[:, 8:24]), (buf[:4, :16], buf[4:, :16]),
                 (buf.view(-1)[:64].view(4, 16), buf.view(-1)[64:128].view(4, 16)), (buf[:1, :16], buf[:1, 16:32])):
        assert not fused._share_rows(a, b) and not fused._share_rows(b, a)


def test_in_place_addition_refuses_a_weight_among_its_rows():
    # the rows are overwritten while other blocks still read the weight
    buf = torch.zeros(8, 40)
    flat = buf.view(-1)
    x, res = buf[:4, :16], buf[4:, 16:32]
    for t in (x, res):
        for w in (t[0], t[2], flat[t.storage_offset() + 5:][:16], flat[t.storage_offset() + 125:][:16]):
            with pytest.raises(ValueError, match="weight"):
                fused.rms_norm_add_(x, res, w)
    with pytest.raises(ValueError, match="weight"):
        fused.rms_norm_add_(flat[16:48].view(2, 16), flat[64:96].view(2, 16), flat[1:17])
    # before, between and behind the rows: such a call goes on, to the library
    for w in (flat[16:32], flat[120 + 16:120 + 32], flat[4 * 40:][:16], torch.ones(16)):
        assert not any(fused._among_rows(w, t) for t in (x, res))


def test_fake_tensors_take_every_call():
    # what traces and compiles: tensors with shapes but no addresses
    from torch._subclasses.fake_tensor import FakeTensorMode

    with FakeTensorMode():
        x, res, w = (torch.empty(s, device="cuda") for s in ((4, 16), (4, 16), (16,)))
        a, b = fused.rms_norm_add_(x, res, w)
        assert a is x and b is res
        assert [t.shape for t in fused.rms_norm_add(x, res, w)] == [x.shape, x.shape]
        assert [t.shape for t in fused.rms_norm_quant(x, w, residual=res)] == [(4, 16), (4, 1), (4, 16)]
        h, pos = torch.empty(4, 2, 8, device="cuda"), torch.empty(4, dtype=torch.int64, device="cuda")
        q, k = fused.rms_norm_rope(h, h, None, None, pos, torch.empty(4, dtype=torch.float64, device="cuda"))
        assert q.shape == k.shape == h.shape


def test_forward_mode_and_frequencies_gradients_are_refused():
    x, w = torch.zeros(4, 8), torch.ones(8)
    h, pos, freq = torch.zeros(4, 2, 8), torch.zeros(4, dtype=torch.int64), torch.ones(4, dtype=torch.float64)
    with torch.autograd.forward_ad.dual_level():
        d = torch.autograd.forward_ad.make_dual(x, torch.ones(4, 8))
        dh = torch.autograd.forward_ad.make_dual(h, torch.ones(4, 2, 8))
        for call in (lambda: fused.rms_norm_add(d, x, w), lambda: fused.rms_norm_add_(x, d, w),
                     lambda: fused.rms_norm_quant(d, w), lambda: fused.rms_norm_rope(dh, None, w, None, pos, freq)):
            with pytest.raises(RuntimeError, match="forward-mode"):
                call()
    with pytest.raises(ValueError):
        fused.rms_norm_rope(h, None, w, None, pos, freq.requires_grad_())


def test_modes_and_transforms_take_the_custom_ops():
    from torch.utils._python_dispatch import TorchDispatchMode

    class Mode(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            return func(*args, **(kwargs or {}))
    x = torch.zeros(3)
    assert fused._eager(x, None, torch.nn.Parameter(x))
    with Mode():
        assert not fused._eager(x)
    seen = []
    torch.func.vmap(lambda t: seen.append(fused._eager(t)) or t)(x)
    torch.func.grad(lambda t: seen.append(fused._eager(t)) or t.sum())(x)
    assert seen == [False, False]


def test_rope_module_from_the_meta_device():
    m = fused.RMSNormRope(16, 8, base=500.0, device="meta")
    assert m.inv_freq.is_meta
    m = m.to_empty(device="cpu")
    assert m.inv_freq.tolist() == fused.rope_frequencies(8, 500.0, device="cpu")[0].tolist()


def test_rotated_heads_refuse_outputs_on_parts_of_heads():
    base, far = 0x100000, 0x900000

    def fwd(*sets, T=4):
        sets = (B.RopeHeads * len(sets))(*(B.RopeHeads(*s) for s in sets))
        return B.rmsnorm_rope_fwd(sets, None, T, 64, 64, 0x7000, 0, 1.0, 1e-6, 2, 0)

    def bwd(*sets, T=4):
        sets = (B.RopeHeadsBwd * len(sets))(*(B.RopeHeadsBwd(*s) for s in sets))
        return B.rmsnorm_rope_bwd(sets, None, T, 64, 64, 0x7000, 0, 1.0, 1e-6, 2, 0, 0x8000000, 1 << 24)
    # (x, strides, weight, y, strides, heads); all that is wrong with what is taken is that there are no positions
    for at, want in ((0, NULL), (2, ARG), (-2, ARG), (128, ARG), (1022, ARG), (1024, NULL), (-1024, NULL), (-1022, ARG)):
        assert fwd((base, 128, 64, None, base + at, 128, 64, 2)) == want
        assert bwd((base, 128, 64, far, 128, 64, far + 0x1000, base + at, 128, 64, far + 0x2000, 2)) == want       # on dy
        assert bwd((far, 128, 64, base, 128, 64, far + 0x1000, base + at, 128, 64, far + 0x2000, 2)) == want       # on x
    assert fwd((far, 128, 64, base, base - 64, 128, 64, 2)) == ARG                                            # on the weight
    assert fwd((far, 64, 64, base, base, 64, 64, 1), T=1) == NULL and fwd((far, 64, 64, base, base + 2, 64, 64, 1), T=1) == ARG
    # queries and keys of one tensor, in place: side by side, interleaved, heads outside of tokens; and not quite so
    for token, head, k, want in ((256, 64, 128, NULL), (260, 64, 128, NULL), (256, 64, 127, ARG), (256, 128, 64, NULL),
                                 (264, 128, 64, NULL), (264, 128, 63, ARG), (64, 256, 512, NULL), (128, 512, 64, NULL),
                                 (128, 512, 63, ARG)):
        q, k = (base, token, head), (base + 2 * k, token, head)
        assert fwd((*q, None, *q, 2), (*k, None, *k, 2)) == want
        assert bwd((*q, None, 0, 0, None, *q, None, 2), (*k, None, 0, 0, None, *k, None, 2)) == want
        # out of place, into a tensor of the same strides
        assert fwd((far, 128, 64, None, *q, 2), (far + 0x1000, 128, 64, None, *k, 2)) == want


def test_rotated_heads_refuse_every_output_that_meets_other_heads():
    import random
    rng, D, base = random.Random(6), 8, 0x1000000

    def lies(p, token, head, heads, T):
        return {p + 2 * (t * token + h * head + d) for t in range(T) for h in range(heads) for d in range(D)}
    met = 0
    for _ in range(3000):
        T, H = rng.randint(1, 5), rng.randint(1, 4)
        tok = D * rng.randint(1, 14) + rng.choice([0, 0, 1, 4])

        def strides():
            return rng.choice([(tok, rng.choice([D, 2 * D, 3 * D, D + 1])), (rng.choice([D, 2 * D]), D * T * 2 + rng.choice([0, 3])),
                               (D * rng.randint(1, 14), rng.choice([D, 3 * D]))])
        sy = strides()
        sx = sy if rng.random() < 0.5 else strides()
        x = base + 2 * rng.choice([0, rng.randint(-150, 150), D * rng.randint(-20, 20)])
        sets = (B.RopeHeads * 1)(B.RopeHeads(x, *sx, None, base, *sy, H))
        st = B.rmsnorm_rope_fwd(sets, None, T, D, D, 0x7000, 0, 1.0, 1e-6, 2, 0)
        if st == SHAPE:
            continue
        in_place = x == base and (T == 1 or sx[0] == sy[0]) and (H == 1 or sx[1] == sy[1])
        if in_place:
            assert st == NULL
        elif lies(base, *sy, H, T) & lies(x, *sx, H, T):
            met += 1
            assert st == ARG, (T, H, sy, sx, x - base)
    assert met > 300


def test_strides_of_a_single_token_or_head_do_not_matter():
    any_stride = (1 << 62) + 12345
    for y, want in ((0x100000, NULL), (0x100000 + 2, ARG), (0x100000 + 128, NULL)):
        sets = (B.RopeHeads * 1)(B.RopeHeads(0x100000, any_stride, any_stride, None, y, any_stride - 7, any_stride, 1))
        assert B.rmsnorm_rope_fwd(sets, None, 1, 64, 64, 0x7000, 0, 1.0, 1e-6, 2, 0) == want
