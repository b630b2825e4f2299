"""The weights' gradients of the fused backwards, sums over all rows or heads, within bounds
that count the additions as the kernels make them: a lane's own rows one after the other,
then the lanes of a block, then the blocks. A bound for one long sum would grow with
the square of the terms and let a lost head pass. The host tests plant such mistakes in
the oracle; the GPU tests hold the kernels to the bounds."""
import pytest
import torch

from rmsnorm_fwd_bwd_gb300 import binding as B
from tests import fused_ref as ref
from tests.test_fused_gpu import (DTYPES, EPS, RING, ROPE_SHAPES, SWAP_SHAPES, add_bwd_inputs, freqs, randn, run_add_bwd,
                                  run_rope_bwd, weight)

SMS = 152
# the column reduce: at most 1216 blocks' rows, 64 of them at a time (19), 5 levels of lanes, 16 warps
REDUCE = 40


def add_depth(M):
    """Additions one after the other in a column of rmsnorm_add_bwd: a block's rows (at least a
    block an SM, where there are as many rows), at most 16 groups of a block, the reduce."""
    return -(-M // SMS) + 16 + REDUCE + 1


def rope_depth(T, heads):
    """Of rmsnorm_rope_bwd: a group's heads (at least 4 groups in each of 3 blocks an SM, which
    take whole runs of up to 8 heads, or a token's heads), at most 32 groups, the reduce."""
    return (heads + 8) * -(-T // (12 * SMS)) + 8 + 32 + REDUCE


def add_dw(dy, h, r):
    """dgamma in 64 bits, and the bound before its rounding: r is saved, two products."""
    terms = dy.double() * (h.double() * r.double().unsqueeze(-1))
    return terms.sum(0), ref.U * (add_depth(dy.shape[0]) + 2) * terms.abs().sum(0)


def rope_dw(dy, x, pos, R, inter, mscale, freq=None):
    """The terms [T, heads, D] of dgamma, dgamma and the bound before its rounding."""
    freq = freqs(R) if freq is None else freq
    v, mag = ref.rotate(dy.double(), pos, freq, inter, mscale, -1.0)
    x = x.double()
    n = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    ev = mag * (ref.TURN + ref.own_angle(pos, freq) + 3 * ref.U)
    terms = v * n
    rel = ref.U * rope_depth(dy.shape[0], dy.shape[1]) + ref.R_REL
    return terms, terms.sum((0, 1)), rel * terms.abs().sum((0, 1)) + (ev * n.abs()).sum((0, 1))


def with_rounding(want, err, dtype):
    return err + ref.rounding(want.abs() + err, ref.TYPES[dtype])


ROPE = sorted(set(SWAP_SHAPES + ROPE_SHAPES + [(30000, 5, 1, 90, 90), (9000, 16, 4, 256, 128)]))
ADD = RING + [(3000, 40), (2500, 200), (20000, 33), (9000, 1000), (30000, 264), (20000, 1030)]


# --------------------------------------------------------------------------- #
# planted mistakes, without a GPU
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("T,Hq,Hk,D,R", ROPE)
def test_a_lost_head_falls_outside_the_bound_of_the_rotation(T, Hq, Hk, D, R):
    pos = torch.arange(T) * 3 + 1
    for H, seed in ((Hq, 110), (Hk, 111)):
        dy, x = randn(T, H, D, dtype="bfloat16", seed=seed), randn(T, H, D, dtype="bfloat16", seed=seed + 2)
        terms, want, err = rope_dw(dy, x, pos, R, False, 1.0)
        bound = with_rounding(want, err, "bfloat16")
        lost = terms[:, H // 2].sum(0)                  # one head of all tokens, left out or taken twice
        for off, share in ((want, 0.8), (lost, 0.5)):
            # in all columns but those where what is lost is near 0 itself
            assert (off.abs() > bound).double().mean() >= share, (H, "zero" if off is want else "a head")
        assert torch.any(terms[T // 2].sum(0).abs() > bound) or T > 1000


@pytest.mark.parametrize("M,N", ADD)
def test_lost_rows_fall_outside_the_bound_of_the_addition(M, N):
    dy, _, h, r, _ = add_bwd_inputs(M, N, "bfloat16", False, seed=112)
    want, err = add_dw(dy, h, r)
    bound = with_rounding(want, err, "float32")
    # A single row's term is 0.1 times the product of two normal numbers, whose magnitude passes
    # 0.3 in 55 of 100 columns; the bound of the most rows, 30000, is 2^-24 * (198 + 57 + 2) *
    # 30000 * 0.1 * 2 / pi = 0.029, and the sum's rounding to fp32 nothing beside it.
    for rows, share in ((slice(None), 0.8), (slice(0, None, 456), 0.8), (slice(M // 2, M // 2 + 1), 0.5)):
        off = (dy[rows].double() * (h[rows].double() * r[rows].double().unsqueeze(-1))).sum(0)
        assert (off.abs() > bound).double().mean() >= share, rows


# --------------------------------------------------------------------------- #
# the kernels
# --------------------------------------------------------------------------- #
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,Hq,Hk,D,R", ROPE)
def test_rope_weight_gradients(T, Hq, Hk, D, R, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert torch.cuda.get_device_properties(0).multi_processor_count >= SMS
    dys = [randn(T, Hq, D, dtype=dtype, seed=110), randn(T, Hk, D, dtype=dtype, seed=111)]
    xs = [randn(T, Hq, D, dtype=dtype, seed=112), randn(T, Hk, D, dtype=dtype, seed=113)]
    ws = [weight(D, dtype, False), weight(D, dtype, False, 8)]
    pos = torch.arange(T) * 3 + 1
    for inter in (False, True):
        _, dws = run_rope_bwd(dys, xs, ws, pos, R, dtype, inter, 1.25)
        for dy, x, dw in zip(dys, xs, dws):
            _, want, err = rope_dw(dy, x, pos, R, inter, 1.25)
            ref.assert_close(dw, want, with_rounding(want, err, dtype), "dgamma of the heads")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", ADD)
def test_add_weight_gradients(M, N, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert torch.cuda.get_device_properties(0).multi_processor_count >= SMS
    dy, dh, h, r, w = add_bwd_inputs(M, N, dtype, True, seed=112)
    want, err = add_dw(dy, h, r)
    for layout, p in (("dense", 0.0), ("dense", 0.3), ("shifted", 0.0), ("mixed", 0.0)):
        rng = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
        _, _, dw = run_add_bwd(dy, dh, h, r, w, dtype, offset=True, p=p, rng=rng, layout=layout)
        ref.assert_close(dw, want, with_rounding(want, err, dtype), f"dgamma, {layout}, p = {p}")
