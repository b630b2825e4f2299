"""PyTorch front end of the operators around an RMSNorm (``include/rmsnorm_fused.h``).

* ``rms_norm_add`` / ``RMSNormAdd``: dropout of a sublayer's output, its addition to
  the residual stream and the RMSNorm of the sum, differentiable; ``rms_norm_add_``
  does it in place for serving.
* ``rms_norm_quant``: addition, norm, and an e4m3 output with scales, for 8-bit
  matrix products.
* ``rms_norm_rope`` / ``RMSNormRope``: RMSNorm of query and key heads and their
  rotation by the tokens' positions, differentiable; ``rope_frequencies`` gives the
  rotation's frequencies, also for scaled contexts.

They are the custom ops ``rmsnorm_gb300::add_fwd`` and so on, with fake-tensor shapes
and autograd formulas, as those of ``autograd``, which tracing and compilation use.
Eager calls run the same code through ``torch.autograd.Function`` (or, where nothing
asks for a gradient, at once): the custom ops' dispatch takes some 300 us of host time
per forward and backward. Rows that a view spaces out are passed with their pitch.
Everything runs on torch's current stream of the inputs' device. They have no second
order and no forward-mode derivative: differentiating a backward, or tensors with
tangents, raises. A captured training step wants leaves whose eager graphs are gone, as
with any op: torch accumulates a leaf's gradient on the stream of its first graph.
"""
from __future__ import annotations

import contextlib
import math
from typing import Optional

import torch
from torch.autograd import forward_ad

from . import binding
from .autograd import _after_op, _row_view, _rows

CALLS = {"add_forward": 0, "add_backward": 0, "quant": 0, "rope_forward": 0, "rope_backward": 0}


def _done(status: int, where: str, counter: str) -> None:
    if status != binding.RMSNORM_OK:
        raise binding.RMSNormError(status, where)
    CALLS[counter] += 1
    _after_op()


def _same(where: str, x: torch.Tensor, **others) -> None:
    """Every given tensor on x's device and in x's dtype."""
    for name, t in others.items():
        if t is not None and (t.dtype != x.dtype or t.device != x.device):
            raise ValueError(f"{where}: x and {name} must share a dtype and a device")


def _check_rows(where: str, x, residual, weight) -> None:
    if weight.dim() != 1 or x.dim() < 1 or x.shape[-1] != weight.shape[0]:
        raise ValueError(f"{where}: weight must be 1-D with x.shape[-1] elements")
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"{where}: x and residual must have the same shape")
    _same(where, x, weight=weight, residual=residual)


def _check_dropout(where: str, x, p: float, rng) -> None:
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"{where}: p must be in [0, 1]")
    if p > 0.0 and (rng is None or rng.dtype != torch.int64 or rng.numel() != 2 or rng.device != x.device
                    or not rng.is_contiguous()):
        raise ValueError(f"{where}: dropout needs rng, an int64 tensor {{seed, offset}} on x's device")


def _eager(*tensors) -> bool:
    """Plain tensors outside of tracing, compilation, dispatch modes and function transforms."""
    return not (torch.compiler.is_compiling() or torch._C._len_torch_dispatch_stack()
                or torch._C._are_functorch_transforms_active() or torch._C._get_tracing_state()) and all(
        t is None or type(t) is torch.Tensor or type(t) is torch.nn.Parameter for t in tensors)


def _no_tangents(where: str, *tensors) -> None:
    """Forward-mode derivatives would be dropped in silence."""
    if forward_ad._current_level >= 0 and any(
            t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise RuntimeError(f"{where} has no forward-mode derivative")


def _wants_grad(*tensors) -> bool:
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _on(t: torch.Tensor):
    """The tensor's device as the current one."""
    if t.device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(t.device)


def _pitched(t: Optional[torch.Tensor]):
    return (None, 0) if t is None else _row_view(t)


# --------------------------------------------------------------------------- #
# dropout, residual addition, RMSNorm
# --------------------------------------------------------------------------- #
def dropout_state(seed: int, offset: int = 0, device="cuda") -> torch.Tensor:
    """{seed, offset} for the dropout of ``rms_norm_add``. The numbers depend on these
    and on the element's row and column alone: give every layer a seed of its own
    and raise the offset every step (``state[1] += 1``, also inside a graph). Where the
    backward runs forwards again (activation checkpointing), raise it after the backward."""
    def signed(v):
        v &= (1 << 64) - 1
        return v - (1 << 64) if v >> 63 else v
    return torch.tensor([signed(int(seed)), signed(int(offset))], dtype=torch.int64, device=device)


def _add_fwd_run(x, residual, weight, eps, offset, p, rng, want_rstd=True):
    with _on(x):
        xr, ldx = _row_view(x)
        rr, ldr = _pitched(residual)
        M, N = _rows(x)
        h = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) if want_rstd else None
        used = torch.empty(2 if p > 0.0 else 0, dtype=torch.int64, device=x.device)
        if p > 0.0 and M == 0:
            used.copy_(rng)
        _done(binding.rmsnorm_add_fwd(xr, ldx, rr, ldr, weight.contiguous(), h, N, y, N, rstd, M, N, eps, x.dtype,
                                      int(offset), p, rng if p > 0.0 else None, used if p > 0.0 else None),
              "rmsnorm_add_fwd", "add_forward")
    return y, h, rstd, used


@torch.library.custom_op("rmsnorm_gb300::add_fwd", mutates_args=())
def _add_fwd(x: torch.Tensor, residual: Optional[torch.Tensor], weight: torch.Tensor, eps: float, offset: bool,
             p: float, rng: Optional[torch.Tensor]) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    return _add_fwd_run(x, residual, weight, eps, offset, p, rng)


@_add_fwd.register_fake
def _(x, residual, weight, eps, offset, p, rng):
    return (x.new_empty(x.shape), x.new_empty(x.shape), x.new_empty(x.shape[:-1], dtype=torch.float32),
            x.new_empty((2 if p > 0.0 else 0,), dtype=torch.int64))


def _add_bwd_run(dy, dh, h, weight, rstd, offset, p, rng):
    """(dresidual, dx, dweight); dx is empty without dropout, where it is dresidual."""
    with _on(h):
        dyr, lddy = _row_view(dy)
        dhr, lddh = _pitched(dh)
        hr, ldh = _row_view(h)
        M, N = _rows(h)
        need = binding.rmsnorm_add_bwd_workspace_size(M, N, h.dtype)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=h.device)
        dres = torch.empty(h.shape, dtype=h.dtype, device=h.device)
        dx = torch.empty(h.shape if p > 0.0 else (0,), dtype=h.dtype, device=h.device)
        dw = torch.empty(weight.shape, dtype=weight.dtype, device=weight.device)
        _done(binding.rmsnorm_add_bwd(dyr, lddy, dhr, lddh, hr, ldh, weight.contiguous(), rstd.contiguous(),
                                      dx if p > 0.0 else None, N, dres, N, dw, M, N, h.dtype, int(offset), p,
                                      rng if p > 0.0 else None, ws, ws.numel()),
              "rmsnorm_add_bwd", "add_backward")
    return dres, dx, dw


@torch.library.custom_op("rmsnorm_gb300::add_bwd", mutates_args=())
def _add_bwd(dy: torch.Tensor, dh: Optional[torch.Tensor], h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
             offset: bool, p: float, rng: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    return _add_bwd_run(dy, dh, h, weight, rstd, offset, p, rng)


@_add_bwd.register_fake
def _(dy, dh, h, weight, rstd, offset, p, rng):
    return h.new_empty(h.shape), h.new_empty(h.shape if p > 0.0 else (0,)), weight.new_empty(weight.shape)


def _add_setup(ctx, inputs, output):
    _x, residual, weight, _eps, offset, p, _rng = inputs
    _y, h, rstd, used = output
    ctx.set_materialize_grads(False)
    ctx.save_for_backward(h, weight, rstd, used)
    ctx.offset, ctx.p, ctx.has_residual = offset, p, residual is not None


def _add_backward(ctx, dy, dh, drstd, dused):
    del drstd, dused  # auxiliary outputs; no gradient flows through them
    h, weight, rstd, used = ctx.saved_tensors
    if dy is None:
        dy = torch.zeros_like(h)
    dres, dx, dw = _add_bwd(dy, dh, h, weight, rstd, ctx.offset, ctx.p, used)
    return dx if ctx.p > 0.0 else dres, dres if ctx.has_residual else None, dw, None, None, None, None


_add_fwd.register_autograd(_add_backward, setup_context=_add_setup)


class _AddFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, offset, p, rng):
        y, h, rstd, used = _add_fwd_run(x, residual, weight, eps, offset, p, rng)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(h, weight, rstd, used)
        ctx.how = (offset, p, residual is not None)
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        h, weight, rstd, used = ctx.saved_tensors
        offset, p, has_residual = ctx.how
        if dy is None:
            dy = torch.zeros_like(h)
        # with a graph of the backward asked for: the op, which refuses to be differentiated
        run = _add_bwd if torch.is_grad_enabled() else _add_bwd_run
        dres, dx, dw = run(dy, dh, h, weight, rstd, offset, p, used)
        return dx if p > 0.0 else dres, dres if has_residual else None, dw, None, None, None, None


def rms_norm_add(x: torch.Tensor, residual: Optional[torch.Tensor], weight: torch.Tensor, eps: float = 1e-6,
                 offset: bool = False, p: float = 0.0,
                 rng: Optional[torch.Tensor] = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(y, h): h = dropout(x, p) + residual in x's dtype, y = RMSNorm(h) * weight (offset:
    * (1 + weight)). ``rng``: see ``dropout_state``; the backward drops the same
    elements, whatever happens to ``rng`` in between."""
    _check_rows("rms_norm_add", x, residual, weight)
    _check_dropout("rms_norm_add", x, p, rng)
    _no_tangents("rms_norm_add", x, residual, weight)
    args = (x, residual, weight, float(eps), bool(offset), float(p), rng)
    if _eager(x, residual, weight, rng):
        if _wants_grad(x, residual, weight):
            return _AddFunction.apply(*args)
        return _add_fwd_run(*args, want_rstd=False)[:2]
    return torch.ops.rmsnorm_gb300.add_fwd(*args)[:2]


def _row_bytes(t: torch.Tensor):
    """(address, pitch, bytes of a row, rows) of a contiguous tensor, or a 2-D one with spaced rows."""
    N = t.shape[-1]
    pitch = t.stride(0) if t.dim() == 2 and t.shape[0] > 1 else N
    return t.data_ptr(), pitch * t.element_size(), N * t.element_size(), t.numel() // N


def _share_rows(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether rows of two tensors of one shape (contiguous, or 2-D with spaced rows) share
    memory; the halves of wider rows do not."""
    (p, pitch, width, M), (q, pitch_b, _, _) = _row_bytes(a), _row_bytes(b)
    if p >= q + (M - 1) * pitch_b + width or q >= p + (M - 1) * pitch + width:
        return False
    # interleaved: of one pitch, the columns of one in the gaps of the other
    return not (pitch == pitch_b and width <= (q - p) % pitch <= pitch - width)


def _among_rows(w: torch.Tensor, t: torch.Tensor) -> bool:
    """Whether a contiguous row ``w`` of t's width shares memory with one of t's rows."""
    (q, _, width, _), (p, pitch, _, M) = _row_bytes(w), _row_bytes(t)
    if q + width <= p or q >= p + (M - 1) * pitch + width:
        return False
    # in a gap between two rows, or not
    return not width <= (q - p) % pitch <= pitch - width


def _add_in_place(x, residual, weight, eps, offset):
    # (here, where tensors have their strides and addresses also in a traced or compiled program)
    for t in (x, residual):
        if not t.is_contiguous() and _row_view(t)[0] is not t:
            raise ValueError("rms_norm_add_ needs contiguous tensors, or 2-D ones with unit column stride")
    if x.numel() and _share_rows(x, residual):
        raise ValueError("rms_norm_add_: x and residual must not share memory")
    # (a weight with a stride is laid out first)
    if x.numel() and weight.is_contiguous() and (_among_rows(weight, x) or _among_rows(weight, residual)):
        raise ValueError("rms_norm_add_: the weight must not share memory with x or residual")
    with _on(x):
        M, N = _rows(x)
        ldx, ldr = (t.stride(0) if t.dim() == 2 and M > 1 else N for t in (x, residual))
        _done(binding.rmsnorm_add_fwd(x, ldx, residual, ldr, weight.contiguous(), residual, ldr, x, ldx, None, M, N, eps,
                                      x.dtype, int(offset)), "rmsnorm_add_fwd", "add_forward")


@torch.library.custom_op("rmsnorm_gb300::add_fwd_", mutates_args=("x", "residual"))
def _add_fwd_(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor, eps: float, offset: bool) -> None:
    _add_in_place(x, residual, weight, eps, offset)


@_add_fwd_.register_fake
def _(x, residual, weight, eps, offset):
    return None


def rms_norm_add_(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                  offset: bool = False) -> tuple[torch.Tensor, torch.Tensor]:
    """In place, for serving: residual becomes x + residual and x its RMSNorm; returns
    (x, residual). Not differentiable. Both are contiguous, or 2-D with spaced rows."""
    _check_rows("rms_norm_add_", x, residual, weight)
    if torch.is_grad_enabled() and any(t.requires_grad for t in (x, residual, weight)):
        raise ValueError("rms_norm_add_ is not differentiable: use rms_norm_add, or torch.no_grad()")
    _no_tangents("rms_norm_add_", x, residual, weight)
    # always the op, which marks both as changed for whoever saved them for a backward
    torch.ops.rmsnorm_gb300.add_fwd_(x, residual, weight, float(eps), bool(offset))
    return x, residual


class RMSNormAdd(torch.nn.Module):
    """The residual branch as a module: ``y, h = norm(x, residual, rng)``, dropout with
    probability ``p`` in training mode only; weight as ``autograd.RMSNorm``'s."""

    def __init__(self, normalized_shape: int, eps: float = 1e-6, offset: bool = False, p: float = 0.0, device=None,
                 dtype=None):
        super().__init__()
        self.eps, self.offset, self.p = eps, offset, p
        init = torch.zeros if offset else torch.ones
        self.weight = torch.nn.Parameter(init(normalized_shape, device=device, dtype=dtype))

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                rng: Optional[torch.Tensor] = None) -> tuple[torch.Tensor, torch.Tensor]:
        return rms_norm_add(x, residual, self.weight, self.eps, self.offset, self.p if self.training else 0.0, rng)


# --------------------------------------------------------------------------- #
# 8-bit output
# --------------------------------------------------------------------------- #
def _quant_run(x, residual, weight, eps, offset, group, pow2):
    with _on(x):
        xr, ldx = _row_view(x)
        rr, ldr = _pitched(residual)
        M, N = _rows(x)
        n = -(-N // group) if group else 1
        codes = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        scales = torch.empty((*x.shape[:-1], n), dtype=torch.float32, device=x.device)
        h = torch.empty(x.shape if residual is not None else (0,), dtype=x.dtype, device=x.device)
        _done(binding.rmsnorm_quant_fwd(xr, ldx, rr, ldr, weight.contiguous(), h if residual is not None else None, N,
                                        codes, N, scales, n, M, N, eps, x.dtype, int(offset), group, int(pow2)),
              "rmsnorm_quant_fwd", "quant")
    return codes, scales, h


@torch.library.custom_op("rmsnorm_gb300::quant_fwd", mutates_args=())
def _quant_fwd(x: torch.Tensor, residual: Optional[torch.Tensor], weight: torch.Tensor, eps: float, offset: bool,
               group: int, pow2: bool) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    return _quant_run(x, residual, weight, eps, offset, group, pow2)


@_quant_fwd.register_fake
def _(x, residual, weight, eps, offset, group, pow2):
    n = -(-x.shape[-1] // group) if group else 1
    return (x.new_empty(x.shape, dtype=torch.float8_e4m3fn), x.new_empty((*x.shape[:-1], n), dtype=torch.float32),
            x.new_empty(x.shape if residual is not None else (0,)))


def rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, offset: bool = False,
                   residual: Optional[torch.Tensor] = None, group: int = 0,
                   pow2: bool = False) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(codes, scales, h): h = x + residual (x itself without one), and RMSNorm(h) as
    float8_e4m3fn codes with a float32 scale per row (``group`` 0: scales [..., 1]) or per
    32, 64 or 128 columns; ``pow2`` rounds the scales up to powers of two. The values
    are codes * scales. Not differentiable."""
    _check_rows("rms_norm_quant", x, residual, weight)
    if group not in (0, 32, 64, 128):
        raise ValueError("rms_norm_quant: group must be 0 (the row), 32, 64 or 128")
    _no_tangents("rms_norm_quant", x, residual, weight)
    args = (x.detach(), None if residual is None else residual.detach(), weight.detach(), float(eps), bool(offset),
            int(group), bool(pow2))
    codes, scales, h = _quant_run(*args) if _eager(x, residual, weight) else torch.ops.rmsnorm_gb300.quant_fwd(*args)
    return codes, scales, x if residual is None else h


# --------------------------------------------------------------------------- #
# head norm and rotary positions
# --------------------------------------------------------------------------- #
def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                     original_length: int = 0, fast_turns: float = 32.0, slow_turns: float = 1.0,
                     device="cuda") -> tuple[torch.Tensor, float]:
    """(inv_freq, mscale) for ``rms_norm_rope``: float64 radians per position of the
    rotary_dim / 2 pairs, base ** (-2 i / rotary_dim), and the factor of the rotated
    entries. For a context ``factor`` times as long:

    * ``"linear"``: every frequency divided by factor (positions are interpolated);
    * ``"ntk"``: the base raised so that the slowest pair is slowed by factor and the
      fastest not at all;
    * ``"yarn"`` (Peng, Quesnelle, Fan and Shippole, 2023): pairs that make more than
      ``fast_turns`` turns within ``original_length`` positions keep their frequency, those
      below ``slow_turns`` are divided by factor, those between are blended by their
      index (which may reach its end behind the last pair), and mscale =
      0.1 ln(factor) + 1.
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not base > 0.0 or not factor >= 1.0:
        raise ValueError("base must be positive and factor at least 1")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    half = rotary_dim // 2
    if scaling == "ntk" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freq = [base ** (-2.0 * i / rotary_dim) for i in range(half)]
    mscale = 1.0
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "yarn":
        if original_length < 1 or not base > 1.0:
            raise ValueError("yarn needs original_length and a base above 1")
        if not 0.0 < slow_turns <= fast_turns < math.inf:
            raise ValueError("yarn needs 0 < slow_turns <= fast_turns")

        def pair_of(turns):  # the pair, as a real number, that makes so many turns in original_length
            return rotary_dim * math.log(original_length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        low = max(math.floor(pair_of(fast_turns)), 0)
        high = min(math.ceil(pair_of(slow_turns)), rotary_dim - 1)  # the published limit
        span = max(high - low, 0.001)
        slow = [min(max((i - low) / span, 0.0), 1.0) for i in range(half)]
        freq = [f * (1.0 - s) + f / factor * s for f, s in zip(freq, slow)]
        mscale = 0.1 * math.log(factor) + 1.0
    return torch.tensor(freq, dtype=torch.float64, device=device), mscale


def _tokens(t: torch.Tensor) -> torch.Tensor:
    """[..., heads, D] as [tokens, heads, D] with unit stride in D; a view where it can be."""
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        t = t.contiguous()
    try:
        t = t.view(-1, *t.shape[-2:]) if t.numel() else t.reshape(math.prod(t.shape[:-2]), *t.shape[-2:])
    except RuntimeError:
        t = t.contiguous().view(-1, *t.shape[-2:])
    D = t.shape[2]
    # strides that repeat or overlap rows (an expanded tensor) are laid out
    if (t.shape[0] > 1 and t.stride(0) < D) or (t.shape[1] > 1 and t.stride(1) < D):
        t = t.contiguous()
    return t


def _rope_fwd_run(q, k, q_weight, k_weight, positions, inv_freq, interleaved, mscale, eps, offset):
    with _on(q):
        qo = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        ko = torch.empty(k.shape if k is not None else (0,), dtype=q.dtype, device=q.device)
        D = q.shape[-1]
        pos, freq = positions.contiguous(), inv_freq.contiguous()
        keep = [(_tokens(q), None if q_weight is None else q_weight.contiguous(), _tokens(qo))]
        if k is not None:
            keep.append((_tokens(k), None if k_weight is None else k_weight.contiguous(), _tokens(ko)))
        _done(binding.rmsnorm_rope_fwd(binding.rope_heads(keep), pos, pos.numel(), D, 2 * freq.numel(), freq,
                                       int(interleaved), mscale, eps, q.dtype, int(offset)),
              "rmsnorm_rope_fwd", "rope_forward")
    return qo, ko


@torch.library.custom_op("rmsnorm_gb300::rope_fwd", mutates_args=())
def _rope_fwd(q: torch.Tensor, k: Optional[torch.Tensor], q_weight: Optional[torch.Tensor],
              k_weight: Optional[torch.Tensor], positions: torch.Tensor, inv_freq: torch.Tensor, interleaved: bool,
              mscale: float, eps: float, offset: bool) -> tuple[torch.Tensor, torch.Tensor]:
    return _rope_fwd_run(q, k, q_weight, k_weight, positions, inv_freq, interleaved, mscale, eps, offset)


@_rope_fwd.register_fake
def _(q, k, q_weight, k_weight, positions, inv_freq, interleaved, mscale, eps, offset):
    return q.new_empty(q.shape), q.new_empty(k.shape if k is not None else (0,))


def _rope_bwd_run(dq, dk, q, k, q_weight, k_weight, positions, inv_freq, interleaved, mscale, eps, offset):
    with _on(q):
        D = q.shape[-1]
        pos, freq = positions.contiguous(), inv_freq.contiguous()
        outs, keep, heads = [], [], 0
        for g, x, w in ((dq, q, q_weight), (dk, k, k_weight)):
            dx = torch.empty(x.shape if x is not None else (0,), dtype=q.dtype, device=q.device)
            dw = torch.empty((D,) if w is not None else (0,), dtype=q.dtype, device=q.device)
            outs.append((dx, dw))
            if x is not None:
                keep.append((_tokens(g), None if w is None else _tokens(x), None if w is None else w.contiguous(),
                             _tokens(dx), None if w is None else dw))
                heads += x.shape[-2]
        need = binding.rmsnorm_rope_bwd_workspace_size(pos.numel(), heads, D, q.dtype)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
        _done(binding.rmsnorm_rope_bwd(binding.rope_heads_bwd(keep), pos, pos.numel(), D, 2 * freq.numel(), freq,
                                       int(interleaved), mscale, eps, q.dtype, int(offset), ws, ws.numel()),
              "rmsnorm_rope_bwd", "rope_backward")
    return outs[0][0], outs[1][0], outs[0][1], outs[1][1]


@torch.library.custom_op("rmsnorm_gb300::rope_bwd", mutates_args=())
def _rope_bwd(dq: torch.Tensor, dk: Optional[torch.Tensor], q: torch.Tensor, k: Optional[torch.Tensor],
              q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor], positions: torch.Tensor,
              inv_freq: torch.Tensor, interleaved: bool, mscale: float, eps: float,
              offset: bool) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    return _rope_bwd_run(dq, dk, q, k, q_weight, k_weight, positions, inv_freq, interleaved, mscale, eps, offset)


@_rope_bwd.register_fake
def _(dq, dk, q, k, q_weight, k_weight, positions, inv_freq, interleaved, mscale, eps, offset):
    D = q.shape[-1]
    return (q.new_empty(q.shape), q.new_empty(k.shape if k is not None else (0,)),
            q.new_empty((D,) if q_weight is not None else (0,)), q.new_empty((D,) if k_weight is not None else (0,)))


def _rope_save(ctx, q, k, q_weight, k_weight, positions, inv_freq, *how):
    # heads without a weight are turned back without their values
    ctx.save_for_backward(None if q_weight is None else q, None if k_weight is None else k, q_weight, k_weight, positions,
                          inv_freq)
    ctx.has_k, ctx.how = k is not None, how


def _rope_setup(ctx, inputs, output):
    _rope_save(ctx, *inputs)


def _rope_grads(ctx, dq, dk, run):
    q, k, q_weight, k_weight, positions, inv_freq = ctx.saved_tensors
    if not ctx.has_k:
        dk = None
    # without a weight the cotangents stand in: of the heads only the shape is needed
    gq, gk, gqw, gkw = run(dq, dk, dq if q is None else q, dk if k is None else k, q_weight, k_weight, positions, inv_freq,
                           *ctx.how)
    return (gq, gk if ctx.has_k else None, gqw if q_weight is not None else None,
            gkw if k_weight is not None else None, None, None, None, None, None, None)


def _rope_backward(ctx, dq, dk):
    return _rope_grads(ctx, dq, dk, _rope_bwd)


_rope_fwd.register_autograd(_rope_backward, setup_context=_rope_setup)


class _RopeFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, *args):
        _rope_save(ctx, *args)
        return _rope_fwd_run(*args)

    @staticmethod
    def backward(ctx, dq, dk):
        return _rope_grads(ctx, dq, dk, _rope_bwd if torch.is_grad_enabled() else _rope_bwd_run)


def rms_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], q_weight: Optional[torch.Tensor],
                  k_weight: Optional[torch.Tensor], positions: torch.Tensor, inv_freq: torch.Tensor,
                  interleaved: bool = False, mscale: float = 1.0, eps: float = 1e-6,
                  offset: bool = False) -> tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(q, k) with every head normalised (RMSNorm over its D entries, times its weight;
    not where the weight is None) and its first 2 * len(inv_freq) entries rotated by
    positions * inv_freq. q is [..., heads, D], k (or None) [..., key heads, D] with the
    same leading shape, which positions (int64) has too; views such as the parts of a
    fused projection are read in place. Pairs are (i, i + R / 2), or (2i, 2i + 1) where
    interleaved. See ``rope_frequencies`` for inv_freq and mscale."""
    for name, t in (("q", q), ("k", k)):
        if t is None:
            continue
        if t.dim() < 3 or t.shape[:-2] != q.shape[:-2] or t.shape[-1] != q.shape[-1]:
            raise ValueError(f"rms_norm_rope: {name} must be [..., heads, D] with q's leading shape and D")
        if t.shape[-2] < 1:
            raise ValueError(f"rms_norm_rope: {name} has no heads")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dim() != 1 or w.shape[0] != q.shape[-1]):
            raise ValueError(f"rms_norm_rope: {name} must be 1-D with D elements")
    if k is None and k_weight is not None:
        raise ValueError("rms_norm_rope: k_weight without k")
    _same("rms_norm_rope", q, k=k, q_weight=q_weight, k_weight=k_weight)
    if positions.shape != q.shape[:-2] or positions.dtype != torch.int64 or positions.device != q.device:
        raise ValueError("rms_norm_rope: positions must be int64 with q's leading shape, on its device")
    if inv_freq.dim() != 1 or inv_freq.dtype != torch.float64 or inv_freq.device != q.device:
        raise ValueError("rms_norm_rope: inv_freq must be a 1-D float64 tensor on q's device")
    if inv_freq.requires_grad and torch.is_grad_enabled():
        raise ValueError("rms_norm_rope is not differentiable by inv_freq")
    _no_tangents("rms_norm_rope", q, k, q_weight, k_weight, inv_freq)
    args = (q, k, q_weight, k_weight, positions, inv_freq, bool(interleaved), float(mscale), float(eps), bool(offset))
    if not _eager(q, k, q_weight, k_weight, positions, inv_freq):
        qo, ko = torch.ops.rmsnorm_gb300.rope_fwd(*args)
    elif _wants_grad(q, k, q_weight, k_weight):
        qo, ko = _RopeFunction.apply(*args)
    else:
        qo, ko = _rope_fwd_run(*args)
    return qo, ko if k is not None else None


class RMSNormRope(torch.nn.Module):
    """Norm and rotation of a layer's query and key heads: ``q, k = rope(q, k, positions)``.
    The weights are ones (zeros with ``offset``), one per kind of head; ``scaling`` and
    the arguments after it go to ``rope_frequencies``."""

    def __init__(self, head_dim: int, rotary_dim: Optional[int] = None, eps: float = 1e-6, offset: bool = False,
                 interleaved: bool = False, device=None, dtype=None, **frequencies):
        super().__init__()
        self.eps, self.offset, self.interleaved = eps, offset, interleaved
        init = torch.zeros if offset else torch.ones
        self.q_weight = torch.nn.Parameter(init(head_dim, device=device, dtype=dtype))
        self.k_weight = torch.nn.Parameter(init(head_dim, device=device, dtype=dtype))
        self.frequencies = dict(frequencies, rotary_dim=head_dim if rotary_dim is None else rotary_dim)
        inv_freq, self.mscale = rope_frequencies(device=self.q_weight.device, **self.frequencies)
        self.register_buffer("inv_freq", inv_freq, persistent=False)

    def _apply(self, fn, *args, **kwargs):
        # a change of the module's dtype leaves the frequencies in 64 bits, a move from
        # the meta device computes them
        inv_freq = self.inv_freq
        super()._apply(fn, *args, **kwargs)
        device = self.q_weight.device
        self.inv_freq = rope_frequencies(device=device, **self.frequencies)[0] if inv_freq.is_meta else inv_freq.to(device)
        return self

    def forward(self, q: torch.Tensor, k: torch.Tensor,
                positions: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
        return rms_norm_rope(q, k, self.q_weight, self.k_weight, positions, self.inv_freq, self.interleaved,
                             self.mscale, self.eps, self.offset)
