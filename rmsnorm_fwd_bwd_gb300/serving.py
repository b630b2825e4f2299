"""PyTorch front end of the operators between an RMSNorm and an attention in serving
(``include/rmsnorm_serving.h``).

* ``quant_weight``: a weight as e4m3 codes with a scale per block of 128 x 128;
* ``quant_matmul``: the product of ``fused.rms_norm_quant``'s codes with such a weight;
  ``QuantLinear`` keeps one, ``RMSNormQuantLinear`` is the norm and the product together;
* ``rms_norm_rope_append``: norm and rotation of query and key heads, with keys and values
  written to the slots of a paged cache; ``PagedCache`` holds one,
  ``fused.RMSNormRope.append`` is the module's way to it.

They are custom ops (``rmsnorm_gb300::quant_weight`` and so on) for tracing and compilation;
eager calls run the same code at once, as in ``fused``. Everything runs on torch's current
stream of the inputs' device. Nothing here is differentiable.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import binding, fused
from .autograd import _after_op, _row_view, _rows
from .fused import _eager, _no_tangents, _on, _tokens, _wants_grad

CALLS = {"quant_weight": 0, "quant_matmul": 0, "rope_append": 0}
CODES = torch.float8_e4m3fn


def _done(status: int, where: str, counter: str) -> None:
    if status != binding.RMSNORM_OK:
        raise binding.RMSNormError(status, where)
    CALLS[counter] += 1
    _after_op()


def _blocks(n: int) -> int:
    return -(-n // 128)


# --------------------------------------------------------------------------- #
# weights
# --------------------------------------------------------------------------- #
def _quant_weight_run(weight, pow2):
    with _on(weight):
        w, ldw = _row_view(weight)
        N, K = weight.shape
        codes = torch.empty((N, K), dtype=CODES, device=weight.device)
        scales = torch.empty((_blocks(N), _blocks(K)), dtype=torch.float32, device=weight.device)
        _done(binding.rmsnorm_quant_weight(w, ldw, codes, K, scales, _blocks(K), N, K, weight.dtype, int(pow2)),
              "rmsnorm_quant_weight", "quant_weight")
    return codes, scales


@torch.library.custom_op("rmsnorm_gb300::quant_weight", mutates_args=())
def _quant_weight(weight: torch.Tensor, pow2: bool) -> tuple[torch.Tensor, torch.Tensor]:
    return _quant_weight_run(weight, pow2)


@_quant_weight.register_fake
def _(weight, pow2):
    N, K = weight.shape
    return weight.new_empty((N, K), dtype=CODES), weight.new_empty((_blocks(N), _blocks(K)), dtype=torch.float32)


def quant_weight(weight: torch.Tensor, pow2: bool = False) -> tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales) of a weight [N, K]: float8_e4m3fn codes [N, K] with a float32 scale per
    block of 128 x 128, [ceil(N / 128), ceil(K / 128)]; ``pow2`` rounds the scales up to powers
    of two. The values are codes * scales. They are those of the weight as it is, a parameter too:
    no gradient goes back to it."""
    if weight.dim() != 2 or weight.shape[1] < 1:
        raise ValueError("quant_weight: weight must be 2-D with at least one column")
    _no_tangents("quant_weight", weight)
    args = (weight.detach(), bool(pow2))
    return _quant_weight_run(*args) if _eager(weight) else torch.ops.rmsnorm_gb300.quant_weight(*args)


# --------------------------------------------------------------------------- #
# products
# --------------------------------------------------------------------------- #
def _quant_matmul_run(codes, scales, weight, weight_scales, bias, dtype):
    with _on(codes):
        a, lda = _row_view(codes)
        sa, ldas = _row_view(scales)
        b, ldb = _row_view(weight)
        sb, ldbs = _row_view(weight_scales)
        M, K = _rows(codes)
        N = weight.shape[0]
        y = torch.empty((*codes.shape[:-1], N), dtype=dtype, device=codes.device)
        group = 128 if scales.shape[-1] > 1 else 0
        _done(binding.rmsnorm_quant_matmul(a, lda, sa, ldas, b, ldb, sb, ldbs, None if bias is None else bias.contiguous(), y,
                                           N, M, N, K, dtype, group),
              "rmsnorm_quant_matmul", "quant_matmul")
    return y


@torch.library.custom_op("rmsnorm_gb300::quant_matmul", mutates_args=())
def _quant_matmul(codes: torch.Tensor, scales: torch.Tensor, weight: torch.Tensor, weight_scales: torch.Tensor,
                  bias: Optional[torch.Tensor], dtype: torch.dtype) -> torch.Tensor:
    return _quant_matmul_run(codes, scales, weight, weight_scales, bias, dtype)


@_quant_matmul.register_fake
def _(codes, scales, weight, weight_scales, bias, dtype):
    return codes.new_empty((*codes.shape[:-1], weight.shape[0]), dtype=dtype)


def quant_matmul(codes: torch.Tensor, scales: torch.Tensor, weight: torch.Tensor, weight_scales: torch.Tensor,
                 bias: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """[..., N] in ``dtype``: the rows codes * scales times the weight [N, K] of ``quant_weight``,
    plus bias [N] (of ``dtype``). codes [..., K] and scales [..., ceil(K / 128)] or [..., 1] are
    what ``rms_norm_quant`` returns with ``group`` 128 or 0. Sums in fp32. Not differentiable."""
    if codes.dtype != CODES or weight.dtype != CODES:
        raise ValueError("quant_matmul: codes and weight must be float8_e4m3fn")
    if scales.dtype != torch.float32 or weight_scales.dtype != torch.float32:
        raise ValueError("quant_matmul: scales must be float32")
    if weight.dim() != 2 or codes.dim() < 1 or codes.shape[-1] != weight.shape[1] or weight.shape[0] < 1 or weight.shape[1] < 1:
        raise ValueError("quant_matmul: codes must be [..., K] and weight [N, K]")
    N, K = weight.shape
    if scales.shape[:-1] != codes.shape[:-1] or scales.dim() != codes.dim() or scales.shape[-1] not in (1, _blocks(K)):
        raise ValueError("quant_matmul: scales must be [..., ceil(K / 128)] or [..., 1] with the codes' leading shape")
    if weight_scales.shape != (_blocks(N), _blocks(K)):
        raise ValueError("quant_matmul: weight_scales must be [ceil(N / 128), ceil(K / 128)]")
    if bias is not None and (bias.shape != (N,) or bias.dtype != dtype):
        raise ValueError("quant_matmul: bias must be [N] of the output's dtype")
    if any(t is not None and t.device != codes.device for t in (scales, weight, weight_scales, bias)):
        raise ValueError("quant_matmul: all tensors must share a device")
    if _wants_grad(codes, scales, weight, weight_scales, bias):
        raise ValueError("quant_matmul is not differentiable: use torch.no_grad()")
    _no_tangents("quant_matmul", scales, weight_scales, bias)
    args = (codes, scales.detach(), weight, weight_scales.detach(), None if bias is None else bias.detach(), dtype)
    return _quant_matmul_run(*args) if _eager(codes, scales, weight, weight_scales, bias) \
        else torch.ops.rmsnorm_gb300.quant_matmul(*args)


class QuantLinear(torch.nn.Module):
    """A linear layer with its weight in e4m3: ``y = layer(codes, scales)``. The codes and scales
    are buffers, and so is the bias; ``from_linear`` makes one of a ``torch.nn.Linear``."""

    def __init__(self, in_features: int, out_features: int, bias: bool = False, device=None, dtype=torch.bfloat16):
        super().__init__()
        self.out_dtype = dtype
        self.register_buffer("weight", torch.zeros((out_features, in_features), device=device).to(CODES))
        scales = torch.ones((_blocks(out_features), _blocks(in_features)), dtype=torch.float32, device=device)
        self.register_buffer("weight_scales", scales)
        self.register_buffer("bias", torch.zeros(out_features, dtype=dtype, device=device) if bias else None)

    def _apply(self, fn, *args, **kwargs):
        # a change of the module's dtype is one of its output's: codes and scales keep theirs
        scales = self.weight_scales

        def moved(t):
            if t.dtype != CODES:
                return fn(t)
            codes = t.view(torch.uint8)
            out = fn(codes)
            # (type() turns whole numbers into another type too: the codes only follow its device)
            return (out if out.dtype == torch.uint8 else codes.to(out.device)).view(CODES)
        super()._apply(moved, *args, **kwargs)
        if self.weight_scales.dtype != torch.float32:
            self.weight_scales = scales.to(self.weight_scales.device)
        # (an empty tensor of the output's dtype goes the way of the bias, which there may not be)
        self.out_dtype = fn(torch.empty(0, dtype=self.out_dtype, device=scales.device)).dtype
        return self

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear, pow2: bool = False) -> "QuantLinear":
        w = linear.weight.detach()
        made = cls(linear.in_features, linear.out_features, linear.bias is not None, w.device, w.dtype)
        made.weight, made.weight_scales = quant_weight(w, pow2)
        if linear.bias is not None:
            made.bias = linear.bias.detach().clone()
        return made

    def forward(self, codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
        return quant_matmul(codes, scales, self.weight, self.weight_scales, self.bias, self.out_dtype)


class RMSNormQuantLinear(torch.nn.Module):
    """Residual addition, RMSNorm and the 8-bit product behind it, for serving: ``y, h =
    layer(x, residual)``. ``norm_weight`` is the norm's (with ``offset`` 1 + it), ``linear`` a
    ``QuantLinear``; ``group`` 128 gives the rows a scale per 128 columns, 0 one."""

    def __init__(self, norm_weight: torch.Tensor, linear: QuantLinear, eps: float = 1e-6, offset: bool = False,
                 group: int = 128, pow2: bool = False):
        super().__init__()
        if group not in (0, 128):
            raise ValueError("RMSNormQuantLinear: group must be 0 (the row) or 128")
        self.eps, self.offset, self.group, self.pow2 = eps, offset, group, pow2
        self.register_buffer("norm_weight", norm_weight.detach())
        self.linear = linear

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> tuple[torch.Tensor, torch.Tensor]:
        codes, scales, h = fused.rms_norm_quant(x, self.norm_weight, self.eps, self.offset, residual, self.group, self.pow2)
        return self.linear(codes, scales), h


# --------------------------------------------------------------------------- #
# paged cache
# --------------------------------------------------------------------------- #
class PagedCache:
    """Keys and values of one layer in pages: ``k`` and ``v`` [pages, page_size, heads, D], and, with
    ``bits8``, e4m3 codes with the scales ``k_scales`` and ``v_scales`` [pages, page_size, heads]
    (else None). Slot s is row s % page_size of page s // page_size. ``heads_first`` lays a
    page's heads outside of its rows."""

    def __init__(self, pages: int, page_size: int, heads: int, head_dim: int, dtype=torch.bfloat16, bits8: bool = False,
                 heads_first: bool = False, device="cuda"):
        def rows(*shape, **kw):
            shape = (pages, heads, page_size, *shape) if heads_first else (pages, page_size, heads, *shape)
            t = torch.zeros(shape, device=device, **kw)
            return t.transpose(1, 2) if heads_first else t
        kind = CODES if bits8 else dtype
        self.k, self.v = (rows(head_dim, dtype=torch.uint8).view(CODES) if bits8 else rows(head_dim, dtype=kind)
                          for _ in range(2))
        self.k_scales, self.v_scales = (rows(dtype=torch.float32) if bits8 else None for _ in range(2))

    def rows(self, slots: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
        """Keys and values [..., heads, D] of the given slots, in float32 of an 8-bit cache. Slots
        below 0 (padded tokens) and behind the last, which have no row, give zeros."""
        none = (slots < 0) | (slots >= self.k.shape[0] * self.k.shape[1])
        at = slots.masked_fill(none, 0)
        page, row = at // self.k.shape[1], at % self.k.shape[1]
        none = none.unsqueeze(-1).unsqueeze(-1)

        def read(cache, scales):
            if scales is None:
                got = cache[page, row]
            else:
                got = cache.view(torch.uint8)[page, row].view(CODES).float() * scales[page, row].unsqueeze(-1)
            return got.masked_fill(none, 0.0)
        return read(self.k, self.k_scales), read(self.v, self.v_scales)


def _rope_append_run(q, k, v, q_weight, k_weight, positions, slots, inv_freq, k_cache, v_cache, k_scales, v_scales,
                     interleaved, mscale, eps, offset):
    with _on(k):
        D = k.shape[-1]
        pos, at, freq = positions.contiguous(), slots.contiguous(), inv_freq.contiguous()
        qo = torch.empty(q.shape if q is not None else (0,), dtype=k.dtype, device=k.device)
        keep = [None if t is None else _tokens(t) for t in (q, k, v)]
        wq, wk = (None if w is None else w.contiguous() for w in (q_weight, k_weight))
        _done(binding.rmsnorm_rope_append(
            None if q is None else binding.rope_heads([(keep[0], wq, _tokens(qo))]),
            binding.cache_heads(keep[1], wk, k_cache, k_scales),
            None if v is None else binding.cache_heads(keep[2], None, v_cache, v_scales), at, k_cache.shape[0],
            k_cache.shape[1], pos, pos.numel(), D, 2 * freq.numel(), freq, int(interleaved), mscale, eps, k.dtype,
            int(offset)), "rmsnorm_rope_append", "rope_append")
    return qo


@torch.library.custom_op("rmsnorm_gb300::rope_append", mutates_args=("k_cache", "v_cache", "k_scales", "v_scales"))
def _rope_append(q: Optional[torch.Tensor], k: torch.Tensor, v: Optional[torch.Tensor], q_weight: Optional[torch.Tensor],
                 k_weight: Optional[torch.Tensor], positions: torch.Tensor, slots: torch.Tensor, inv_freq: torch.Tensor,
                 k_cache: torch.Tensor, v_cache: Optional[torch.Tensor], k_scales: Optional[torch.Tensor],
                 v_scales: Optional[torch.Tensor], interleaved: bool, mscale: float, eps: float,
                 offset: bool) -> torch.Tensor:
    return _rope_append_run(q, k, v, q_weight, k_weight, positions, slots, inv_freq, k_cache, v_cache, k_scales, v_scales,
                            interleaved, mscale, eps, offset)


@_rope_append.register_fake
def _(q, k, v, q_weight, k_weight, positions, slots, inv_freq, k_cache, v_cache, k_scales, v_scales, interleaved, mscale,
      eps, offset):
    return k.new_empty(q.shape if q is not None else (0,))


def _check_cache(name, heads, cache, scales, size):
    if cache is None or cache.dim() != 4 or cache.shape[2:] != heads.shape[-2:] or cache.shape[0] < 1 or cache.shape[1] < 1:
        raise ValueError(f"rms_norm_rope_append: {name}_cache must be [pages, page_size, heads, D] with {name}'s heads and D")
    if cache.shape[-1] > 1 and cache.stride(-1) != 1:
        raise ValueError(f"rms_norm_rope_append: {name}_cache must have unit stride in D")
    if size is not None and cache.shape[:2] != size:
        raise ValueError("rms_norm_rope_append: both caches must have the same pages")
    if cache.dtype == CODES:
        if scales is None or scales.dtype != torch.float32 or scales.shape != cache.shape[:3]:
            raise ValueError(f"rms_norm_rope_append: an e4m3 {name}_cache needs float32 {name}_scales [pages, page_size, heads]")
    elif cache.dtype != heads.dtype or scales is not None:
        raise ValueError(f"rms_norm_rope_append: {name}_cache must be of {name}'s dtype, without scales, or float8_e4m3fn "
                         "with them")


def rms_norm_rope_append(q: Optional[torch.Tensor], k: torch.Tensor, v: Optional[torch.Tensor],
                         q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor], positions: torch.Tensor,
                         slots: torch.Tensor, inv_freq: torch.Tensor, k_cache: torch.Tensor,
                         v_cache: Optional[torch.Tensor] = None, k_scales: Optional[torch.Tensor] = None,
                         v_scales: Optional[torch.Tensor] = None, interleaved: bool = False, mscale: float = 1.0,
                         eps: float = 1e-6, offset: bool = False) -> Optional[torch.Tensor]:
    """The queries [..., heads, D], normalised and rotated as by ``fused.rms_norm_rope``; keys, so
    treated, and values [..., key heads, D] go to ``slots`` (int64, the leading shape, as
    ``positions``) of the caches [pages, page_size, key heads, D]: of the heads' dtype, or
    float8_e4m3fn with float32 scales [pages, page_size, key heads], one per head row. Slots
    below 0 (padded tokens) store nothing; the others must differ from each other. A slot
    behind the caches' last stores nothing and is reported by ``check_device_error``. q, and v with
    its cache, may be None. The caches are changed in place; not differentiable."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t is None:
            continue
        if t.dim() < 3 or t.shape[:-2] != k.shape[:-2] or t.shape[-1] != k.shape[-1] or t.shape[-2] < 1:
            raise ValueError(f"rms_norm_rope_append: {name} must be [..., heads, D] with k's leading shape and D")
        if t.dtype != k.dtype or t.device != k.device:
            raise ValueError(f"rms_norm_rope_append: k and {name} must share a dtype and a device")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.shape != k.shape[-1:] or w.dtype != k.dtype or w.device != k.device):
            raise ValueError(f"rms_norm_rope_append: {name} must be 1-D with D elements, of k's dtype and device")
    if q is None and q_weight is not None:
        raise ValueError("rms_norm_rope_append: q_weight without q")
    if (v is None) != (v_cache is None) or (v is None and v_scales is not None):
        raise ValueError("rms_norm_rope_append: v and v_cache go together")
    for name, t in (("positions", positions), ("slots", slots)):
        if t.shape != k.shape[:-2] or t.dtype != torch.int64 or t.device != k.device:
            raise ValueError(f"rms_norm_rope_append: {name} must be int64 with k's leading shape, on its device")
    if inv_freq.dim() != 1 or inv_freq.dtype != torch.float64 or inv_freq.device != k.device:
        raise ValueError("rms_norm_rope_append: inv_freq must be a 1-D float64 tensor on k's device")
    _check_cache("k", k, k_cache, k_scales, None)
    if v is not None:
        _check_cache("v", v, v_cache, v_scales, k_cache.shape[:2])
    changed = [t for t in (k_cache, v_cache, k_scales, v_scales) if t is not None]
    if any(t.device != k.device for t in changed):
        raise ValueError("rms_norm_rope_append: the caches must be on k's device")
    tensors = (q, k, v, q_weight, k_weight, inv_freq, *changed)
    if _wants_grad(*tensors):
        raise ValueError("rms_norm_rope_append is not differentiable: use torch.no_grad()")
    _no_tangents("rms_norm_rope_append", *(t for t in (q, k, v, q_weight, k_weight, inv_freq) if t is not None))
    args = (q, k, v, q_weight, k_weight, positions, slots, inv_freq, k_cache, v_cache, k_scales, v_scales,
            bool(interleaved), float(mscale), float(eps), bool(offset))
    if _eager(positions, slots, *tensors):
        out = _rope_append_run(*args)
        for t in changed:  # for whoever saved them for a backward
            if not t.is_inference():
                torch.autograd.graph.increment_version(t)
    else:
        out = torch.ops.rmsnorm_gb300.rope_append(*args)
    return None if q is None else out
