"""The operators between an RMSNorm and an attention in serving, as cases to measure.

* ``matmul``: the product of e4m3 codes with scales, as the norm's 8-bit output has them,
  and a weight in e4m3 with a scale per block of 128 x 128;
* ``weight``: a weight matrix turned into those codes and scales;
* ``append``: RMSNorm of query and key heads, their rotation by the token's position, and
  keys and values written to the rows ("slots") of a paged cache, in their own type or as
  e4m3 codes with a scale per head row.

``run`` computes a case with elementary torch operations, or, where ``own`` is true,
with this repository's entry points. ``exact`` computes it in 64 bits.

Definitions. y[m, n] = sum over k of (a[m, k] * sa[m, k // 128]) * (b[n, k] * sb[n // 128,
k // 128]) + bias[n]; with ``group`` 0 a row of a has one scale. A scale is max|v| / 448 of its
block (or head row), at least 2^-126, with ``pow2`` rounded up to a power of two; a code is
v / scale rounded to nearest-even in e4m3. Head norm and rotation are those of
``operators.py``: n = x / sqrt(mean(x^2) + eps) * w, and the pair (a, b) of the first R entries
turned by position * inv_freq, both times mscale; pairs are (2i, 2i + 1) or (i, i + R / 2). Slot s
is row s % page_size of page s // page_size; a token with a negative slot is not
stored (its query is still rotated), and rows that no token names stay as they were.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_F8 = torch.float8_e4m3fn
_EPS = 1e-6
_LEAST = 2.0 ** -126


def _matmul(name, dtype, M, N, K, group, bias=False, pow2=False):
    case = {"op": "matmul", "dtype": dtype, "M": M, "N": N, "K": K, "group": group, "bias": bias, "pow2": pow2}
    return dict(case, name=name) if name else case


def _weight(name, dtype, N, K, pow2=False):
    case = {"op": "weight", "dtype": dtype, "N": N, "K": K, "pow2": pow2}
    return dict(case, name=name) if name else case


def _append(name, dtype, T, Hq, Hk, D, R, page, bits8, interleaved=False, far=False, heads_first=False, padded=False):
    case = {"op": "append", "dtype": dtype, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "page": page, "bits8": bits8,
            "interleaved": interleaved, "far": far, "heads_first": heads_first, "padded": padded}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one decoding step of 8 sequences: the fused projection of 32 query and 2 x 8 key and value heads
        _matmul("matmul_decode", "bf16", 8, 6144, 4096, 128),
        # decoding a batch of 64 behind the norm with a scale per row
        _matmul("matmul_batch", "bf16", 64, 8192, 8192, 0),
        # a short prompt into full precision, with a bias
        _matmul("matmul_short", "fp32", 2048, 4096, 5120, 128, bias=True, pow2=True),
        # codes of a width that is no multiple of 16 bytes: every row starts at another phase
        _matmul("matmul_odd", "fp16", 1001, 5120, 4099, 128),
        # a long prompt
        _matmul("matmul_prompt", "bf16", 16384, 8192, 8192, 128),
        # a layer's weight when a model is loaded
        _weight("weight_load", "bf16", 8192, 8192),
        # full precision, ragged blocks, scales of powers of two
        _weight("weight_odd", "fp32", 4099, 5000, pow2=True),
        # decoding 64 sequences at far positions
        _append("append_decode", "bf16", 64, 32, 8, 128, 128, 16, False, far=True),
        # decoding a larger batch into an 8-bit cache
        _append("append_decode_8bit", "bf16", 256, 32, 8, 128, 128, 64, True),
        # a long prompt into an 8-bit cache, half of each head rotated, interleaved pairs
        _append("append_prompt", "bf16", 32768, 32, 8, 128, 64, 64, True, interleaved=True, far=True),
        # wide heads, a cache with the heads outside a page's rows
        _append("append_wide", "fp16", 16384, 16, 4, 256, 256, 128, False, heads_first=True),
        # a padded batch, heads of 80 entries, pages of 48 rows
        _append("append_padded", "bf16", 8191, 28, 4, 80, 80, 48, False, padded=True),
    ]


def _spread(rng, lo, hi):
    """An integer in [lo, hi], uniform over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng):
    n = _spread(rng, 64, 16384)
    return n if rng.random() < 0.4 else max(64, n // 64 * 64)


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 3e15


def draw(rng):
    op = rng.choice(["matmul", "matmul", "weight", "append", "append"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "matmul":
        cap = _cost(_matmul(None, "bf16", 16384, 8192, 8192, 128))
        case = _matmul(None, dtype, _spread(rng, 1, 16384), _width(rng), _width(rng), rng.choice([0, 128, 128]),
                       rng.random() < 0.4, rng.random() < 0.3)
        size = "M"
    elif op == "weight":
        cap = _cost(_weight(None, "bf16", 8192, 8192))
        case = _weight(None, dtype, _width(rng), _width(rng), rng.random() < 0.3)
        size = "N"
    else:
        cap = _cost(_append(None, "bf16", 32768, 32, 8, 128, 64, 64, True))
        D = rng.choice([64, 80, 96, 128, 128, 192, 256, 2 * rng.randint(8, 128)])
        R = D if rng.random() < 0.5 else 2 * rng.randint(1, D // 2)
        Hk = rng.choice([1, 2, 4, 8])
        case = _append(None, dtype, _spread(rng, 1, 32768), Hk * rng.choice([1, 2, 4, 7, 8]), Hk, D, R,
                       rng.choice([1, 16, 32, 48, 64, 128, rng.randint(2, 300)]), rng.random() < 0.5,
                       rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.3)
        size = "T"
    scale = 0.6 * cap / _cost(case)
    if scale < 1:
        case[size] = max(1, int(case[size] * scale))
    return case


def _bytes(case):
    return 4 if case["dtype"] == "fp32" else 2


def work(case):
    s = _bytes(case)
    if case["op"] == "append":
        T, Hq, Hk, D = (case[k] for k in ("T", "Hq", "Hk", "D"))
        row = D + 4 if case["bits8"] else D * s                # a stored head row
        return {"bytes": T * (2 * Hq * D * s + 2 * Hk * (D * s + row) + 16) + 2 * D * s + 4 * case["R"],
                "flops": T * (8 * (Hq + Hk) * D + (4 if case["bits8"] else 0) * Hk * D)}
    N, K = case["N"], case["K"]
    blocks = -(-N // 128) * -(-K // 128)
    if case["op"] == "weight":
        return {"bytes": N * K * (s + 1) + 4 * blocks, "flops": 3 * N * K}
    M = case["M"]
    per_row = -(-K // 128) if case["group"] else 1
    return {"bytes": M * K + 4 * M * per_row + N * K + 4 * blocks + M * N * s + (N * s if case["bias"] else 0),
            "flops": 2 * M * N * K}


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 62) + 29)


def _normal(gen, shape, dt, scale=1.0):
    t = torch.empty(shape, dtype=dt, device="cuda")
    t.normal_(0.0, scale, generator=gen)
    return t


def _scales(amax, pow2):
    s = (amax / 448.0).clamp_min(_LEAST)
    return torch.exp2(torch.ceil(torch.log2(s.double()))).float() if pow2 else s


def _quantised_rows(v, group, pow2):
    """Codes and scales of the rows of v (fp32), one scale per group of columns."""
    M, K = v.shape
    n = -(-K // group)
    v = torch.nn.functional.pad(v, (0, n * group - K)).view(M, n, group)
    s = _scales(v.abs().amax(-1), pow2)
    codes = (v / s.unsqueeze(-1)).to(_F8).view(M, n * group)[:, :K]
    return codes.contiguous(), s


def _rows_of(gen, M, K):
    """Normalised rows: entries of size one, a few columns far larger, as a norm leaves them."""
    t = _normal(gen, (M, K), torch.float32)
    t[:, torch.randint(0, K, (max(1, K // 512),), device="cuda", generator=gen)] *= 20.0
    return t


def _matrix(gen, N, K, dt):
    """A weight: entries around 1 / sqrt(K), rows of different size."""
    t = _normal(gen, (N, K), torch.float32, K ** -0.5)
    t.mul_(torch.exp(_normal(gen, (N, 1), torch.float32, 0.5)))
    return t.to(dt)


def prepare(case, seed):
    gen = _generator(seed)
    dt = _TYPES[case["dtype"]]
    st = {"case": case, "dt": dt}
    if case["op"] == "append":
        return _prepare_append(st, gen)
    N, K = case["N"], case["K"]
    if case["op"] == "weight":
        st["w"] = _matrix(gen, N, K, dt)
        if own:
            st["codes"] = torch.empty((N, K), dtype=_F8, device="cuda")
            st["scales"] = torch.empty((-(-N // 128), -(-K // 128)), dtype=torch.float32, device="cuda")
        return st
    M = case["M"]
    st["a"] = torch.empty((M, K), dtype=_F8, device="cuda")
    st["sa"] = torch.empty((M, -(-K // case["group"]) if case["group"] else 1), dtype=torch.float32, device="cuda")
    for first in range(0, M, 4096):
        rows = slice(first, min(M, first + 4096))
        st["a"][rows], st["sa"][rows] = _quantised_rows(_rows_of(gen, st["a"][rows].shape[0], K), case["group"] or K,
                                                        case["pow2"])
    st["b"], st["sb"] = _plain_weight(_matrix(gen, N, K, torch.bfloat16), case["pow2"])
    st["bias"] = _normal(gen, (N,), dt, 0.2) if case["bias"] else None
    if own:
        st["y"] = torch.empty((M, N), dtype=dt, device="cuda")
    return st


def _prepare_append(st, gen):
    case, dt = st["case"], st["dt"]
    T, Hq, Hk, D, R, page = (case[k] for k in ("T", "Hq", "Hk", "D", "R", "page"))
    # q, k and v are parts of the fused projection's rows, as a model's are
    st["qkv"] = _normal(gen, (T, (Hq + 2 * Hk) * D), dt, 1.5)
    st["q"] = st["qkv"][:, :Hq * D].view(T, Hq, D)
    st["k"] = st["qkv"][:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    st["v"] = st["qkv"][:, (Hq + Hk) * D:].view(T, Hk, D)
    st["wq"] = (_normal(gen, (D,), torch.float32, 0.1) + 1.0).to(dt)
    st["wk"] = (_normal(gen, (D,), torch.float32, 0.1) + 1.0).to(dt)
    # pages for the tokens and for what sequences hold already, handed out in any order
    pages = -(-T // page) + -(-min(T + 4096, 16384) // page) + 1
    order = torch.randperm(pages, device="cuda", generator=gen)
    at = torch.arange(T, device="cuda") + page // 3            # the first sequence starts inside a page
    slots = order[at // page] * page + at % page
    if T <= 256:                                                # decoding: every token in a page of its own sequence
        at = torch.randperm(pages * page, device="cuda", generator=gen)[:T]
        slots = at
    if case["padded"]:
        # sequences of different lengths in a padded batch: the ends of some have no slot
        length = max(1, T // 7)
        ends = torch.randint(1, length + 1, (-(-T // length),), device="cuda", generator=gen)
        t = torch.arange(T, device="cuda")
        slots = torch.where(t % length < ends[t // length], slots, -1)
    st["slots"], st["pages"] = slots, pages
    base = torch.randint(0, 1 << 20, (1,), device="cuda", generator=gen) if case["far"] else 0
    st["pos"] = torch.arange(T, device="cuda") + base
    stretch = 4.0 if case["far"] else 1.0
    st["inv_freq"] = torch.tensor([10000.0 ** (-2.0 * i / R) / stretch for i in range(R // 2)], dtype=torch.float64,
                                  device="cuda")
    st["mscale"] = 0.1 * math.log(4.0) + 1.0 if case["far"] else 1.0
    shape = (pages, Hk, page, D) if case["heads_first"] else (pages, page, Hk, D)
    for name in ("kc", "vc"):
        cache = _normal(gen, shape, torch.float32 if case["bits8"] else dt, 60.0 if case["bits8"] else 1.0)
        st[name + "_all"] = cache.to(_F8) if case["bits8"] else cache
        st[name + "_scales_all"] = None
        if case["bits8"]:
            st[name + "_scales_all"] = torch.rand(shape[:3], device="cuda", generator=gen) * 0.02 + 0.001
        # [pages, page, heads, D], whatever lies outside of what
        for part in ("", "_scales"):
            t = st[name + part + "_all"]
            st[name + part] = t.transpose(1, 2) if t is not None and case["heads_first"] else t
    if own:
        from rmsnorm_fwd_bwd_gb300 import binding as B
        st["oq"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
        st["q_heads"] = B.rope_heads([(st["q"], st["wq"], st["oq"])])
        st["k_heads"] = B.cache_heads(st["k"], st["wk"], st["kc"], st["kc_scales"])
        st["v_heads"] = B.cache_heads(st["v"], None, st["vc"], st["vc_scales"])
    return st


# --------------------------------------------------------------------------- #
# plain forms
# --------------------------------------------------------------------------- #
def _spread_blocks(s, N, K):
    return s.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def _plain_weight(w, pow2):
    N, K = w.shape
    n, k = -(-N // 128), -(-K // 128)
    w = w.float()
    blocks = torch.nn.functional.pad(w, (0, k * 128 - K, 0, n * 128 - N)).view(n, 128, k, 128)
    s = _scales(blocks.abs().amax((1, 3)), pow2)
    return (w / _spread_blocks(s, N, K)).to(_F8), s


def _plain_matmul(st):
    case = st["case"]
    K = case["K"]
    sa = st["sa"].repeat_interleave(128, 1)[:, :K] if case["group"] else st["sa"]
    a = st["a"].float() * sa
    b = st["b"].float() * _spread_blocks(st["sb"], case["N"], K)
    y = a @ b.t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return y.to(st["dt"])


def _plain_heads(st, x, w):
    case = st["case"]
    R = case["R"]
    x = x.float()
    x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + _EPS) * w.float()
    # in 64 bits, for far positions
    angle = st["pos"].double().unsqueeze(-1) * st["inv_freq"]
    cos, sin = ((f * st["mscale"]).float().unsqueeze(1) for f in (angle.cos(), angle.sin()))
    if case["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([head, x[..., R:]], dim=-1)


def _plain_append(st):
    case, dt = st["case"], st["dt"]
    stored = st["slots"] >= 0
    slots = st["slots"][stored]
    page, row = slots // case["page"], slots % case["page"]
    for name, rows in (("kc", _plain_heads(st, st["k"], st["wk"])), ("vc", st["v"].float())):
        rows = rows[stored]
        if case["bits8"]:
            s = _scales(rows.abs().amax(-1), False)
            st[name].view(torch.uint8)[page, row] = (rows / s.unsqueeze(-1)).to(_F8).view(torch.uint8)
            st[name + "_scales"][page, row] = s
        else:
            st[name][page, row] = rows.to(dt)
    return _appended(st, _plain_heads(st, st["q"], st["wq"]).to(dt))


def _appended(st, q):
    out = [q, st["kc"], st["vc"]]
    return out + [st["kc_scales"], st["vc_scales"]] if st["case"]["bits8"] else out


# --------------------------------------------------------------------------- #
# the framework's calls
# --------------------------------------------------------------------------- #
def _run_own(st):
    from rmsnorm_fwd_bwd_gb300 import binding as B
    case, dt = st["case"], st["dt"]
    if case["op"] == "append":
        _ok(B.rmsnorm_rope_append(st["q_heads"], st["k_heads"], st["v_heads"], st["slots"], st["pages"], case["page"],
                                  st["pos"], case["T"], case["D"], case["R"], st["inv_freq"], case["interleaved"],
                                  st["mscale"], _EPS, dt, False), "rmsnorm_rope_append")
        return _appended(st, st["oq"])
    N, K = case["N"], case["K"]
    if case["op"] == "weight":
        _ok(B.rmsnorm_quant_weight(st["w"], K, st["codes"], K, st["scales"], st["scales"].shape[1], N, K, dt,
                                   case["pow2"]), "rmsnorm_quant_weight")
        return st["codes"], st["scales"]
    _ok(B.rmsnorm_quant_matmul(st["a"], K, st["sa"], st["sa"].shape[1], st["b"], K, st["sb"], st["sb"].shape[1],
                               st["bias"], st["y"], N, case["M"], N, K, dt, case["group"]), "rmsnorm_quant_matmul")
    return st["y"]


def _ok(status, what):
    if status:
        raise RuntimeError(f"{what}: status {status}")


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "matmul":
        return _plain_matmul(state)
    if case["op"] == "weight":
        return _plain_weight(state["w"], case["pow2"])
    return _plain_append(state)


# --------------------------------------------------------------------------- #
# 64 bits
# --------------------------------------------------------------------------- #
def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    return {"matmul": _exact_matmul, "weight": _exact_weight, "append": _exact_append}[case["op"]](st)


def _exact_scale(amax, pow2):
    s = torch.clamp(amax / 448.0, min=_LEAST)
    if pow2:
        m, e = torch.frexp(s)                                 # s = m * 2^e with m in [1/2, 1)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    return s


def _exact_weight(st):
    """Codes before their rounding, and the scales."""
    w = st["w"].double()
    codes, scales = [], []
    for rows in w.split(128, 0):
        parts = rows.split(128, 1)
        s = [_exact_scale(p.abs().max(), st["case"]["pow2"]) for p in parts]
        codes.append(torch.cat([p / f for p, f in zip(parts, s)], 1))
        scales.append(torch.stack(s))
    return torch.cat(codes), torch.stack(scales)


def _exact_matmul(st):
    case = st["case"]
    M, N, K = case["M"], case["N"], case["K"]
    b = st["b"].double()
    for i in range(0, N, 128):
        for j in range(0, K, 128):
            b[i:i + 128, j:j + 128] *= st["sb"][i // 128, j // 128].double()
    y = torch.empty((M, N), dtype=torch.float64, device="cuda")
    for first in range(0, M, 4096):
        rows = slice(first, min(M, first + 4096))
        a = st["a"][rows].double()
        for j in range(0, K, 128):
            a[:, j:j + 128] *= st["sa"][rows, j // 128 if case["group"] else 0].double().unsqueeze(1)
        torch.mm(a, b.t(), out=y[rows])
    return y if st["bias"] is None else y.add_(st["bias"].double())


def _exact_append(st):
    case = st["case"]
    T, R = case["T"], case["R"]
    theta = torch.outer(st["pos"].double(), st["inv_freq"])
    turn = torch.polar(torch.full_like(theta, st["mscale"]), theta).unsqueeze(1)

    def heads(x, w):
        out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 25) // (x.shape[1] * x.shape[2]))
        for first in range(0, T, step):
            part = slice(first, min(T, first + step))
            v = x[part].double()
            v = torch.einsum("thd,th,d->thd", v, (torch.linalg.vecdot(v, v) / v.shape[2] + _EPS).pow(-0.5), w.double())
            pairs = v[..., :R].unflatten(-1, (R // 2, 2) if case["interleaved"] else (2, R // 2))
            if not case["interleaved"]:
                pairs = pairs.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[part])
            if not case["interleaved"]:
                z = z.transpose(-1, -2)
            v[..., :R] = z.flatten(-2)
            out[part] = v
        return out

    tokens = torch.nonzero(st["slots"] >= 0).flatten()
    slots = st["slots"][tokens]
    caches, scales = [], []
    for name, rows in (("kc", heads(st["k"], st["wk"])), ("vc", st["v"].double())):
        cache = st[name].double()
        rows = rows[tokens]
        if case["bits8"]:
            s = _exact_scale(rows.abs().amax(-1), False)
            rows = rows / s.unsqueeze(-1)                     # codes before their rounding
            all_scales = st[name + "_scales"].double()
            all_scales[torch.div(slots, case["page"], rounding_mode="floor"), slots.remainder(case["page"])] = s
            scales.append(all_scales)
        cache[torch.div(slots, case["page"], rounding_mode="floor"), slots.remainder(case["page"])] = rows
        caches.append(cache)
    return [heads(st["q"], st["wq"])] + caches + scales
