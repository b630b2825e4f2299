"""The operators around an RMSNorm in a transformer block, as cases to measure.

* ``add``: dropout of a sublayer's output, its addition to the residual stream and
  the RMSNorm of the sum (``fwd``), its gradients (``bwd``), and both through
  autograd (``step``);
* ``quant``: the same addition and norm for serving, with an 8-bit output and a
  scale per row or per group of columns;
* ``rope``: RMSNorm of every query and key head and the rotation of its first
  entries by the token's position (``fwd``), and its gradients (``bwd``).

``run`` computes a case with elementary torch operations, or, where ``own`` is true,
with this repository's entry points. ``exact`` computes it in 64 bits.

Definitions. s = D(x) + residual with D(x) = x * 65536 / (65536 - t) where the
element is kept and 0 where it is dropped, t = round(65536 p); an element is dropped
when its 16-bit random number is below t. Those are the low and high halves, in order,
of the four words that Philox4x32-10 gives for the counter (column // 8, row, offset
low, offset high) and the key (seed low, seed high): one call for 8 columns.
h = s rounded to the inputs' type, which is what the residual stream holds;
r = 1 / sqrt(mean(h^2) + eps), y = h r g with g = weight, or 1 + weight (``offset``). The
backward takes the h and r that the forward returned. 8-bit codes are y / scale, rounded
to nearest-even in e4m3, with scale = max|y| / 448 of the row or of the group of columns,
at least 2^-126. A rotation turns the pair (a, b) by the angle
position * inv_freq and multiplies it by ``mscale``; pairs are (2i, 2i + 1) or
(i, i + R/2) of the first R entries.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_EPS = 1e-6


def _add(name, direction, dtype, M, N, p, offset=False):
    case = {"op": "add", "dir": direction, "dtype": dtype, "M": M, "N": N, "p": p, "offset": offset}
    return dict(case, name=name) if name else case


def _quant(name, dtype, M, N, group, residual, offset=False):
    case = {"op": "quant", "dir": "fwd", "dtype": dtype, "M": M, "N": N, "group": group, "residual": residual,
            "offset": offset}
    return dict(case, name=name) if name else case


def _rope(name, direction, dtype, T, Hq, Hk, D, R, interleaved, far, offset=False):
    case = {"op": "rope", "dir": direction, "dtype": dtype, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R,
            "interleaved": interleaved, "far": far, "offset": offset}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one decoding step of a small batch: a few rows, latency is all that counts
        _add("add_fwd_decode", "fwd", "bf16", 8, 4096, 0.0),
        # training, the residual branch of a block with dropout
        _add("add_fwd_train", "fwd", "bf16", 16384, 4096, 0.1),
        # a width that is no multiple of 16 bytes: every row starts at another phase
        _add("add_fwd_odd", "fwd", "fp16", 8192, 4099, 0.0),
        # the largest training batch, with dropout: five tensors of 512 MiB
        _add("add_bwd_large", "bwd", "bf16", 65536, 4096, 0.1),
        # the odd width backward
        _add("add_bwd_odd", "bwd", "bf16", 8192, 4099, 0.0),
        # a training step's forward and backward through autograd, in full precision
        _add("add_step", "step", "fp32", 4096, 8192, 0.1, offset=True),
        # decoding a batch of 64 with 8-bit matrix products behind the norm
        _quant("quant_decode", "bf16", 64, 8192, 0, True),
        # a prompt, one scale per 128 columns
        _quant("quant_prompt", "bf16", 16384, 8192, 128, True),
        # one scale per row, no residual (the first norm of a model)
        _quant("quant_first", "fp16", 8192, 5120, 0, False),
        # decoding 64 sequences at far positions: 32 query and 8 key heads
        _rope("rope_decode", "fwd", "bf16", 64, 32, 8, 128, 128, False, True),
        # a long prompt, half of each head rotated, interleaved pairs
        _rope("rope_prompt", "fwd", "bf16", 32768, 32, 8, 128, 64, True, True),
        # the gradients for a training batch with wide heads
        _rope("rope_bwd", "bwd", "bf16", 16384, 16, 4, 256, 256, False, False),
    ]


def _spread(rng, lo, hi):
    """An integer in [lo, hi], uniform over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng):
    N = _spread(rng, 64, 16384)
    return N if rng.random() < 0.4 else max(64, N // 64 * 64)


def draw(rng):
    cap = work(_add(None, "bwd", "bf16", 65536, 4096, 0.1))["bytes"]
    op = rng.choice(["add", "add", "quant", "rope"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    offset = rng.random() < 0.3
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 128, 192, 256, 2 * rng.randint(8, 128)])
        R = D if rng.random() < 0.5 else 2 * rng.randint(1, D // 2)
        Hk = rng.choice([1, 2, 4, 8])
        case = _rope(None, rng.choice(["fwd", "bwd"]), dtype, _spread(rng, 1, 65536), Hk * rng.choice([1, 2, 4, 7, 8]),
                     Hk, D, R, rng.random() < 0.5, rng.random() < 0.5, offset)
        size = "T"
    elif op == "add":
        case = _add(None, rng.choice(["fwd", "bwd", "step"]), dtype, _spread(rng, 1, 65536), _width(rng),
                    rng.choice([0.0, 0.0, 0.1, 0.25]), offset)
        size = "M"
    else:
        case = _quant(None, dtype, _spread(rng, 1, 65536), _width(rng), rng.choice([0, 32, 64, 128]),
                      rng.random() < 0.7, offset)
        size = "M"
    scale = {"step": 0.3}.get(case["dir"], 0.6) * cap / work(case)["bytes"]
    if scale < 1:
        case[size] = max(1, int(case[size] * scale))
    return case


def work(case):
    s = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rope":
        T, H, D = case["T"], case["Hq"] + case["Hk"], case["D"]
        fwd = case["dir"] == "fwd"
        sides = 2 if fwd else 3                              # x, y or dy, x, dx
        return {"bytes": sides * T * H * D * s + (2 if fwd else 4) * D * s + 8 * T + 4 * case["R"],
                "flops": (8 if fwd else 20) * T * H * D}
    M, N = case["M"], case["N"]
    if case["op"] == "quant":
        sides = 3 if case["residual"] else 1                 # x, residual, h or x
        groups = -(-N // case["group"]) if case["group"] else 1
        return {"bytes": sides * M * N * s + M * N + 4 * M * groups + N * s, "flops": 8 * M * N}
    fwd = 4 * M * N * s + N * s + 4 * M                      # x, residual, h, y
    bwd = (5 if case["p"] else 4) * M * N * s + 2 * N * s + 4 * M  # dy, dh, h, dresidual, dx
    return {"fwd": {"bytes": fwd, "flops": 6 * M * N},
            "bwd": {"bytes": bwd, "flops": 12 * M * N},
            "step": {"bytes": fwd + bwd, "flops": 18 * M * N}}[case["dir"]]


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 62) + 17)


def _normal(gen, shape, dt, scale=1.0):
    t = torch.empty(shape, dtype=dt, device="cuda")
    t.normal_(0.0, scale, generator=gen)
    return t


def _weight(gen, n, dt, offset):
    return (_normal(gen, (n,), torch.float32, 0.1) + (0.0 if offset else 1.0)).to(dt)


def _stream_rows(gen, M, N, dt):
    """A residual stream: rows of different size, a few columns far larger than the rest."""
    t = _normal(gen, (M, N), dt)
    t.mul_(torch.exp(_normal(gen, (M, 1), torch.float32, 0.7)).to(dt))
    cols = torch.randint(0, N, (max(1, N // 512),), device="cuda", generator=gen)
    t[:, cols] *= 20.0
    return t


def prepare(case, seed):
    gen = _generator(seed)
    dt = _TYPES[case["dtype"]]
    st = {"case": case, "dt": dt}
    if case["op"] == "rope":
        T, Hq, Hk, D, R = (case[k] for k in ("T", "Hq", "Hk", "D", "R"))
        # q and k are parts of the fused projection's rows, as a model's are
        st["qkv"] = _normal(gen, (T, (Hq + 2 * Hk) * D), dt, 1.5)
        st["q"] = st["qkv"][:, :Hq * D].view(T, Hq, D)
        st["k"] = st["qkv"][:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        st["wq"] = _weight(gen, D, dt, case["offset"])
        st["wk"] = _weight(gen, D, dt, case["offset"])
        # far: sequences deep inside a long context, slowed four times for it
        base = torch.randint(0, 1 << 20, (1,), device="cuda", generator=gen) if case["far"] else 0
        order = torch.randperm(T, device="cuda", generator=gen) if T <= 256 else torch.arange(T, device="cuda")
        st["pos"] = order + base
        stretch = 4.0 if case["far"] else 1.0
        st["inv_freq"] = torch.tensor([10000.0 ** (-2.0 * i / R) / stretch for i in range(R // 2)],
                                      dtype=torch.float64, device="cuda")
        st["mscale"] = 0.1 * math.log(4.0) + 1.0 if case["far"] else 1.0
        if case["dir"] == "bwd":
            st["gq"] = _normal(gen, (T, Hq, D), dt, 0.01)
            st["gk"] = _normal(gen, (T, Hk, D), dt, 0.01)
        if own:
            _prepare_rope(st)
        return st
    M, N = case["M"], case["N"]
    st["w"] = _weight(gen, N, dt, case["offset"])
    st["res"] = _stream_rows(gen, M, N, dt) if case.get("residual", True) else None
    st["rng"] = torch.randint(0, 1 << 62, (2,), device="cuda", generator=gen)
    if case["dir"] == "bwd":
        st["h"] = st.pop("res")
        st["rstd"] = torch.empty(M, dtype=torch.float32, device="cuda")
        for a in range(0, M, 8192):
            st["rstd"][a:a + 8192] = (st["h"][a:a + 8192].double().square().mean(-1) + _EPS).rsqrt()
    else:
        st["x"] = _normal(gen, (M, N), dt, 0.5)
    if case["dir"] in ("bwd", "step"):
        st["dy"] = _normal(gen, (M, N), dt, 0.01)
        st["dh"] = _normal(gen, (M, N), dt, 0.01)
    if case["dir"] == "step":
        for key in ("x", "res", "w"):
            st[key].requires_grad_(True)
    elif own:
        _prepare_rows(st)
    return st


def _prepare_rows(st):
    """The outputs and the workspace that a user of the C entry points keeps."""
    from rmsnorm_fwd_bwd_gb300 import binding
    case, dt = st["case"], st["dt"]
    M, N = case["M"], case["N"]

    def rows():
        return torch.empty((M, N), dtype=dt, device="cuda")
    if case["op"] == "quant":
        groups = -(-N // case["group"]) if case["group"] else 1
        st["h"] = rows() if case["residual"] else None
        st["codes"] = torch.empty((M, N), dtype=torch.float8_e4m3fn, device="cuda")
        st["scales"] = torch.empty((M, groups), dtype=torch.float32, device="cuda")
    elif case["dir"] == "fwd":
        st["h"], st["y"] = rows(), rows()
        st["rstd"] = torch.empty(M, dtype=torch.float32, device="cuda")
    else:
        st["dres"] = rows()
        st["dx"] = rows() if case["p"] else None
        st["dw"] = torch.empty_like(st["w"])
        need = binding.rmsnorm_add_bwd_workspace_size(M, N, dt)
        st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")


def _prepare_rope(st):
    from rmsnorm_fwd_bwd_gb300 import binding
    case, dt = st["case"], st["dt"]
    st["oq"] = torch.empty(st["q"].shape, dtype=dt, device="cuda")
    st["ok"] = torch.empty(st["k"].shape, dtype=dt, device="cuda")
    if case["dir"] == "fwd":
        st["sets"] = binding.rope_heads([(st["q"], st["wq"], st["oq"]), (st["k"], st["wk"], st["ok"])])
        return
    st["dwq"], st["dwk"] = torch.empty_like(st["wq"]), torch.empty_like(st["wk"])
    st["sets"] = binding.rope_heads_bwd([(st["gq"], st["q"], st["wq"], st["oq"], st["dwq"]),
                                         (st["gk"], st["k"], st["wk"], st["ok"], st["dwk"])])
    need = binding.rmsnorm_rope_bwd_workspace_size(case["T"], case["Hq"] + case["Hk"], case["D"], dt)
    st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------------------- #
# plain forms
# --------------------------------------------------------------------------- #
_M32 = 0xFFFFFFFF


def _kept(rng, M, N, p):
    """Truth values [M, N] of the elements that dropout keeps."""
    nb = -(-N // 8)
    k0, k1 = rng[0] & _M32, (rng[0] >> 32) & _M32
    c0 = torch.arange(nb, device=rng.device).expand(M, nb)
    c1 = torch.arange(M, device=rng.device).view(M, 1).expand(M, nb)
    c2, c3 = (rng[1] & _M32).expand(M, nb), ((rng[1] >> 32) & _M32).expand(M, nb)
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57     # the 64-bit pattern is that of the unsigned product
        c0, c1, c2, c3 = ((b >> 32) & _M32) ^ c1 ^ k0, b & _M32, ((a >> 32) & _M32) ^ c3 ^ k1, a & _M32
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    words = torch.stack([c0, c1, c2, c3], dim=-1)
    halves = torch.stack([words & 0xFFFF, words >> 16], dim=-1).view(M, nb * 8)
    return halves[:, :N] >= round(65536 * p)


def _gain(w, offset):
    return w.float() + 1.0 if offset else w.float()


def _plain_sum(st, x, res):
    case = st["case"]
    s = x.float()
    if case.get("p"):
        t = round(65536 * case["p"])
        s = torch.where(_kept(st["rng"], case["M"], case["N"], case["p"]), s * (65536.0 / (65536 - t)), 0.0)
    return s if res is None else s + res.float()


def _plain_add_fwd(st, x, w, res):
    h = _plain_sum(st, x, res).to(st["dt"])
    r = 1.0 / torch.sqrt(h.float().square().mean(-1) + _EPS)
    y = h.float() * r.unsqueeze(-1) * _gain(w, st["case"]["offset"])
    return y.to(st["dt"]), h, r


def _plain_add_bwd(st, h, r, w):
    case, dt = st["case"], st["dt"]
    n = h.float() * r.unsqueeze(-1)
    dy = st["dy"].float()
    u = dy * _gain(w, case["offset"])
    d = st["dh"].float() + r.unsqueeze(-1) * (u - n * (u * n).mean(-1, keepdim=True))
    # a sum over tens of thousands of rows: in 64 bits
    dw = (dy * n).sum(0, dtype=torch.float64).to(dt)
    if not case["p"]:
        return d.to(dt), dw
    t = round(65536 * case["p"])
    kept = _kept(st["rng"], case["M"], case["N"], case["p"])
    return torch.where(kept, d * (65536.0 / (65536 - t)), 0.0).to(dt), d.to(dt), dw


def _plain_quant(st):
    case = st["case"]
    h = _plain_sum(st, st["x"], st["res"]).to(st["dt"])
    r = 1.0 / torch.sqrt(h.float().square().mean(-1, keepdim=True) + _EPS)
    y = h.float() * r * _gain(st["w"], case["offset"])
    M, N = y.shape
    group = case["group"] or N
    groups = -(-N // group)
    y = torch.nn.functional.pad(y, (0, groups * group - N)).view(M, groups, group)
    scales = (y.abs().amax(-1, keepdim=True) / 448.0).clamp_min(2.0 ** -126)
    codes = (y / scales).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(M, groups * group)[:, :N], scales.view(M, groups), h if case["residual"] else None


def _plain_turn(st, sign):
    """Cosine and sine [T, 1, R/2] of the angles; in 64 bits, for far positions."""
    angle = st["pos"].double().unsqueeze(-1) * st["inv_freq"]
    return ((angle.cos() * st["mscale"]).float().unsqueeze(1), (angle.sin() * (sign * st["mscale"])).float().unsqueeze(1))


def _plain_rotate(case, x, cos, sin):
    R = case["R"]
    if case["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([head, x[..., R:]], dim=-1)


def _plain_rope(st):
    case, dt = st["case"], st["dt"]
    fwd = case["dir"] == "fwd"
    cos, sin = _plain_turn(st, 1.0 if fwd else -1.0)
    outs = []
    for x, w, g in ((st["q"], st["wq"], st.get("gq")), (st["k"], st["wk"], st.get("gk"))):
        x, w = x.float(), _gain(w, case["offset"])
        r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + _EPS)
        n = x * r
        if fwd:
            outs.append(_plain_rotate(case, n * w, cos, sin).to(dt))
            continue
        v = _plain_rotate(case, g.float(), cos, sin)
        u = v * w
        outs.append((r * (u - n * (u * n).mean(-1, keepdim=True))).to(dt))
        outs.append((v * n).sum((0, 1), dtype=torch.float64).to(dt))
    return outs


def _run_plain(st):
    case = st["case"]
    if case["op"] == "rope":
        return _plain_rope(st)
    if case["op"] == "quant":
        return _plain_quant(st)
    if case["dir"] == "fwd":
        return _plain_add_fwd(st, st["x"], st["w"], st["res"])
    if case["dir"] == "bwd":
        return _plain_add_bwd(st, st["h"], st["rstd"], st["w"])
    x, w, res = (st[k].detach() for k in ("x", "w", "res"))
    y, h, r = _plain_add_fwd(st, x, w, res)
    grads = _plain_add_bwd(st, h, r, w)
    return [y, h] + ([grads[0]] + list(grads) if len(grads) == 2 else list(grads))


# --------------------------------------------------------------------------- #
# the framework's calls
# --------------------------------------------------------------------------- #
def _run_own(st):
    from rmsnorm_fwd_bwd_gb300 import binding as B
    case, dt = st["case"], st["dt"]
    if case["op"] == "rope":
        common = (st["pos"], case["T"], case["D"], case["R"], st["inv_freq"], case["interleaved"], st["mscale"], _EPS,
                  dt, case["offset"])
        if case["dir"] == "fwd":
            _ok(B.rmsnorm_rope_fwd(st["sets"], *common), "rmsnorm_rope_fwd")
            return [st["oq"], st["ok"]]
        _ok(B.rmsnorm_rope_bwd(st["sets"], *common, st["ws"], st["ws"].numel()), "rmsnorm_rope_bwd")
        return [st["oq"], st["dwq"], st["ok"], st["dwk"]]
    M, N = case["M"], case["N"]
    if case["op"] == "quant":
        _ok(B.rmsnorm_quant_fwd(st["x"], N, st["res"], N, st["w"], st["h"], N, st["codes"], N, st["scales"],
                                st["scales"].shape[1], M, N, _EPS, dt, case["offset"], case["group"], False),
            "rmsnorm_quant_fwd")
        return st["codes"], st["scales"], st["h"]
    if case["dir"] == "fwd":
        _ok(B.rmsnorm_add_fwd(st["x"], N, st["res"], N, st["w"], st["h"], N, st["y"], N, st["rstd"], M, N, _EPS, dt,
                              case["offset"], case["p"], st["rng"], None), "rmsnorm_add_fwd")
        return st["y"], st["h"], st["rstd"]
    if case["dir"] == "bwd":
        _ok(B.rmsnorm_add_bwd(st["dy"], N, st["dh"], N, st["h"], N, st["w"], st["rstd"], st["dx"], N, st["dres"], N,
                              st["dw"], M, N, dt, case["offset"], case["p"], st["rng"], st["ws"], st["ws"].numel()),
            "rmsnorm_add_bwd")
        return (st["dx"], st["dres"], st["dw"]) if case["p"] else (st["dres"], st["dw"])
    from rmsnorm_fwd_bwd_gb300 import fused
    y, h = fused.rms_norm_add(st["x"], st["res"], st["w"], _EPS, case["offset"], case["p"], st["rng"])
    grads = torch.autograd.grad([y, h], [st["x"], st["res"], st["w"]], [st["dy"], st["dh"]])
    return [y.detach(), h.detach()] + list(grads)


def _ok(status, what):
    if status:
        raise RuntimeError(f"{what}: status {status}")


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------- #
# 64 bits
# --------------------------------------------------------------------------- #
def _times32(a, c):
    """High and low words of the product of a 32-bit constant and 32-bit numbers, in 16-bit parts."""
    low = (c & 0xFFFF) * a
    mid = (c >> 16) * a + (low >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) + (low & 0xFFFF)


def _exact_drop(rng, v, p, first):
    """Dropout of the rows v, the first of which is row ``first``: [rows, N] in 64 bits."""
    rows, N = v.shape
    seed, off = (int(a) for a in rng.tolist())
    key = [seed % 2 ** 32, seed // 2 ** 32]
    ctr = [torch.arange((N + 7) // 8, device=v.device).repeat(rows, 1),
           torch.arange(first, first + rows, device=v.device).unsqueeze(1).repeat(1, (N + 7) // 8)]
    ctr += [torch.full_like(ctr[0], off % 2 ** 32), torch.full_like(ctr[0], off // 2 ** 32)]
    for i in range(10):
        hi0, lo0 = _times32(ctr[0], 0xD2511F53)
        hi1, lo1 = _times32(ctr[2], 0xCD9E8D57)
        ctr = [hi1.bitwise_xor(ctr[1]).bitwise_xor((key[0] + i * 0x9E3779B9) % 2 ** 32), lo1,
               hi0.bitwise_xor(ctr[3]).bitwise_xor((key[1] + i * 0xBB67AE85) % 2 ** 32), lo0]
    draws = torch.empty((rows, len(ctr) * 2, (N + 7) // 8), dtype=torch.int32, device=v.device)
    for i, word in enumerate(ctr):
        draws[:, 2 * i] = (word % 65536).int()
        draws[:, 2 * i + 1] = (word // 65536).int()
    dropped = (draws < round(65536 * p)).transpose(1, 2).reshape(rows, -1)[:, :N]
    return (v / (1.0 - round(65536 * p) / 65536)).masked_fill(dropped, 0.0)


def _exact_rows(st, first, last, w, grads, h=None, r=None):
    """y, s, r and the gradients of the rows [first, last); h, r: a saved forward."""
    case = st["case"]
    part = slice(first, last)
    out = {}
    if h is None:
        s = st["x"].detach()[part].double()
        if case.get("p"):
            s = _exact_drop(st["rng"], s, case["p"], first)
        if st.get("res") is not None:
            s = s.add(st["res"].detach()[part].double())
        out["s"] = s
        s = s.to(st["dt"]).double()
        r = torch.linalg.vecdot(s, s).div(s.shape[1]).add(_EPS).pow(-0.5)
        out["r"] = r
        out["y"] = torch.einsum("ij,i,j->ij", s, r, w)
    else:
        s, r = h[part].double(), r[part].double()
    if grads:
        dy = st["dy"][part].double()
        xhat = s.mul(r.view(-1, 1))
        u = dy.mul(w)
        along = torch.linalg.vecdot(u, xhat).div(s.shape[1])
        d = torch.addcmul(u, xhat, along.view(-1, 1), value=-1.0).mul_(r.view(-1, 1)).add_(st["dh"][part].double())
        out["dres"] = d
        out["dx"] = _exact_drop(st["rng"], d, case["p"], first) if case["p"] else d
        out["dw"] = torch.einsum("ij,ij->j", dy, xhat)
    return out


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    if case["op"] == "rope":
        return _exact_rope(st)
    M, N = case["M"], case["N"]
    w = st["w"].detach().double() + (1.0 if case["offset"] else 0.0)
    grads = case["dir"] in ("bwd", "step")
    chunk = max(1, (1 << 25) // N)
    parts = [_exact_rows(st, a, min(M, a + chunk), w, grads, st.get("h"), st.get("rstd")) for a in range(0, M, chunk)]
    got = {k: (sum(p[k] for p in parts) if k == "dw" else torch.cat([p[k] for p in parts])) for k in parts[0]}
    del parts
    if case["op"] == "quant":
        # the codes before their rounding
        parts = got["y"].split(case["group"] or N, dim=1)
        scales = [c.abs().amax(1, keepdim=True).div(448.0).clamp_min(2.0 ** -126) for c in parts]
        codes = torch.cat([c.div(f) for c, f in zip(parts, scales)], dim=1)
        return codes, torch.cat(scales, dim=1), got["s"] if case["residual"] else None
    if case["dir"] == "fwd":
        return got["y"], got["s"], got["r"]
    if case["dir"] == "bwd":
        return (got["dx"], got["dres"], got["dw"]) if case["p"] else (got["dres"], got["dw"])
    return [got["y"], got["s"], got["dx"], got["dres"], got["dw"]]


def _exact_rope(st):
    case = st["case"]
    T, D, R = case["T"], case["D"], case["R"]
    fwd = case["dir"] == "fwd"
    theta = torch.outer(st["pos"].double(), st["inv_freq"])
    turn = torch.polar(torch.full_like(theta, st["mscale"]), theta).unsqueeze(1)
    if not fwd:
        turn = turn.conj().resolve_conj()

    def rotated(v):
        pairs = v[..., :R].unflatten(-1, (R // 2, 2) if case["interleaved"] else (2, R // 2))
        if not case["interleaved"]:
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[first:last])
        if not case["interleaved"]:
            z = z.transpose(-1, -2)
        out = v.clone()
        out[..., :R] = z.flatten(-2)
        return out
    outs = []
    for x, w, g in ((st["q"], st["wq"], st.get("gq")), (st["k"], st["wk"], st.get("gk"))):
        w = w.double() + (1.0 if case["offset"] else 0.0)
        rows = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        dw = torch.zeros(D, dtype=torch.float64, device=x.device)
        chunk = max(1, (1 << 25) // (x.shape[1] * D))
        for first in range(0, T, chunk):
            last = min(T, first + chunk)
            v = x[first:last].double()
            r = (torch.linalg.vecdot(v, v) / D + _EPS).pow(-0.5).unsqueeze(-1)
            if fwd:
                rows[first:last] = rotated(v * r * w)
                continue
            back = rotated(g[first:last].double())
            xhat = v * r
            dw += torch.einsum("thd,thd->d", back, xhat)
            u = back * w
            rows[first:last] = r * (u - xhat * (torch.linalg.vecdot(u, xhat) / D).unsqueeze(-1))
        outs.append(rows)
        if not fwd:
            outs.append(dw)
    return outs
