"""The operators of include/rmsnorm_fused.h from their formulas in 64 bits (torch on
the CPU, Philox in numpy), and bounds on what fp32 arithmetic with one rounding at
the end may be off. Shares no code with the library.

A rounding to nearest is off by at most u = 2^-24 of the value in fp32 and by
half_step(T) of it in T. The bounds count those: a row's sums take at most DEPTH
additions one after the other (up to 32 products by a thread, 5 levels of lanes, 5
of warps), so a sum is off by at most DEPTH * u times the sum of its terms'
magnitudes; r = 1 / sqrt(sum / N + eps) by half of that plus the division, the
addition, the root and the quotient.
"""
import numpy as np
import torch

U = 2.0 ** -24
DEPTH = 44
R_REL = (DEPTH / 2 + 4) * U           # relative error of r
Y_REL = R_REL + 4 * U                 # of (h * r) * (1 + gamma) before its rounding
TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(v, dtype):
    """What rounding v to dtype may be off: half a step, or half the least subnormal."""
    if dtype == torch.float32:
        return v.abs() * U + 2.0 ** -150
    fi = torch.finfo(dtype)
    return v.abs() * half_step(dtype) + fi.tiny * fi.eps / 2


def philox(counter, key, rounds=10):
    """Philox4x32 on uint32 arrays (Salmon et al. 2011): counter [..., 4], key (k0, k1)."""
    c = [np.asarray(counter[..., i], dtype=np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    low = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    for _ in range(rounds):
        a = np.uint64(0xD2511F53) * c[0]
        b = np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> s32) ^ c[1] ^ np.uint64(k0), b & low, (a >> s32) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, axis=-1).astype(np.uint32)


def threshold(p):
    return int(np.floor(65536.0 * float(np.float32(p)) + 0.5))


def kept(seed, offset, M, N, p):
    """Truth values [M, N]: the elements that dropout keeps."""
    nb = (N + 7) // 8
    ctr = np.zeros((M, nb, 4), dtype=np.uint32)
    ctr[..., 0] = np.arange(nb)[None, :]
    ctr[..., 1] = np.arange(M)[:, None]
    ctr[..., 2] = offset & 0xFFFFFFFF
    ctr[..., 3] = (offset >> 32) & 0xFFFFFFFF
    w = philox(ctr, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    halves = np.stack([w & np.uint32(0xFFFF), w >> np.uint32(16)], axis=-1).reshape(M, nb * 8)
    return torch.from_numpy(halves[:, :N] >= threshold(p))


def drop_scale(p):
    t = threshold(p)
    return 65536.0 / (65536 - t) if t < 65536 else 0.0


def gain(w, offset):
    return w.double() + (1.0 if offset else 0.0)


def add_sum(x, res, p=0.0, seed=0, offset=0):
    """s [M, N] before its rounding, and the bound on fp32's error before the rounding."""
    s = x.double()
    err = torch.zeros_like(s)
    if threshold(p):
        k = kept(seed, offset, *x.shape, p)
        s = torch.where(k, s * drop_scale(p), torch.zeros((), dtype=torch.float64))
        err = 2 * U * s.abs()                       # the scale's rounding and the product's
    if res is not None:
        s = s + res.double()
        err = err + U * s.abs()
    return s, err


def norm(h, w, eps, offset=False):
    """y and r [M, 1] of the rows h, in 64 bits."""
    h = h.double()
    r = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
    return h * r * gain(w, offset), r


def add_bwd(dy, dh, h, r, w, offset=False, keep=None, p=0.0):
    """dresidual, dx and dgamma in 64 bits and the bounds on their errors before the
    rounding; r is the saved one, [M]."""
    dy, h, r = dy.double(), h.double(), r.double().unsqueeze(-1)
    dh = torch.zeros_like(h) if dh is None else dh.double()
    g = gain(w, offset)
    n = h * r
    u = dy * g
    c = (u * n).mean(-1, keepdim=True)
    c_abs = (u * n).abs().mean(-1, keepdim=True)
    d = dh + r * (u - n * c)
    # roundings: n, u (with 1 + gamma) and n * c, the difference, the product with r and the
    # sum; and c's, a sum of products of three rounded factors
    e = U * (dh.abs() + d.abs() + r.abs() * (6 * u.abs() + 8 * (n * c).abs() + n.abs() * (DEPTH + 8) * c_abs))
    dw = (dy * n).sum(0)
    # the rows one after the other and the column reduction
    dw_err = U * (h.shape[0] + 40) * (dy * n).abs().sum(0)
    dx, ex = d, e
    if keep is not None:
        dx = torch.where(keep, d * drop_scale(p), torch.zeros((), dtype=torch.float64))
        ex = torch.where(keep, (e + 2 * U * d.abs()) * drop_scale(p), torch.zeros((), dtype=torch.float64))
    return (d, dx, dw), (e, ex, dw_err)


def rotate(z, pos, inv_freq, interleaved, mscale, sign=1.0):
    """z [T, H, D] turned, and sum of the magnitudes of each output's two terms."""
    R = 2 * inv_freq.numel()
    t = pos.double().unsqueeze(-1) * inv_freq.double()
    c, s = (mscale * torch.cos(t)).unsqueeze(1), (sign * mscale * torch.sin(t)).unsqueeze(1)
    out, mag = z.clone(), z.abs()
    ia = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    ib = ia + 1 if interleaved else ia + R // 2
    a, b = z[..., ia], z[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    mag[..., ia] = mag[..., ib] = abs(mscale) * (a.abs() + b.abs())
    return out, mag


# cos and sin: the angle is off by at most 2^-25 half turns (its rounding to fp32) and
# 2^-32 turns, in all below 2^-23 radians; the function by less than 2^-23, the product
# with mscale by u
TURN = 2.0 ** -23 + 2.0 ** -23 + 2 * U


def own_angle(pos, inv_freq):
    """What the product in 64 bits may leave the oracle's own angles off by."""
    return 2.0 ** -53 * float(pos.double().abs().max() * inv_freq.abs().max())


def rope_fwd(x, w, pos, inv_freq, interleaved, mscale, eps, offset=False):
    """The output in 64 bits and the bound on its error before the rounding."""
    z = x.double()
    rel = 0.0
    if w is not None:
        z, _ = norm(z, w, eps, offset)
        rel = Y_REL
    out, mag = rotate(z, pos, inv_freq, interleaved, mscale)
    return out, mag * (rel + TURN + own_angle(pos, inv_freq) + 3 * U)


def rope_bwd(dy, x, w, pos, inv_freq, interleaved, mscale, eps, offset=False):
    """(dx, dgamma) in 64 bits and the bounds on their errors before the rounding."""
    v, mag = rotate(dy.double(), pos, inv_freq, interleaved, mscale, -1.0)
    ev = mag * (TURN + own_angle(pos, inv_freq) + 3 * U)
    if w is None:
        return (v, None), (ev, None)
    x = x.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    g = gain(w, offset)
    n, u, eu = x * r, v * g, ev * g.abs()
    c = (u * n).mean(-1, keepdim=True)
    c_abs = (u * n).abs().mean(-1, keepdim=True)
    c_err = (DEPTH + 8) * U * c_abs + (eu * n.abs()).mean(-1, keepdim=True) + 2 * R_REL * c_abs
    d = r * (u - n * c)
    e = U * d.abs() + r * (eu + (6 * U + R_REL) * (u.abs() + (n * c).abs()) + (R_REL + 4 * U) * (n * c).abs()
                           + n.abs() * c_err)
    terms = (v * n).reshape(-1, x.shape[-1])
    dw = terms.sum(0)
    dw_err = (U * (terms.shape[0] + 40) + R_REL) * terms.abs().sum(0) + (ev * n.abs()).reshape(-1, x.shape[-1]).sum(0)
    return (d, dw), (e, dw_err)


def assert_close(got, want, err, what):
    """|got - want| <= err everywhere, both finite in the same places."""
    got, want = got.detach().cpu().double(), want.detach().cpu().double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= err.cpu())
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at {i}: got "
                             f"{got.flatten()[i].item()!r}, want {want.flatten()[i].item()!r}, bound "
                             f"{err.expand_as(want).flatten()[i].item():.3g}")
