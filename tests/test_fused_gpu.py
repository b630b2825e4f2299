"""The operators of include/rmsnorm_fused.h on the GPU, against their formulas in 64
bits, within the bounds that fused_ref.py derives. Outputs lie between guard
elements and with gaps between rows where a pitch leaves them; both stay as they were."""
import pytest
import torch

from rmsnorm_fwd_bwd_gb300 import binding as B
from rmsnorm_fwd_bwd_gb300 import fused
from tests import fused_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = ["bfloat16", "float16", "float32"]
SENTINEL = -77.0
EPS = 1e-6


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Rows:
    """A matrix inside a larger buffer: ``shift`` elements off the buffer's start, rows
    ``gap`` elements further apart than their length; the rest holds a sentinel."""

    def __init__(self, M, N, dtype, shift=0, gap=0, data=None):
        self.ld = N + gap
        self.buf = torch.full((shift + M * self.ld + 64,), SENTINEL, dtype=torch.float32).to(dtype).cuda()
        self.t = self.buf[shift:shift + M * self.ld].view(M, self.ld)[:, :N]
        if data is not None:
            self.t.copy_(data)
        self.inside = torch.zeros(self.buf.shape, dtype=torch.bool, device="cuda")
        self.inside[shift:shift + M * self.ld].view(M, self.ld)[:, :N] = True

    def data_ptr(self):
        return self.t.data_ptr()

    def get(self):
        torch.cuda.synchronize()
        assert torch.all(self.buf[~self.inside].float() == SENTINEL), "written outside the rows"
        return self.t.cpu()


def layouts(name):
    """(shift, gap) of the tensors of a call."""
    return {"dense": lambda i: (0, 0), "shifted": lambda i: (1, 0), "mixed": lambda i: ((3 * i) % 8, (5 * i) % 7),
            "wide pitch": lambda i: (0, 8)}[name]


def randn(*shape, dtype, scale=1.0, seed=0):
    g = torch.Generator().manual_seed(1000 * seed + len(shape) + shape[-1])
    return (torch.randn(*shape, generator=g) * scale).to(ref.TYPES[dtype])


def weight(N, dtype, offset, seed=9):
    return (randn(N, dtype="float32", scale=0.1, seed=seed) + (0.0 if offset else 1.0)).to(ref.TYPES[dtype])


def state(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def run_add_fwd(x, res, w, dtype, offset=False, p=0.0, rng=None, layout="dense", want_h=True, stream=None):
    M, N = x.shape
    dt = ref.TYPES[dtype]
    at = layouts(layout)
    xr = Rows(M, N, dt, *at(0), data=x)
    rr = Rows(M, N, dt, *at(1), data=res) if res is not None else None
    hr = Rows(M, N, dt, *at(2)) if want_h else None
    yr = Rows(M, N, dt, *at(3))
    wr = Rows(1, N, dt, at(4)[0], 0, data=w)
    rstd = Rows(1, M, torch.float32)
    used = torch.full((2,), 99, dtype=torch.int64, device="cuda")
    st = B.rmsnorm_add_fwd(xr, xr.ld, rr, rr.ld if rr else 0, wr, hr, hr.ld if hr else 0, yr, yr.ld, rstd, M, N, EPS,
                           dtype, int(offset), p, rng, used, stream)
    assert st == 0, B.rmsnorm_status_string(st)
    assert torch.equal(xr.get().contiguous().view(torch.uint8), x.contiguous().view(torch.uint8))  # the bits, NaN too
    return yr.get(), hr.get() if hr else None, rstd.get()[0], used.cpu().tolist()


def check_add_fwd(x, res, w, dtype, y, h, r, offset=False, p=0.0, seed=0, ctr=0):
    dt = ref.TYPES[dtype]
    s, err = ref.add_sum(x, res, p, seed, ctr)
    if h is None:
        h = s.to(dt)
    else:
        ref.assert_close(h, s, err + ref.rounding(s.abs() + err, dt), "h")
    y64, r64 = ref.norm(h, w, EPS, offset)
    ref.assert_close(r, r64.squeeze(-1), ref.R_REL * r64.squeeze(-1), "rstd")
    ref.assert_close(y, y64, ref.Y_REL * y64.abs() + ref.rounding(y64.abs() * (1 + ref.Y_REL), dt), "y")


SHAPES = [(1, 1), (3, 2), (5, 7), (2, 8), (33, 64), (9, 65), (7, 128), (5, 129), (17, 256), (6, 257), (4, 511), (3, 512),
          (3, 1000), (5, 1024), (3, 1025), (2, 2051), (9, 4096), (3, 4099), (2, 5120), (3, 8192), (2, 8200), (2, 16383),
          (2, 16384)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", SHAPES)
def test_add_fwd_shapes(M, N, dtype):
    x, res, w = randn(M, N, dtype=dtype, seed=1), randn(M, N, dtype=dtype, scale=3.0, seed=2), weight(N, dtype, False)
    y, h, r, used = run_add_fwd(x, res, w, dtype)
    check_add_fwd(x, res, w, dtype, y, h, r)
    if dtype != "float32":
        assert torch.equal(h, (x.float() + res.float()).to(x.dtype))    # one rounding: the nearest
    assert used == [99, 99]                                             # untouched without dropout


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["shifted", "mixed", "wide pitch"])
@pytest.mark.parametrize("M,N", [(5, 64), (9, 65), (4, 512), (3, 1000), (5, 4099), (3, 4096), (2, 8200)])
def test_add_fwd_layouts(M, N, layout, dtype):
    x, res, w = randn(M, N, dtype=dtype, seed=3), randn(M, N, dtype=dtype, seed=4), weight(N, dtype, True)
    y, h, r, _ = run_add_fwd(x, res, w, dtype, offset=True, layout=layout)
    check_add_fwd(x, res, w, dtype, y, h, r, offset=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,layout", [(64, 96, "dense"), (7, 1001, "dense"), (5, 4096, "dense"), (4, 4099, "mixed"),
                                        (3, 16384, "dense")])
@pytest.mark.parametrize("p", [0.1, 0.9, 1.0])
def test_add_fwd_dropout(M, N, layout, p, dtype):
    seed, ctr = (7 << 40) + 123456789, (3 << 33) + 5
    x, res, w = randn(M, N, dtype=dtype, seed=5), randn(M, N, dtype=dtype, seed=6), weight(N, dtype, False)
    y, h, r, used = run_add_fwd(x, res, w, dtype, p=p, rng=state(seed, ctr), layout=layout)
    check_add_fwd(x, res, w, dtype, y, h, r, p=p, seed=seed, ctr=ctr)
    assert used == [seed, ctr]
    dropped = ~ref.kept(seed, ctr, M, N, p)
    assert torch.equal(h[dropped], res[dropped])                        # exactly the residual


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,p", [(4500, 1027, 0.0), (4099, 1035, 0.3), (4100, 2051, 0.0)])
def test_add_fwd_many_odd_rows(M, N, p, dtype):
    # blocks of several rows, the last ones without a full share
    x, res, w = randn(M, N, dtype=dtype, seed=91), randn(M, N, dtype=dtype, seed=92), weight(N, dtype, True)
    y, h, r, _ = run_add_fwd(x, res, w, dtype, offset=True, p=p, rng=state(3, 9))
    check_add_fwd(x, res, w, dtype, y, h, r, offset=True, p=p, seed=3, ctr=9)
    xr, rr = Rows(M, N, x.dtype, data=x), Rows(M, N, x.dtype, data=res)
    wt = w.cuda()
    assert B.rmsnorm_add_fwd(xr, N, rr, N, wt, rr, N, xr, N, None, M, N, EPS, dtype, 1, p, state(3, 9)) == 0
    assert torch.equal(rr.get(), h) and torch.equal(xr.get(), y)      # in place: the same bits


@pytest.mark.parametrize("dtype", DTYPES)
def test_add_fwd_without_residual_or_h(dtype):
    for N in (72, 4096, 4099):
        x, w = randn(5, N, dtype=dtype, seed=7), weight(N, dtype, False)
        y, h, r, _ = run_add_fwd(x, None, w, dtype)
        assert torch.equal(h, x)
        check_add_fwd(x, None, w, dtype, y, h, r)
        y2, h2, r2, _ = run_add_fwd(x, None, w, dtype, want_h=False)
        assert h2 is None and torch.equal(y, y2) and torch.equal(r, r2)


@pytest.mark.parametrize("N", [40, 1000, 4096, 4099, 16384])
def test_add_fwd_in_place(N):
    for dtype in DTYPES:
        x, res, w = randn(6, N, dtype=dtype, seed=8), randn(6, N, dtype=dtype, seed=9), weight(N, dtype, False)
        wt = w.cuda()

        def buffers():
            return Rows(6, N, x.dtype, 1, 3, data=x), Rows(6, N, x.dtype, 0, 0, data=res)
        (xr, rr), (yr, hr) = buffers(), buffers()           # outputs laid out as the inputs: the same sums, the same bits
        assert B.rmsnorm_add_fwd(xr, xr.ld, rr, rr.ld, wt, hr, hr.ld, yr, yr.ld, None, 6, N, EPS, dtype, 0) == 0
        y, h = yr.get(), hr.get()
        r = ref.norm(h, w, EPS)[1].squeeze(-1)
        check_add_fwd(x, res, w, dtype, y, h, r)
        assert B.rmsnorm_add_fwd(xr, xr.ld, rr, rr.ld, wt, rr, rr.ld, xr, xr.ld, None, 6, N, EPS, dtype, 0) == 0
        assert torch.equal(rr.get(), h) and torch.equal(xr.get(), y)


def test_add_fwd_special_values():
    for N in (48, 4096, 4099):
        x = randn(8, N, dtype="bfloat16", seed=10)
        res = randn(8, N, dtype="bfloat16", seed=11)
        x[0], res[0] = 0.0, 0.0                       # y = 0, r = 1 / sqrt(eps)
        x[1, 3] = float("inf")                        # h inf there, r = 0: y = 0 and NaN
        x[2, 5] = float("nan")                        # the whole row
        x[3], res[3] = 1e-20, 0.0                     # the square underflows, eps holds
        x[4] = torch.finfo(torch.bfloat16).min        # h overflows: every entry -inf
        res[4] = torch.finfo(torch.bfloat16).min
        w = weight(N, "bfloat16", False)
        y, h, r, _ = run_add_fwd(x, res, w, "bfloat16")
        assert torch.all(y[0] == 0) and abs(r[0].item() - 1000.0) < 1e-2
        assert h[1, 3] == float("inf") and r[1] == 0 and torch.isnan(y[1, 3]) and torch.all(y[1, :3] == 0)
        assert torch.isnan(y[2]).all() and torch.isnan(r[2])
        assert torch.isnan(y[4]).all() and torch.all(h[4] == -float("inf"))
        ok = [0, 3, 5, 6, 7]
        check_add_fwd(x[ok], res[ok], w, "bfloat16", y[ok], h[ok], r[ok])
        # a dropped element is 0 whatever it was
        x[:] = float("nan")
        y, h, r, _ = run_add_fwd(x[5:], res[5:], w, "bfloat16", p=1.0, rng=state(1, 1))
        assert torch.equal(h, res[5:])


# --------------------------------------------------------------------------- #
# add, backward
# --------------------------------------------------------------------------- #
def run_add_bwd(dy, dh, h, r, w, dtype, offset=False, p=0.0, rng=None, layout="dense", want=("dres", "dx"), ws_fill=255):
    M, N = dy.shape
    dt = ref.TYPES[dtype]
    at = layouts(layout)
    yr, hr = Rows(M, N, dt, *at(0), data=dy), Rows(M, N, dt, *at(1), data=h)
    er = Rows(M, N, dt, *at(2), data=dh) if dh is not None else None
    dres = Rows(M, N, dt, *at(3)) if "dres" in want else None
    dx = Rows(M, N, dt, *at(5)) if "dx" in want else None
    wr, dw = Rows(1, N, dt, at(4)[0], 0, data=w), Rows(1, N, dt, at(1)[0])
    rt = r.cuda()
    need = B.rmsnorm_add_bwd_workspace_size(M, N, dtype)
    ws = torch.full((need + 64,), ws_fill, dtype=torch.uint8, device="cuda")
    st = B.rmsnorm_add_bwd(yr, yr.ld, er, er.ld if er else 0, hr, hr.ld, wr, rt, dx, dx.ld if dx else 0, dres,
                           dres.ld if dres else 0, dw, M, N, dtype, int(offset), p, rng, ws, need)
    assert st == 0, B.rmsnorm_status_string(st)
    torch.cuda.synchronize()
    assert torch.all(ws[need:] == ws_fill), "written behind the workspace"
    return dres.get() if dres else None, dx.get() if dx else None, dw.get()[0]


def add_bwd_inputs(M, N, dtype, offset, seed=20):
    dy, dh = randn(M, N, dtype=dtype, scale=0.1, seed=seed), randn(M, N, dtype=dtype, scale=0.1, seed=seed + 1)
    h, w = randn(M, N, dtype=dtype, scale=2.0, seed=seed + 2), weight(N, dtype, offset)
    return dy, dh, h, ref.norm(h, w, EPS)[1].squeeze(-1).float(), w


def check_add_bwd(dy, dh, h, r, w, dtype, dres, dx, dw, offset=False, keep=None, p=0.0):
    dt = ref.TYPES[dtype]
    (d64, x64, w64), (ed, ex, ew) = ref.add_bwd(dy, dh, h, r, w, offset, keep, p)
    if dres is not None:
        ref.assert_close(dres, d64, ed + ref.rounding(d64.abs() + ed, dt), "dresidual")
    if dx is not None:
        ref.assert_close(dx, x64, ex + ref.rounding(x64.abs() + ex, dt), "dx")
    ref.assert_close(dw, w64, ew + ref.rounding(w64.abs() + ew, dt), "dgamma")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", SHAPES + [(3000, 40), (2500, 200), (1300, 1024), (1000, 1032), (700, 4099), (700, 4096)])
def test_add_bwd_shapes(M, N, dtype):
    a = add_bwd_inputs(M, N, dtype, False)
    dres, dx, dw = run_add_bwd(*a, dtype)
    check_add_bwd(*a, dtype, dres, dx, dw)
    assert torch.equal(dres, dx)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["shifted", "mixed", "wide pitch"])
@pytest.mark.parametrize("M,N", [(5, 64), (9, 65), (4, 512), (300, 1000), (400, 4099), (3, 4096), (2, 8200)])
def test_add_bwd_layouts(M, N, layout, dtype):
    a = add_bwd_inputs(M, N, dtype, True)
    dres, dx, dw = run_add_bwd(*a, dtype, offset=True, layout=layout)
    check_add_bwd(*a, dtype, dres, dx, dw, offset=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,layout", [(64, 96, "dense"), (7, 1001, "dense"), (400, 4096, "dense"), (4, 4099, "mixed"),
                                        (3, 16384, "dense")])
@pytest.mark.parametrize("p", [0.1, 1.0])
def test_add_bwd_dropout(M, N, layout, p, dtype):
    seed, ctr = (1 << 62) + 12345, 1 << 40
    a = add_bwd_inputs(M, N, dtype, False)
    keep = ref.kept(seed, ctr, M, N, p)
    dres, dx, dw = run_add_bwd(*a, dtype, p=p, rng=state(seed, ctr), layout=layout)
    check_add_bwd(*a, dtype, dres, dx, dw, keep=keep, p=p)
    assert torch.all(dx[~keep] == 0)


RING = [(1100, 1032), (1500, 2048), (1030, 4099), (1040, 5120), (1100, 8192), (1025, 8193), (1030, 12288), (1027, 301),
        (1500, 1001), (1029, 16384), (1024, 16381)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", RING)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_add_bwd_many_rows(M, N, p, dtype):
    # enough rows for the ring of staged rows, where one fits; few blocks have equally many
    a = add_bwd_inputs(M, N, dtype, True)
    keep = ref.kept(17, 3, M, N, p) if p else None
    dres, dx, dw = run_add_bwd(*a, dtype, offset=True, p=p, rng=state(17, 3))
    check_add_bwd(*a, dtype, dres, dx, dw, offset=True, keep=keep, p=p)
    again = run_add_bwd(*a, dtype, offset=True, p=p, rng=state(17, 3), ws_fill=0)
    assert all(torch.equal(u, v) for u, v in zip((dres, dx, dw), again))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["shifted", "mixed", "wide pitch"])
def test_add_bwd_many_rows_layouts(layout, dtype):
    for M, N, p in ((1100, 1032, 0.0), (1030, 2051, 0.3), (1030, 4096, 0.0)):
        a = add_bwd_inputs(M, N, dtype, False)
        keep = ref.kept(17, 3, M, N, p) if p else None
        dres, dx, dw = run_add_bwd(*a, dtype, p=p, rng=state(17, 3), layout=layout)
        check_add_bwd(*a, dtype, dres, dx, dw, keep=keep, p=p)


@pytest.mark.parametrize("M,N", [(1030, 4096), (1031, 1001)])
def test_add_bwd_many_rows_optional_tensors_and_in_place(M, N):
    dy, dh, h, r, w = add_bwd_inputs(M, N, "bfloat16", False)
    none = run_add_bwd(dy, None, h, r, w, "bfloat16")
    check_add_bwd(dy, None, h, r, w, "bfloat16", *none)
    full = run_add_bwd(dy, dh, h, r, w, "bfloat16")
    for want in (("dres",), ("dx",), ()):
        got = run_add_bwd(dy, dh, h, r, w, "bfloat16", want=want)
        assert all(v is None or torch.equal(u, v) for u, v in zip(full, got))
    wt, rt = w.cuda(), r.cuda()
    need = B.rmsnorm_add_bwd_workspace_size(M, N, "bfloat16")
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for k in (0, 1):
        t = [Rows(M, N, dy.dtype, data=v) for v in (dy, dh, h)]
        dw = torch.empty(N, dtype=dy.dtype, device="cuda")
        assert B.rmsnorm_add_bwd(t[0], N, t[1], N, t[2], N, wt, rt, None, 0, t[k], N, dw, M, N, "bfloat16", 0, 0.0, None, ws,
                                 need) == 0
        assert torch.equal(t[k].get(), full[0]) and torch.equal(dw.cpu(), full[2])


@pytest.mark.parametrize("N", [40, 4096, 4099])
def test_add_bwd_optional_tensors(N):
    for dtype in DTYPES:
        dy, dh, h, r, w = add_bwd_inputs(30, N, dtype, False)
        full = run_add_bwd(dy, dh, h, r, w, dtype)
        none = run_add_bwd(dy, None, h, r, w, dtype)
        check_add_bwd(dy, None, h, r, w, dtype, *none)
        only = run_add_bwd(dy, dh, h, r, w, dtype, want=("dres",))
        assert torch.equal(only[0], full[0]) and only[1] is None and torch.equal(only[2], full[2])
        only = run_add_bwd(dy, dh, h, r, w, dtype, want=("dx",))
        assert torch.equal(only[1], full[1]) and torch.equal(only[2], full[2])
        only = run_add_bwd(dy, dh, h, r, w, dtype, want=())
        assert torch.equal(only[2], full[2])
        # in place on dy, and on dh, against an output laid out as they are: the same sums, the same bits
        need = B.rmsnorm_add_bwd_workspace_size(30, N, dtype)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        wt, rt = w.cuda(), r.cuda()
        want = None
        for k in (None, 0, 1):
            t = [Rows(30, N, dy.dtype, 0, 3, data=v) for v in (dy, dh, h)]
            out = Rows(30, N, dy.dtype, 0, 3) if k is None else t[k]
            dw = torch.empty(N, dtype=dy.dtype, device="cuda")
            assert B.rmsnorm_add_bwd(t[0], t[0].ld, t[1], t[1].ld, t[2], t[2].ld, wt, rt, None, 0, out, out.ld, dw, 30, N,
                                     dtype, 0, 0.0, None, ws, need) == 0
            got = (out.get(), dw.cpu())
            if k is None:
                want = got
                check_add_bwd(dy, dh, h, r, w, dtype, got[0], None, got[1])
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_add_bwd_workspace_contents_do_not_matter_and_it_is_checked():
    for M, N in ((2500, 200), (700, 4099), (900, 4096)):
        a = add_bwd_inputs(M, N, "bfloat16", False)
        first = run_add_bwd(*a, "bfloat16")
        for fill in (0, 127):
            again = run_add_bwd(*a, "bfloat16", ws_fill=fill)
            assert all(torch.equal(p, q) for p, q in zip(first, again))
        t = [v.cuda() for v in a]
        out, dw = torch.full_like(t[0], 5), torch.full_like(t[4], 5)
        ws = torch.empty(16, dtype=torch.uint8, device="cuda")
        assert B.rmsnorm_add_bwd(t[0], N, t[1], N, t[2], N, t[4], t[3], None, 0, out, N, dw, M, N, "bfloat16", 0, 0.0, None,
                                 ws, 16) == 6
        assert torch.all(out == 5) and torch.all(dw == 5)


def test_no_rows():
    for dtype in DTYPES:
        dt = ref.TYPES[dtype]
        dw, w = torch.full((72,), 3.0, dtype=dt, device="cuda"), torch.ones(72, dtype=dt, device="cuda")
        assert B.rmsnorm_add_bwd_workspace_size(0, 72, dtype) == 0
        assert B.rmsnorm_add_bwd(None, 72, None, 72, None, 72, w, None, None, 72, None, 72, dw, 0, 72, dtype, 0, 0.0, None,
                                 None, 0) == 0
        assert torch.all(dw == 0)
        dw.fill_(3.0)
        sets = (B.RopeHeadsBwd * 1)(B.RopeHeadsBwd(None, 72, 72, None, 72, 72, w.data_ptr(), None, 72, 72, dw.data_ptr(), 1))
        assert B.rmsnorm_rope_bwd(sets, None, 0, 72, 8, None, 0, 1.0, EPS, dtype, 0, None, 0) == 0
        assert torch.all(dw == 0)


def test_add_bwd_of_rows_with_nan_stays_in_them():
    for N in (48, 4096, 4099):
        dy, dh, h, r, w = add_bwd_inputs(6, N, "float32", False)
        clean = run_add_bwd(dy, dh, h, r, w, "float32")
        dy2 = dy.clone()
        dy2[2, 1] = float("nan")
        got = run_add_bwd(dy2, dh, h, r, w, "float32")
        assert torch.isnan(got[0][2]).all()
        keep = [0, 1, 3, 4, 5]
        assert torch.equal(got[0][keep], clean[0][keep])
        assert torch.isnan(got[2]).sum() == 1 and torch.isnan(got[2][1])


def test_add_against_differences():
    """fp32: the kernels' loss at two points against the kernels' gradient."""
    for N in (41, 1600):
        M, step = 3, 2.0 ** -6
        x, res = randn(M, N, dtype="float32", seed=40), randn(M, N, dtype="float32", seed=41)
        w = weight(N, "float32", False)
        dy, dh, t = (randn(M, N, dtype="float32", seed=s) for s in (42, 43, 44))
        y, h, r, _ = run_add_fwd(x, res, w, "float32")
        dres, _, _ = run_add_bwd(dy, dh, h, r, w, "float32")

        def loss(v):
            y, h, _, _ = run_add_fwd(v, res, w, "float32")
            return (y.double() * dy.double()).sum() + (h.double() * dh.double()).sum(), \
                ((y.abs() * dy.abs()).sum() * (ref.Y_REL + ref.U) + (h.abs() * dh.abs()).sum() * 2 * ref.U).double()

        def loss64(v):
            s = v + res.double()
            return (ref.norm(s, w, EPS)[0] * dy.double()).sum() + (s * dh.double()).sum()
        hi, lo = (x.double() + step * t.double()).float(), (x.double() - step * t.double()).float()
        real = hi.double() - lo.double()                     # the step that fp32 took
        (a, ea), (b, eb) = loss(hi), loss(lo)
        want = (dres.double() * real).sum()
        # what the truncation of the difference makes, from the formula in 64 bits
        g64 = ref.add_bwd(dy, dh, x.double() + res.double(), ref.norm(x.double() + res.double(), w, EPS)[1].squeeze(-1), w)
        trunc = (loss64(hi.double()) - loss64(lo.double()) - (g64[0][0] * real).sum()).abs()
        assert abs(a - b - want) <= ea + eb + trunc + (g64[1][0] * real.abs()).sum() + 1e-5 * abs(want)


# --------------------------------------------------------------------------- #
# 8-bit output
# --------------------------------------------------------------------------- #
def run_quant(x, res, w, dtype, group, pow2, offset=False, layout="dense", want_h=True):
    M, N = x.shape
    dt = ref.TYPES[dtype]
    at = layouts(layout)
    n = -(-N // group) if group else 1
    xr = Rows(M, N, dt, *at(0), data=x)
    rr = Rows(M, N, dt, *at(1), data=res) if res is not None else None
    hr = Rows(M, N, dt, *at(2)) if want_h else None
    wr = Rows(1, N, dt, at(4)[0], 0, data=w)
    shift, gap = at(3)
    ldc, lds = N + gap, n + (0 if layout == "dense" else 3)
    codes = torch.full((shift + M * ldc + 64,), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((M * lds + 8,), SENTINEL, device="cuda")
    st = B.rmsnorm_quant_fwd(xr, xr.ld, rr, rr.ld if rr else 0, wr, hr, hr.ld if hr else 0, codes[shift:], ldc, scales, lds,
                             M, N, EPS, dtype, int(offset), group, int(pow2))
    assert st == 0, B.rmsnorm_status_string(st)
    torch.cuda.synchronize()
    c = codes[shift:shift + M * ldc].view(M, ldc)
    assert torch.all(codes[:shift] == 0x55) and torch.all(c[:, N:] == 0x55) and torch.all(codes[shift + M * ldc:] == 0x55)
    s = scales[:M * lds].view(M, lds)
    assert torch.all(s[:, n:] == SENTINEL) and torch.all(scales[M * lds:] == SENTINEL)
    return c[:, :N].contiguous().view(torch.float8_e4m3fn).cpu(), s[:, :n].cpu(), hr.get() if hr else None


def check_quant(x, res, w, dtype, codes, scales, h, group, pow2, offset=False):
    dt = ref.TYPES[dtype]
    s, err = ref.add_sum(x, res)
    want_h = s.to(dt)
    if h is not None:
        ref.assert_close(h, s, err + ref.rounding(s.abs() + err, dt), "h")
        want_h = h
    y, _ = ref.norm(want_h, w, EPS, offset)
    M, N = y.shape
    g = group or N
    n = -(-N // g)
    amax = torch.nn.functional.pad(y.abs(), (0, n * g - N)).view(M, n, g).amax(-1)
    s64 = (amax / 448.0).clamp_min(2.0 ** -126)
    rel = ref.Y_REL + 2 * ref.U
    if pow2:
        m, _ = torch.frexp(scales)
        assert torch.all(m == 0.5), "a scale is no power of two"
        assert torch.all(scales.double() >= s64 * (1 - rel)) and torch.all(scales.double() < 2 * s64 * (1 + rel))
    else:
        ref.assert_close(scales, s64, s64 * rel, "scales")
    wide = scales.double().repeat_interleave(g, dim=1)[:, :N]
    # e4m3 rounds by at most 2^-4 of the value, 2^-10 below the least normal number; y, 1 / scale
    # and the product are off by `rel` and three roundings before that
    off = (rel + 3 * ref.U) * y.abs()
    bound = off + torch.maximum((y.abs() + off) * 2.0 ** -4, wide * 2.0 ** -10)
    ref.assert_close(codes.float().double() * wide, y, bound, "codes")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("M,N", [(1, 1), (3, 31), (9, 64), (5, 200), (4, 512), (3, 1000), (5, 1024), (2, 1025), (3, 4096),
                                 (2, 4099), (2, 8192), (2, 16383), (2, 16384)])
def test_quant_shapes(M, N, group, dtype):
    x, res, w = randn(M, N, dtype=dtype, seed=50), randn(M, N, dtype=dtype, seed=51), weight(N, dtype, False)
    codes, scales, h = run_quant(x, res, w, dtype, group, False)
    check_quant(x, res, w, dtype, codes, scales, h, group, False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["shifted", "mixed", "wide pitch"])
@pytest.mark.parametrize("M,N", [(9, 64), (5, 200), (3, 1000), (3, 4096), (3, 4099), (2, 8200)])
def test_quant_layouts(M, N, layout, dtype):
    x, w = randn(M, N, dtype=dtype, seed=52), weight(N, dtype, True)
    for group, pow2, res in ((0, True, None), (64, True, randn(M, N, dtype=dtype, seed=53)), (128, False, None)):
        codes, scales, h = run_quant(x, res, w, dtype, group, pow2, True, layout, want_h=res is not None)
        check_quant(x, res, w, dtype, codes, scales, h, group, pow2, True)


def test_quant_special_values():
    for N in (160, 4096, 4099):
        x = randn(6, N, dtype="float32", seed=54)
        x[0] = 0.0                                     # codes 0, the least scale
        x[1, 70] = float("nan")                        # r is NaN: the whole row
        x[2, 70] = float("inf")                        # y = 0 but for a NaN
        x[3] = 1e-30                                   # y = 1e-27: scales far below fp32's usual
        w = weight(N, "float32", False)
        w[100] = float("inf")                          # y inf in the second group of 64
        codes, scales, _ = run_quant(x, None, w, "float32", 64, False, want_h=False)
        assert torch.all(codes[0, :64].float() == 0) and scales[0, 0] == 2.0 ** -126
        assert torch.isnan(codes[1].float()).all() and torch.isnan(scales[1]).all()
        assert torch.isnan(scales[2, 1]) and scales[2, 0] == 2.0 ** -126
        assert scales[4, 1] == float("inf") and torch.isnan(codes[4, 100].float()) and torch.all(codes[4, 64:100].float() == 0)
        ok = torch.ones(N, dtype=torch.bool)
        ok[64:128] = False
        wf = w.clone()
        wf[100] = 1.0
        rows = [0, 3, 4, 5]
        y, _ = ref.norm(x[rows], wf, EPS)
        got = codes.float()[rows].double() * scales[rows].double().repeat_interleave(64, dim=1)[:, :N]
        big = scales[rows].double().repeat_interleave(64, dim=1)[:, :N]
        bound = y.abs() * 2.0 ** -4 * (1 + 2.0 ** -16) + big * 2.0 ** -10
        ref.assert_close(got[:, ok], y[:, ok], bound[:, ok], "codes")


@pytest.mark.parametrize("group", [0, 32])
def test_quant_of_the_smallest_products(group):
    # h * g = 2^-140 k, k whole: exact in fp32, and r (2^40) restores y = 2^-100 k / 1.25 or so
    N = 64
    k = torch.tensor([0.0, 1.0, -1.0, 1.5] * 16)
    x, w = (k * 2.0 ** -40).unsqueeze(0), torch.full((N,), 2.0 ** -100)
    codes, scales, _ = (t.cpu() for t in fused.rms_norm_quant(x.cuda(), w.cuda(), 2.0 ** -100, group=group))
    y = x.double() * w.double() / (x.double().square().mean() + 2.0 ** -100).sqrt()
    s = scales.double().repeat_interleave(group or N, 1)
    # the largest value's code is 448; a code is off by half a step (2^-4 relative), the scale by
    # a few roundings
    assert torch.all((codes.float().double() * s - y).abs() <= y.abs() * (2.0 ** -4 + 2.0 ** -20))
    assert codes[0, 3].float().item() == 448.0 and codes[0, 0].float().item() == 0.0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,group", [(64, 8192, 128), (300, 4096, 0), (70, 4099, 64), (500, 520, 32), (40, 16384, 0)])
def test_quant_codes_are_the_nearest_but_at_the_borders(M, N, group, dtype):
    # y / scale comes out within 2 (Y_REL + 2 u) + 3 u < 70 u < 2^-17 of itself: a code may differ from the exactly rounded one
    # only where the exact quotient is that near to a border between two codes (products of
    # bf16 numbers lie exactly on one now and then), and is its neighbour there
    x, res, w = randn(M, N, dtype=dtype, seed=57), randn(M, N, dtype=dtype, seed=58), weight(N, dtype, False)
    codes, scales, h = run_quant(x, res, w, dtype, group, False)
    y, _ = ref.norm(h, w, EPS)
    g = group or N
    amax = torch.nn.functional.pad(y.abs(), (0, -N % g)).view(M, -1, g).amax(-1)
    q = y / (amax / 448.0).repeat_interleave(g, dim=1)[:, :N]
    got = codes.double()
    near, far = (q * (1 + s * 2.0 ** -17) for s in (-1, 1))
    low, high = (t.clamp(-448, 448).float().to(torch.float8_e4m3fn).double() for t in (near, far))
    assert torch.all((got == low) | (got == high))
    assert (low != high).double().mean() < 2e-3             # the others: exactly the nearest


def test_quant_rounds_to_even_and_uses_the_whole_range():
    # y is exactly x here up to r: rows scaled so that the codes before rounding are known
    N = 4096
    x = torch.zeros(1, N)
    x[0, 0], x[0, 1:9] = 448.0, torch.tensor([17.0, 19.0, -17.0, 0.0009765625 * 3, 432.0, 416.0, -448.0, 2.0 ** -10])
    codes, scales, _ = run_quant(x, None, torch.ones(N), "float32", 0, False, want_h=False)
    got = codes[0, :9].float().tolist()
    assert got[0] == 448.0 and got[7] == -448.0
    # 17 and 19 lie between 16, 18 and 20: half way up to fp32's rounding of y / scale
    assert got[1] in (16.0, 18.0) and got[2] in (18.0, 20.0) and got[6] == 416.0


# --------------------------------------------------------------------------- #
# rope
# --------------------------------------------------------------------------- #
class Heads:
    """[T, H, D] heads in one of the layouts a model has them in, between sentinels."""

    def __init__(self, T, H, D, dtype, how, data=None):
        dt = ref.TYPES[dtype]
        lead, tok, head = {"dense": (0, H * D, D), "fused": (2 * D, (H + 5) * D, D), "heads first": (0, D, T * D),
                           "spaced": (3, H * (D + 5) + 1, D + 5), "wide": (8, H * (D + 8), D + 8)}[how]
        self.buf = torch.full((lead + T * tok + H * head + D + 64,), SENTINEL, dtype=torch.float32).to(dt).cuda()
        self.t = self.buf.as_strided((T, H, D), (tok, head, 1), lead)
        if data is not None:
            self.t.copy_(data)
        mask = torch.zeros(self.buf.shape, dtype=torch.bool, device="cuda")
        mask.as_strided((T, H, D), (tok, head, 1), lead).fill_(True)
        self.mask = mask

    def get(self):
        torch.cuda.synchronize()
        assert torch.all(self.buf[~self.mask].float() == SENTINEL), "written outside the heads"
        return self.t.cpu()


def freqs(R, base=10000.0):
    return torch.tensor([base ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64)


def run_rope(xs, ws, pos, R, dtype, inter, mscale=1.0, offset=False, how="dense", freq=None):
    T, _, D = xs[0].shape
    freq = freqs(R) if freq is None else freq
    ins = [Heads(T, x.shape[1], D, dtype, how, data=x) for x in xs]
    outs = [Heads(T, x.shape[1], D, dtype, how) for x in xs]
    wt = [None if w is None else w.cuda() for w in ws]
    pt, ft = pos.cuda(), freq.cuda()
    sets = B.rope_heads([(i.t, w, o.t) for i, w, o in zip(ins, wt, outs)])
    st = B.rmsnorm_rope_fwd(sets, pt, T, D, R, ft, int(inter), mscale, EPS, dtype, int(offset))
    assert st == 0, B.rmsnorm_status_string(st)
    return [o.get() for o in outs]


def check_rope(xs, ws, pos, R, dtype, inter, outs, mscale=1.0, offset=False, freq=None):
    dt = ref.TYPES[dtype]
    for x, w, o in zip(xs, ws, outs):
        want, err = ref.rope_fwd(x, w, pos, freqs(R) if freq is None else freq, inter, mscale, EPS, offset)
        ref.assert_close(o, want, err + ref.rounding(want.abs() + err, dt), "rotated heads")


ROPE_SHAPES = [(1, 1, 1, 2, 2), (5, 3, 1, 8, 8), (3, 2, 2, 16, 16), (7, 4, 2, 64, 64), (6, 5, 1, 64, 32), (4, 8, 2, 80, 80),
               (4, 3, 3, 96, 48), (9, 7, 1, 128, 128), (3, 32, 8, 128, 128), (5, 2, 1, 128, 24), (3, 4, 4, 192, 128),
               (4, 3, 1, 256, 256), (2, 3, 1, 512, 512), (2, 2, 2, 512, 16), (5, 2, 1, 33, 32), (3, 2, 1, 77, 6),
               (4, 2, 1, 511, 510), (2, 5, 3, 90, 90), (2, 2, 2, 504, 16), (700, 5, 2, 64, 64), (3, 70, 9, 40, 16)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R", ROPE_SHAPES)
def test_rope_fwd_shapes(T, Hq, Hk, D, R, inter, dtype):
    xs = [randn(T, Hq, D, dtype=dtype, seed=60), randn(T, Hk, D, dtype=dtype, seed=61)]
    ws = [weight(D, dtype, False), weight(D, dtype, False, 8)]
    pos = torch.arange(T) * 37 + 5
    outs = run_rope(xs, ws, pos, R, dtype, inter)
    check_rope(xs, ws, pos, R, dtype, inter, outs)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("how", ["fused", "heads first", "spaced", "wide"])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_fwd_layouts(how, inter, dtype):
    for T, Hq, Hk, D, R in ((6, 3, 2, 64, 32), (5, 4, 1, 128, 128), (4, 3, 3, 36, 20)):
        xs = [randn(T, Hq, D, dtype=dtype, seed=62), randn(T, Hk, D, dtype=dtype, seed=63)]
        ws = [weight(D, dtype, True), None]
        pos = torch.tensor([3, 100000, 0, 1, 1, 7])[:T]
        outs = run_rope(xs, ws, pos, R, dtype, inter, mscale=1.25, offset=True, how=how)
        check_rope(xs, ws, pos, R, dtype, inter, outs, mscale=1.25, offset=True)


def test_rope_without_weights_and_with_one_set():
    for dtype in DTYPES:
        for D, R in ((64, 64), (50, 30)):
            x = [randn(9, 4, D, dtype=dtype, seed=64)]
            pos = torch.arange(9) - 4
            outs = run_rope(x, [None], pos, R, dtype, False)
            check_rope(x, [None], pos, R, dtype, False, outs)
            if R < D:
                assert torch.equal(outs[0][..., R:], x[0][..., R:])
            zero = run_rope(x, [None], torch.zeros(9, dtype=torch.int64), R, dtype, True)
            assert torch.equal(zero[0], x[0])


@pytest.mark.parametrize("inter", [False, True])
def test_rope_far_and_odd_positions_and_frequencies(inter):
    pos = torch.tensor([0, 1, -1, 131071, 1 << 20, (1 << 24) + 1, -(1 << 22), (1 << 26) - 1])
    x = [randn(8, 3, 64, dtype="float32", seed=65)]
    for D, freq in ((64, freqs(64)), (64, freqs(64) * 1e-3), (64, torch.tensor([3.0, 4.5, 1.0, -0.5] * 8, dtype=torch.float64)),
                    (64, torch.tensor([0.0, 2.0 ** -70, 1e-300, 0.999] * 8, dtype=torch.float64)), (42, freqs(30, 500000.0))):
        xs = [x[0][..., :D].contiguous()]
        outs = run_rope(xs, [None], pos, 2 * freq.numel(), "float32", inter, freq=freq)
        check_rope(xs, [None], pos, 2 * freq.numel(), "float32", inter, outs, freq=freq)
    # a period of exactly 2^10 positions: positions a period apart give the same bits, however far
    freq = torch.full((32,), 2 * torch.pi / 1024, dtype=torch.float64)
    far = torch.tensor([5, 5 + (1 << 10), 5 + (1 << 20)])
    xs = [randn(1, 2, 64, dtype="float32", seed=66).expand(3, 2, 64).contiguous()]
    outs = run_rope(xs, [None], far, 64, "float32", inter, freq=freq)
    # 2 pi / 1024 in 64 bits is off by 2^-53 of itself: 2^20 positions make that 2^-40 radians
    assert (outs[0][0] - outs[0][2]).abs().max() <= 8 * ref.U * xs[0].abs().max() * 2


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,R,base", [(64, 64, 500000.0), (128, 64, 1e7), (128, 24, 1e6), (50, 20, 1e6), (256, 256, 1e10)])
def test_rope_small_angles_to_the_last_bits(D, R, base, inter):
    # a pair (0, 1) becomes (-sin, cos), the backward's (sin, cos): relative to a small sine, too, only
    # roundings to fp32 count. The angle's words', the unit's and the sum's (3), the last step of
    # the sine's series and the rest of it (2), mscale's (1) and the output's (1), and one for
    # the terms left out: 8. Frequencies are off by 2^-63 turns, of at least 2^-37.
    pos = torch.tensor([0, 1, 2, 3, 17, 1000, -1, -5])
    freq = freqs(R, base)
    x = torch.zeros(len(pos), 2, D)
    second = torch.arange(1, R, 2) if inter else torch.arange(R // 2, R)
    first = second - (1 if inter else R // 2)
    x[..., second] = 1.0
    t = (pos.double().unsqueeze(-1) * freq).unsqueeze(1).expand(-1, 2, -1)
    near = t.abs() < 0.75
    assert near.sum() > 4 * R // 2 and (t[near].abs() > 0).any() and freq.min() > 2.0 ** -34
    q = x.cuda().requires_grad_()
    out, _ = fused.rms_norm_rope(q, None, None, None, pos.cuda(), freq.cuda(), inter)
    out.backward(x.cuda())
    out, back = out.detach().cpu().double(), q.grad.cpu().double()
    for got, sign in ((out, -1.0), (back, 1.0)):
        s, c = got[..., first], got[..., second]
        ref.assert_close(s[near], sign * torch.sin(t)[near], 8 * ref.U * torch.sin(t)[near].abs(), "sine")
        ref.assert_close(c[near], torch.cos(t)[near], 8 * ref.U * torch.cos(t)[near], "cosine")


@pytest.mark.parametrize("D,R", [(64, 64), (128, 32), (50, 20)])
def test_rope_in_place(D, R):
    for dtype in DTYPES:
        for inter in (False, True):
            xs = [randn(11, 5, D, dtype=dtype, seed=67), randn(11, 2, D, dtype=dtype, seed=68)]
            ws = [weight(D, dtype, False), weight(D, dtype, False, 8)]
            pos = torch.arange(11) * 1000
            want = run_rope(xs, ws, pos, R, dtype, inter, how="fused")
            t = [Heads(11, x.shape[1], D, dtype, "fused", data=x) for x in xs]
            wt, pt, ft = [w.cuda() for w in ws], pos.cuda(), freqs(R).cuda()
            sets = B.rope_heads([(h.t, w, h.t) for h, w in zip(t, wt)])
            assert B.rmsnorm_rope_fwd(sets, pt, 11, D, R, ft, int(inter), 1.0, EPS, dtype, 0) == 0
            assert torch.equal(t[0].get(), want[0]) and torch.equal(t[1].get(), want[1])


def run_rope_bwd(dys, xs, ws, pos, R, dtype, inter, mscale=1.0, offset=False, how="dense"):
    T, _, D = dys[0].shape
    dt = ref.TYPES[dtype]
    gs = [Heads(T, d.shape[1], D, dtype, "dense", data=d) for d in dys]
    ins = [Heads(T, x.shape[1], D, dtype, how, data=x) if w is not None else None for x, w in zip(xs, ws)]
    outs = [Heads(T, d.shape[1], D, dtype, how) for d in dys]
    wt = [None if w is None else w.cuda() for w in ws]
    dw = [None if w is None else Rows(1, D, dt) for w in ws]
    pt, ft = pos.cuda(), freqs(R).cuda()
    sets = B.rope_heads_bwd([(g.t, i.t if i else None, w, o.t, d) for g, i, w, o, d in zip(gs, ins, wt, outs, dw)])
    need = B.rmsnorm_rope_bwd_workspace_size(T, sum(d.shape[1] for d in dys), D, dtype)
    ws_t = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    st = B.rmsnorm_rope_bwd(sets, pt, T, D, R, ft, int(inter), mscale, EPS, dtype, int(offset), ws_t, need)
    assert st == 0, B.rmsnorm_status_string(st)
    torch.cuda.synchronize()
    assert torch.all(ws_t[need:] == 255), "written behind the workspace"
    return [o.get() for o in outs], [None if d is None else d.get()[0] for d in dw]


def check_rope_bwd(dys, xs, ws, pos, R, dtype, inter, dxs, dws, mscale=1.0, offset=False):
    dt = ref.TYPES[dtype]
    for dy, x, w, dx, dw in zip(dys, xs, ws, dxs, dws):
        (x64, w64), (ex, ew) = ref.rope_bwd(dy, x, w, pos, freqs(R), inter, mscale, EPS, offset)
        ref.assert_close(dx, x64, ex + ref.rounding(x64.abs() + ex, dt), "dx of the heads")
        if w is not None:
            ref.assert_close(dw, w64, ew + ref.rounding(w64.abs() + ew, dt), "dgamma of the heads")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R", ROPE_SHAPES)
def test_rope_bwd_shapes(T, Hq, Hk, D, R, inter, dtype):
    dys = [randn(T, Hq, D, dtype=dtype, seed=70), randn(T, Hk, D, dtype=dtype, seed=71)]
    xs = [randn(T, Hq, D, dtype=dtype, seed=72), randn(T, Hk, D, dtype=dtype, seed=73)]
    ws = [weight(D, dtype, False), weight(D, dtype, False, 8)]
    pos = torch.arange(T) * 37 + 5
    dxs, dws = run_rope_bwd(dys, xs, ws, pos, R, dtype, inter)
    check_rope_bwd(dys, xs, ws, pos, R, dtype, inter, dxs, dws)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("how", ["fused", "heads first", "spaced"])
def test_rope_bwd_layouts_and_weights(how, dtype):
    for T, Hq, Hk, D, R, inter in ((6, 3, 2, 64, 32, True), (5, 4, 1, 128, 128, False), (4, 3, 3, 36, 20, False)):
        dys = [randn(T, Hq, D, dtype=dtype, seed=74), randn(T, Hk, D, dtype=dtype, seed=75)]
        xs = [randn(T, Hq, D, dtype=dtype, seed=76), randn(T, Hk, D, dtype=dtype, seed=77)]
        w = [weight(D, dtype, True), weight(D, dtype, True, 8)]
        pos = torch.tensor([3, 100000, 0, 1, 1, 7])[:T]
        for ws in (w, [w[0], None], [None, w[1]], [None, None]):
            dxs, dws = run_rope_bwd(dys, xs, ws, pos, R, dtype, inter, 1.25, True, how)
            check_rope_bwd(dys, xs, ws, pos, R, dtype, inter, dxs, dws, 1.25, True)


# rows of whole octets whose halves do not meet octet by octet (partners through shared
# memory), with runs of several heads and without, and whole-octet halves with runs
SWAP_SHAPES = [(3, 2, 1, 8, 6), (3, 2, 1, 8, 2), (6, 3, 2, 24, 18), (5, 5, 1, 64, 62), (5, 3, 2, 72, 72), (4, 3, 1, 120, 8),
               (4, 9, 2, 128, 126), (4, 3, 1, 136, 134), (3, 2, 2, 256, 250), (3, 3, 1, 264, 2), (2, 2, 1, 512, 510),
               (21000, 9, 2, 64, 12), (7000, 7, 6, 128, 40), (2300, 21, 1, 200, 104), (7000, 7, 6, 128, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,Hq,Hk,D,R", SWAP_SHAPES)
def test_rope_of_halves_off_the_octets(T, Hq, Hk, D, R, dtype):
    xs = [randn(T, Hq, D, dtype=dtype, seed=100), randn(T, Hk, D, dtype=dtype, seed=101)]
    dys = [randn(T, Hq, D, dtype=dtype, seed=102), randn(T, Hk, D, dtype=dtype, seed=103)]
    pos = torch.arange(T) * 3 + 1
    for how, ws, offset in (("dense", [weight(D, dtype, False), weight(D, dtype, False, 8)], False),
                            ("wide", [None, weight(D, dtype, True)], True)):
        check_rope(xs, ws, pos, R, dtype, False, run_rope(xs, ws, pos, R, dtype, False, 1.25, offset, how), 1.25, offset)
        dxs, dws = run_rope_bwd(dys, xs, ws, pos, R, dtype, False, 1.25, offset, how)
        check_rope_bwd(dys, xs, ws, pos, R, dtype, False, dxs, dws, 1.25, offset)


@pytest.mark.parametrize("T,H", [(11, 5), (6000, 9)])
def test_rope_of_halves_off_the_octets_in_place(T, H):
    for dtype in DTYPES:
        D, R = 128, 40
        x, dy, w = randn(T, H, D, dtype=dtype, seed=104), randn(T, H, D, dtype=dtype, seed=105), weight(D, dtype, False)
        pos = torch.arange(T)
        want = run_rope([x], [w], pos, R, dtype, False)[0]
        want_d, want_w = run_rope_bwd([dy], [x], [w], pos, R, dtype, False)
        xt, dt, wt, pt, ft = x.cuda(), dy.cuda(), w.cuda(), pos.cuda(), freqs(R).cuda()
        dw = torch.empty_like(wt)
        ws = torch.empty(B.rmsnorm_rope_bwd_workspace_size(T, H, D, dtype), dtype=torch.uint8, device="cuda")
        assert B.rmsnorm_rope_bwd(B.rope_heads_bwd([(dt, xt, wt, dt, dw)]), pt, T, D, R, ft, 0, 1.0, EPS, dtype, 0, ws,
                                  ws.numel()) == 0
        assert B.rmsnorm_rope_fwd(B.rope_heads([(xt, wt, xt)]), pt, T, D, R, ft, 0, 1.0, EPS, dtype, 0) == 0
        assert torch.equal(dt.cpu(), want_d[0]) and torch.equal(dw.cpu(), want_w[0]) and torch.equal(xt.cpu(), want)


def test_rope_bwd_is_deterministic():
    T, H, D = 3000, 3, 128
    dys, xs = [randn(T, H, D, dtype="bfloat16", seed=78)], [randn(T, H, D, dtype="bfloat16", seed=79)]
    ws, pos = [weight(D, "bfloat16", False)], torch.arange(T)
    first = run_rope_bwd(dys, xs, ws, pos, 64, "bfloat16", False)
    again = run_rope_bwd(dys, xs, ws, pos, 64, "bfloat16", False)
    assert torch.equal(first[0][0], again[0][0]) and torch.equal(first[1][0], again[1][0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,R", [(64, 32), (64, 6), (128, 64), (50, 20), (128, 24)])
def test_rope_infinities_behind_the_rotated_entries_stay_where_they_are(D, R, inter, dtype):
    x, pos = randn(5, 3, D, dtype=dtype, seed=90), torch.arange(5) * 9 + 1
    bad = x.clone()
    for col, v in ((R, float("inf")), (D - 1, float("nan")), ((R + D) // 2, float("-inf"))):
        bad[2, 1, col] = v
    put = ~torch.isfinite(bad)
    for run in (lambda t: run_rope([t], [None], pos, R, dtype, inter)[0],
                lambda t: run_rope_bwd([t], [None], [None], pos, R, dtype, inter)[0][0]):
        want, got = run(x), run(bad)
        assert torch.equal(got[~put], want[~put])
        assert torch.equal(got[put].isnan(), bad[put].isnan())
        assert torch.equal(got[put][~bad[put].isnan()], bad[put][~bad[put].isnan()])


@pytest.mark.parametrize("inter", [False, True])
def test_rope_weight_gradient_of_infinite_cotangents(inter):
    # dgamma's columns add up products of their own column (and its pair's) alone
    D, R = 64, 16
    dy, x = randn(4, 2, D, dtype="float32", seed=91), randn(4, 2, D, dtype="float32", seed=92)
    w, pos = weight(D, "float32", False), torch.arange(4)
    bad = dy.clone()
    bad[1, 1, 40] = float("inf")
    want, got = (run_rope_bwd([d], [x], [w], pos, R, "float32", inter)[1][0] for d in (dy, bad))
    rest = torch.arange(D) != 40
    assert torch.equal(got[rest], want[rest]) and not torch.isfinite(got[40])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,R", [(64, 32), (64, 6), (128, 64), (128, 36), (50, 20), (128, 24), (256, 192)])
def test_rope_infinite_weights_behind_the_rotated_entries_stay_where_they_are(D, R, inter, dtype):
    x, dy = randn(5, 3, D, dtype=dtype, seed=93), randn(5, 3, D, dtype=dtype, seed=94)
    w, pos = weight(D, dtype, False), torch.arange(5) * 9 + 1
    bad = w.clone()
    for col, v in ((R, float("inf")), (D - 1, float("nan")), ((R + D) // 2, float("-inf"))):
        bad[col] = v
    put = ~torch.isfinite(bad)
    # both sets, one of them with the weight that is finite
    want = run_rope([x, x], [w, w], pos, R, dtype, inter)
    got = run_rope([x, x], [bad, w], pos, R, dtype, inter)
    assert torch.equal(got[1], want[1]) and torch.equal(got[0][..., ~put], want[0][..., ~put])
    assert torch.equal(got[0][..., put].isnan(), bad[put].isnan().expand(5, 3, -1))
    inf = torch.isinf(bad)
    assert torch.equal(got[0][..., inf], x[..., inf] * bad[inf])
    # the weight's gradient does not depend on the weight
    (_, want), (_, got) = (run_rope_bwd([dy], [x], [v], pos, R, dtype, inter) for v in (w, bad))
    assert torch.equal(got[0], want[0])


# --------------------------------------------------------------------------- #
# streams, graphs, offsets beyond 32 bits
# --------------------------------------------------------------------------- #
def test_on_another_stream_and_after_work_queued_on_it():
    N = 4096
    x, res, w = randn(64, N, dtype="bfloat16", seed=80), randn(64, N, dtype="bfloat16", seed=81), weight(N, "bfloat16", False)
    want, h_want, _, _ = run_add_fwd(x, res, w, "bfloat16")
    s = torch.cuda.Stream()
    xt, rt, wt = torch.zeros_like(x, device="cuda"), res.cuda(), w.cuda()
    y, h = torch.empty_like(xt), torch.empty_like(xt)
    xs = x.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(8):
            xt.copy_(xs)                                   # the kernel has to wait for this
            assert B.rmsnorm_add_fwd(xt, N, rt, N, wt, h, N, y, N, None, 64, N, EPS, "bfloat16", 0) == 0
            xt.zero_()                                     # and this for the kernel
    s.synchronize()
    assert torch.equal(y.cpu(), want) and torch.equal(h.cpu(), h_want)


@pytest.mark.parametrize("M,N", [(300, 4096), (50, 4099), (400, 200)])
def test_captured_forward_and_backward_draw_new_numbers(M, N):
    p, dtype = 0.25, "bfloat16"
    dt = torch.bfloat16
    x, res, w = randn(M, N, dtype=dtype, seed=82), randn(M, N, dtype=dtype, seed=83), weight(N, dtype, False)
    dy, dh = randn(M, N, dtype=dtype, seed=84), randn(M, N, dtype=dtype, seed=85)
    xt, rt, wt, dyt, dht = (v.cuda() for v in (x, res, w, dy, dh))
    y, h, dres, dx = (torch.empty(M, N, dtype=dt, device="cuda") for _ in range(4))
    rstd, dw = torch.empty(M, device="cuda"), torch.empty(N, dtype=dt, device="cuda")
    rng, used = state(5, 0), state(0, 0)
    need = B.rmsnorm_add_bwd_workspace_size(M, N, dtype)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step():
        assert B.rmsnorm_add_fwd(xt, N, rt, N, wt, h, N, y, N, rstd, M, N, EPS, dtype, 0, p, rng, used) == 0
        rng[1] += 1                                        # moves on before the backward
        assert B.rmsnorm_add_bwd(dyt, N, dht, N, h, N, wt, rstd, dx, N, dres, N, dw, M, N, dtype, 0, p, used, ws, need) == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    torch.cuda.synchronize()
    assert rng.tolist() == [5, 1]
    for k in range(1, 4):
        g.replay()
        torch.cuda.synchronize()
        check_add_fwd(x, res, w, dtype, y.cpu(), h.cpu(), rstd.cpu(), p=p, seed=5, ctr=k)
        check_add_bwd(dy, dh, h.cpu(), rstd.cpu(), w, dtype, dres.cpu(), dx.cpu(), dw.cpu(), keep=ref.kept(5, k, M, N, p), p=p)


def test_two_calls_at_once_on_two_streams():
    """Calls that may overlap, each with a workspace of its own, and other kernels between them."""
    M, N = 2000, 4096
    a = add_bwd_inputs(M, N, "bfloat16", False)
    want = run_add_bwd(*a, "bfloat16", p=0.1, rng=state(1, 2))
    t = [v.cuda() for v in a]
    need = B.rmsnorm_add_bwd_workspace_size(M, N, "bfloat16")
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    rng = state(1, 2)
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            o = [torch.empty_like(t[0]), torch.empty_like(t[0]), torch.empty(N, dtype=torch.bfloat16, device="cuda"),
                 torch.empty(need, dtype=torch.uint8, device="cuda")]
            for _ in range(5):
                o[3].fill_(255)
                assert B.rmsnorm_add_bwd(t[0], N, t[1], N, t[2], N, t[4], t[3], o[1], N, o[0], N, o[2], M, N, "bfloat16", 0, 0.1,
                                         rng, o[3], need) == 0
            outs.append(o)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0].cpu(), want[0]) and torch.equal(o[1].cpu(), want[1]) and torch.equal(o[2].cpu(), want[2])


def test_rows_beyond_32_bit_offsets():
    M, N = 140001, 16384                                    # 2.3e9 elements
    x = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    y, h = torch.empty_like(x), torch.empty_like(x)
    tail = randn(5, N, dtype="bfloat16", seed=86)
    x[-5:] = tail.cuda()
    w = weight(N, "bfloat16", False)
    wt, rstd = w.cuda(), torch.empty(M, device="cuda")
    p, seed = 0.1, 77
    assert B.rmsnorm_add_fwd(x, N, None, N, wt, h, N, y, N, rstd, M, N, EPS, "bfloat16", 0) == 0
    torch.cuda.synchronize()
    assert torch.equal(h[-5:].cpu(), tail) and torch.all(y[:1000] == 0)
    check_add_fwd(tail, None, w, "bfloat16", y[-5:].cpu(), h[-5:].cpu(), rstd[-5:].cpu())
    codes = torch.empty(M, N, dtype=torch.uint8, device="cuda")
    scales = torch.empty(M, 1, device="cuda")
    assert B.rmsnorm_quant_fwd(x, N, None, N, wt, None, N, codes, N, scales, 1, M, N, EPS, "bfloat16", 0) == 0
    check_quant(tail, None, w, "bfloat16", codes[-5:].view(torch.float8_e4m3fn).cpu(), scales[-5:].cpu(), None, 0, False)
    del codes
    # the backward: only the last rows have a cotangent
    y.zero_()
    dyt = randn(5, N, dtype="bfloat16", seed=87)
    y[-5:] = dyt.cuda()
    dres, dw = h, torch.empty(N, dtype=torch.bfloat16, device="cuda")
    need = B.rmsnorm_add_bwd_workspace_size(M, N, "bfloat16")
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert B.rmsnorm_add_bwd(y, N, None, N, x, N, wt, rstd, None, N, dres, N, dw, M, N, "bfloat16", 0, 0.0, None, ws, need) == 0
    torch.cuda.synchronize()
    check_add_bwd(dyt, None, tail, rstd[-5:].cpu(), w, "bfloat16", dres[-5:].cpu(), None, dw.cpu())
    assert torch.all(dres[:1000] == 0)
    # heads: a token stride of 16384 entries
    T, D = M, 64
    pos, f = torch.arange(T, device="cuda"), freqs(D).cuda()
    heads, out = x[:, :D].unflatten(1, (1, D)), y[:, :D].unflatten(1, (1, D))
    assert B.rmsnorm_rope_fwd(B.rope_heads([(heads, wt[:D], out)]), pos, T, D, D, f, 0, 1.0, EPS, "bfloat16", 0) == 0
    torch.cuda.synchronize()
    check_rope([tail[:, :D].unflatten(1, (1, D))], [w[:D]], pos[-5:].cpu(), D, "bfloat16", False, [out[-5:].cpu()])


def test_no_device_error():
    assert B.rmsnorm_device_error(clear=True) == 0
