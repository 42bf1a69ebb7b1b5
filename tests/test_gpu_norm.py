"""add_rmsnorm_mxfp8 and its backward against plain 64-bit implementations.

Tolerances.  u = 2^-24.  The sum of n squares is formed by at most 16 sequential fma per thread and piece (n / T
terms) and a tree; its relative error is at most (n / T + 16) u <= 80 u, halved by the square root; mean, eps, root
and reciprocal add 3 u and y's two products 2 u: below 2^-18 in all.  Backward: each term of the row mean has a
relative error of 4 u, summed like the squares: |c error| <= 100 u * mean|g xh|; dr's three terms are rounded a few
times each.  dw: a thread adds rows / 304 (or / 2432) terms in order, then at most 304 partial sums: error at most
(rows / 304 + 320) u * sum|terms|."""
import ctypes

import numpy as np
import pytest
import torch

import mx64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
REL = 2.0 ** -18
EPS = 1e-6
SHAPES = [(1, 32), (1, 4096), (3, 64), (9, 288), (130, 1024), (5, 1056), (7, 2080), (33, 4096), (700, 512), (6, 8192),
          (2, 16384), (3, 8224)]


@pytest.fixture(scope="module")
def pmn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


def f64(t):
    return t.double().cpu().numpy()


def make(rows, cols, kind, seed=0, pitch=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def draw(std, dtype=torch.bfloat16):
        return (torch.randn((rows, cols + pitch), generator=g, device="cuda") * std).to(dtype)[:, :cols]

    x = draw(0.7)
    res = None if kind is None else draw(3.0, kind)
    w = (1 + 0.2 * torch.randn((cols,), generator=g, device="cuda")).to(torch.bfloat16)
    return x, res, w


def reference(x, res, w):
    r = f64(x)
    if res is not None:  # the stream's own rounding is part of the definition
        r = (x.double() + res.double()).to(res.dtype)
        r = f64(r)
    rstd = 1 / np.sqrt((r * r).mean(1) + EPS)
    return r, rstd, r * rstd[:, None] * f64(w)


@pytest.mark.parametrize("kind", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(pmn, rows, cols, kind):
    x, res, w = make(rows, cols, kind, rows + cols)
    if rows > 2:
        x[1] = 0
        if res is not None:
            res[1] = 0
        x[2] *= 1e-4
    out, r, y, rstd = pmn.add_rmsnorm_mxfp8(x, res, w, EPS, want_y=True, want_rstd=True)
    r64, rstd64, y64 = reference(x, res, w)
    assert (r is None) == (res is None)
    if r is not None:
        # float32 addition, then (bf16) a second rounding: differs from the definition's single rounding of the
        # exact sum only where the float32 sum falls on a bf16 tie
        same = f64(r) == r64
        assert same.all() if kind == torch.float32 else same.mean() > 0.999
        r64 = f64(r)
        rstd64 = 1 / np.sqrt((r64 * r64).mean(1) + EPS)
        y64 = r64 * rstd64[:, None] * f64(w)
    assert np.abs(f64(rstd) / rstd64 - 1).max() <= REL
    mx64.check_rn(out[0].cpu().numpy(), out[1].cpu().numpy(), y64, REL)
    assert (np.abs(f64(y) - y64) <= np.abs(y64) * (2.0 ** -8)).all()  # bf16: half a place of 2^-8 relative, doubled
    if rows > 2:
        assert (out[0][1].cpu().numpy() & 0x7F == 0).all() and (out[1][1] == 0).all()
    # without the optional outputs: the same bytes
    out2, r2, y2, rstd2 = pmn.add_rmsnorm_mxfp8(x, res, w, EPS)
    assert y2 is None and rstd2 is None and torch.equal(out[0], out2[0]) and torch.equal(out[1], out2[1])


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_strided_rows_and_in_place_residual(pmn, kind):
    x, res, w = make(37, 1056, kind, 5, pitch=24)
    assert not x.is_contiguous()
    got = pmn.add_rmsnorm_mxfp8(x, res, w, EPS)
    want = pmn.add_rmsnorm_mxfp8(x.contiguous(), res.contiguous(), w, EPS)
    dense = res.contiguous()
    place = pmn.add_rmsnorm_mxfp8(x, dense, w, EPS, res_out=dense)
    for o in (want, place):
        assert torch.equal(got[0][0], o[0][0]) and torch.equal(got[0][1], o[0][1]) and torch.equal(got[1], o[1])


def test_rows_that_are_not_finite(pmn):
    x, _, w = make(4, 128, None, 9)
    x[1, 5], x[2, 7], x[3, 9] = float("nan"), float("inf"), -float("inf")
    out, _, _, rstd = pmn.add_rmsnorm_mxfp8(x, None, w, EPS, want_rstd=True)
    q = out[0].cpu().numpy() & 0x7F
    assert (q[0] != 0x7F).all() and (q[1] == 0x7F).all()
    for row, col in ((2, 7), (3, 9)):
        assert q[row, col] == 0x7F and (np.delete(q[row], col) == 0).all() and rstd[row] == 0


def backward64(dy, r, rstd, w, dres):
    xh, g = r * rstd[:, None], dy * w
    c = (g * xh).mean(1, keepdims=True)
    return rstd[:, None] * (g - xh * c) + dres, (dy * xh).sum(0)


def test_the_formula_against_differences():
    """the 64-bit formula that the kernel is checked with, against central differences of the norm"""
    rng = np.random.default_rng(0)
    r, w, dy = rng.standard_normal((3, 32)), rng.standard_normal(32), rng.standard_normal((3, 32))

    def loss(r, w):
        return (dy * r / np.sqrt((r * r).mean(1, keepdims=True) + EPS) * w).sum()

    dr, dw = backward64(dy, r, 1 / np.sqrt((r * r).mean(1) + EPS), w, 0.0)
    h = 1e-5
    for i, j in [(0, 0), (1, 7), (2, 31)]:
        d = np.zeros_like(r)
        d[i, j] = h
        assert abs((loss(r + d, w) - loss(r - d, w)) / (2 * h) - dr[i, j]) < 1e-8
        assert abs((loss(r, w + d[i]) - loss(r, w - d[i])) / (2 * h) - dw[j]) < 1e-8


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES + [(2500, 96), (1000, 2048)])
def test_backward(pmn, rows, cols, kind):
    dy, r, w = make(rows, cols, kind, 3 * rows + cols)
    dres = make(rows, cols, kind, 7)[1]
    rstd = torch.from_numpy(1 / np.sqrt((f64(r) ** 2).mean(1) + EPS)).float().cuda()
    for extra in (dres, None):
        want_dx = kind == torch.float32
        dr, dx, dw = pmn.add_rmsnorm_backward(dy, r, rstd, w, dres=extra, want_dx=want_dx)
        e64 = 0.0 if extra is None else f64(extra)
        R, DY, RS, W = f64(r), f64(dy), f64(rstd), f64(w)
        dr64, dw64 = backward64(DY, R, RS, W, e64)
        xh, g = R * RS[:, None], DY * W
        mass = RS[:, None] * (np.abs(g) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True)) + np.abs(e64)
        tol = 110 * U * mass
        if kind == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(dr64)
        assert (np.abs(f64(dr) - dr64) <= tol).all()
        if want_dx:
            assert torch.equal(dx, dr.to(torch.bfloat16))
        terms = np.abs(DY * xh).sum(0)
        assert (np.abs(f64(dw) - dw64) <= (rows / 304 + 320) * U * terms).all()
        again = pmn.add_rmsnorm_backward(dy, r, rstd, w, dres=extra, want_dx=want_dx)
        assert torch.equal(dr, again[0]) and torch.equal(dw, again[2])


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(4096, 544), (5003, 1024), (4099, 1056), (4200, 2048)])
def test_backward_of_many_rows(pmn, rows, cols, kind):
    """three or six CTAs per SM: the sums' chains are shorter than the tolerance of dw allows for"""
    test_backward(pmn, rows, cols, kind)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(3, 64), (5003, 512), (4099, 1056), (700, 4096), (900, 8192), (400, 16384)])
def test_backward_in_place(pmn, rows, cols, kind):
    """dr written over dres: rows ahead are read before theirs are written"""
    dy, r, w = make(rows, cols, kind, 31)
    dres = make(rows, cols, kind, 32)[1]
    rstd = torch.rand((rows,), device="cuda") + 0.5
    want = pmn.add_rmsnorm_backward(dy, r, rstd, w, dres=dres)
    got = pmn.add_rmsnorm_backward(dy, r, rstd, w, dres=dres, dr=dres)
    assert got[0] is dres and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_no_rows(pmn):
    x, _, w = make(0, 64, None)
    out, _, _, _ = pmn.add_rmsnorm_mxfp8(x, None, w)
    assert out[0].shape == (0, 64)
    dw = torch.full((64,), 7.0, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    pmn.add_rmsnorm_backward(e, e, torch.empty((0,), device="cuda"), w, dw=dw)
    assert (dw == 0).all()


def test_nothing_is_written_outside(pmn):
    rows, cols, guard = 13, 2080, 64
    x, res, w = make(rows, cols, torch.float32, 11)

    def buf(n, dtype):
        whole = torch.zeros((n + 2 * guard,), dtype=dtype, device="cuda")
        whole.view(torch.uint8).fill_(0xA5)
        return whole, whole[guard:guard + n]

    wholes = [buf(rows * cols, torch.uint8), buf(rows * cols // 32, torch.uint8), buf(rows * cols, torch.float32),
              buf(rows * cols, torch.bfloat16), buf(rows, torch.float32)]
    q, sc, r, y, rs = [b for _, b in wholes]
    pmn.add_rmsnorm_mxfp8(x, res, w, out=(q.view(rows, cols), sc.view(rows, cols // 32)), res_out=r.view(rows, cols),
                          y=y.view(rows, cols), rstd=rs)
    for whole, _ in wholes:
        b = whole.view(torch.uint8)
        k = guard * whole.element_size()
        assert (b[:k] == 0xA5).all() and (b[-k:] == 0xA5).all()


def test_refusals(pmn):
    x, res, w = make(4, 64, torch.bfloat16)
    with pytest.raises(pmn.PmnError):
        pmn.add_rmsnorm_mxfp8(x[:, :48], None, w[:48])            # cols % 32
    with pytest.raises(pmn.PmnError):
        pmn.add_rmsnorm_mxfp8(x, res, w, eps=0.0)
    with pytest.raises(pmn.PmnError):
        pmn.add_rmsnorm_mxfp8(x, res, w, eps=float("nan"))
    with pytest.raises(pmn.PmnError):
        pmn.add_rmsnorm_mxfp8(x, res.half(), w)                   # residual's type
    with pytest.raises(pmn.PmnError):
        pmn.add_rmsnorm_mxfp8(x, res[:2], w)                      # residual's shape
    with pytest.raises(pmn.PmnError):
        pmn.add_rmsnorm_mxfp8(x, None, w, res_out=res)            # res_out without a residual
    with pytest.raises(pmn.PmnError):
        pmn.add_rmsnorm_mxfp8(x, res, w, res_out=res.float())     # res_out's type
    with pytest.raises(pmn.PmnError):
        pmn.add_rmsnorm_mxfp8(x.t(), None, w)                     # rows that are not contiguous
    odd = torch.zeros((4 * 64 + 1,), dtype=torch.bfloat16, device="cuda")[1:].view(4, 64)
    with pytest.raises(pmn.PmnError):
        pmn.add_rmsnorm_mxfp8(odd, None, w)                       # not 16-byte aligned
    rstd = torch.ones((4,), device="cuda")
    with pytest.raises(pmn.PmnError):
        pmn.add_rmsnorm_backward(x, res, rstd, w, want_dx=True)   # dx beside a bf16 dr
    with pytest.raises(pmn.PmnError):
        pmn.add_rmsnorm_backward(x, res, rstd, w, workspace=torch.empty((8,), dtype=torch.uint8, device="cuda"))
    with pytest.raises(pmn.PmnError):
        pmn.add_rmsnorm_backward(x, res, rstd[:3], w)
    assert pmn.get_device_error() == 0


def test_side_stream(pmn):
    x, res, w = make(64, 4096, torch.bfloat16, 21)
    want = pmn.add_rmsnorm_mxfp8(x, res, w, want_rstd=True)
    bwd = pmn.add_rmsnorm_backward(x, want[1], want[3], w)
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)  # the input appears on the side stream only
        got = pmn.add_rmsnorm_mxfp8(late, res, w, want_rstd=True)
        gb = pmn.add_rmsnorm_backward(late, got[1], got[3], w)
    side.synchronize()
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(gb[0], bwd[0]) and torch.equal(gb[2], bwd[2])
    assert ctypes.sizeof(pmn.AdamWTensor) == 64
