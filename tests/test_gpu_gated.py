"""The gated projection of an MXFP8 expert and its backward against plain 64-bit implementations.

Tolerances.  u = 2^-24.  A product of K terms accumulated in float32 is within K u S of the exact one, S the sum of
the terms' magnitudes.  The sigmoid s from the hardware's exponential has a relative error of at most
(|g| + 8) 2^-23 (the argument's rounding |g| u 1.45, two ulps of the exponential, the division's two).  The errors of
h and dY1 follow from their derivatives, plus 8 u per formed product.  Rounding to bf16: half a place, 2^-9."""
import numpy as np
import pytest
import torch

import mx64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def pmn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


def f64(t):
    return t.double().cpu().numpy()


def mx(x):
    """random-looking MXFP8 bytes of a float32 array (numpy): the values are whatever the bytes decode to"""
    b = mx64.blocks(np.asarray(x, np.float64))
    e = mx64.exponent(np.abs(b).max(-1))
    y = torch.from_numpy(b / np.ldexp(1.0, e)[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return y.reshape(x.shape).numpy(), (e + 127).astype(np.uint8)


def cuda(pair):
    return tuple(torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in pair)


def host(pair):
    return tuple(t.cpu().numpy() for t in pair)


def problem(rows, experts, f, d, offsets, bwd, seed=0, big=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, d)).astype(np.float32)
    x[rng.random(x.shape) < 0.002] *= 30
    w = rng.standard_normal((experts, f if bwd else 2 * f, d)).astype(np.float32) / np.sqrt(d)
    w[-1] *= big
    y = torch.from_numpy(rng.standard_normal((rows, 2 * f)).astype(np.float32) * 1.5 * big).to(torch.bfloat16)
    return mx(x), mx(w), y, np.asarray(offsets, np.int32)


def product(a, b, offsets):
    """(A . B_e^T by expert, the sum of the terms' magnitudes), zero outside the segments"""
    A, B = mx64.decode(*a), mx64.decode(*b)
    z, s = np.zeros((2, A.shape[0], B.shape[1]))
    for e in range(len(offsets) - 1):
        r = slice(offsets[e], offsets[e + 1])
        z[r], s[r] = A[r] @ B[e].T, np.abs(A[r]) @ np.abs(B[e]).T
    return z, s


def sigmoid(g):
    return np.exp(-np.logaddexp(0.0, -g))


def check_forward(pmn, pr, train):
    a, b, _, off = pr
    d, f = a[0].shape[1], b[0].shape[1] // 2
    h, h_t, y = pmn.w1_gemm_swiglu_mxfp8(cuda(a), cuda(b), torch.from_numpy(off).cuda(), want_t=train, want_y=train)
    assert pmn.get_device_error() == 0
    z, mass = product(a, b, off)
    err = d * U * mass
    g, u, eg, eu = z[:, :f], z[:, f:], err[:, :f], err[:, f:]
    s = sigmoid(g)
    h64 = g * s * u
    eh = np.abs(u) * 1.1 * eg + np.abs(g * s) * eu + eg * eu + np.abs(h64) * ((np.abs(g) + 8) * 2.0 ** -23 + 8 * U)
    rows = slice(off[0], off[-1])
    mx64.check_rn_abs(h[0].cpu().numpy()[rows], h[1].cpu().numpy()[rows], h64[rows], eh[rows], "h")
    if train:
        q, sc = host(h_t)
        mx64.check_rn_abs(q[:, rows], sc[:, off[0] // 32:off[-1] // 32], h64[rows].T, eh[rows].T, "h_t")
        assert (np.abs(f64(y)[rows] - z[rows]) <= 2.0 ** -8 * np.abs(z[rows]) + 2 * err[rows]).all()
    return h, h_t, y


def check_backward(pmn, pr):
    a, b, y, off = pr
    d, f = a[0].shape[1], b[0].shape[1]
    out, out_t = pmn.dh_gemm_swiglu_backward_mxfp8(cuda(a), cuda(b), y.cuda(), torch.from_numpy(off).cuda())
    assert pmn.get_device_error() == 0
    dh, mass = product(a, b, off)
    e = d * U * mass
    g, u = f64(y)[:, :f], f64(y)[:, f:]
    s = sigmoid(g)
    es = (np.abs(g) + 8) * 2.0 ** -23
    k = 1 + g * (1 - s)
    du, dg = dh * g * s, dh * u * s * k
    edu = np.abs(g * s) * e + np.abs(du) * (es + 8 * U)
    edg = np.abs(u * s * k) * e + np.abs(dh * u * s) * (np.abs(k) * (es + 8 * U) + np.abs(g) * (s * es + 4 * U))
    v, err = np.concatenate([dg, du], 1), np.concatenate([edg, edu], 1)
    rows = slice(off[0], off[-1])
    q, sc = host(out)
    mx64.check_rn_abs(q[rows], sc[rows], v[rows], err[rows], "dY1")
    q, sc = host(out_t)
    mx64.check_rn_abs(q[:, rows], sc[:, off[0] // 32:off[-1] // 32], v[rows].T, err[rows].T, "dY1^T")
    return out, out_t


SEGMENTS = [
    (1, [0, 1]), (3, [0, 3]), (8, [0, 1, 2, 2, 5, 8]), (16, [0, 16]), (17, [0, 0, 17]), (31, [0, 5, 31]), (64, [0, 20, 64]), (127, [0, 127]),
    (129, [0, 129]), (300, [0, 0, 7, 135, 300]), (513, [0, 256, 256, 513]), (257, [0, 100, 257]),
]


@pytest.mark.parametrize("f,d", [(128, 512), (384, 1024)])
@pytest.mark.parametrize("rows,offsets", SEGMENTS)
def test_forward(pmn, rows, offsets, f, d):
    check_forward(pmn, problem(rows, len(offsets) - 1, f, d, offsets, False, rows), False)


@pytest.mark.parametrize("f,d", [(128, 512), (384, 1024), (1152, 512)])
@pytest.mark.parametrize("rows,offsets", [(32, [0, 32]), (128, [0, 128]), (160, [0, 32, 32, 160]),
                                          (512, [0, 128, 384, 512]), (736, [0, 256, 736]), (1184, [0, 1184])])
def test_training_forward_and_backward(pmn, rows, offsets, f, d):
    check_forward(pmn, problem(rows, len(offsets) - 1, f, d, offsets, False, rows + 1), True)
    check_backward(pmn, problem(rows, len(offsets) - 1, f, d, offsets, True, rows + 2))


@pytest.mark.parametrize("rows,offsets", [(1, [0, 1]), (45, [0, 7, 45]), (300, [0, 0, 7, 135, 300]), (513, [0, 256, 256, 513])])
def test_y_alone_on_ragged_segments(pmn, rows, offsets):
    """y without h^T: any offsets, slices cut by a segment's end"""
    a, b, _, off = problem(rows, len(offsets) - 1, 384, 512, offsets, False, rows + 5)
    h, h_t, y = pmn.w1_gemm_swiglu_mxfp8(cuda(a), cuda(b), torch.from_numpy(off).cuda(), want_y=True)
    z, mass = product(a, b, off)
    err = 512 * U * mass
    assert h_t is None and (np.abs(f64(y) - z) <= 2.0 ** -8 * np.abs(z) + 2 * err).all()
    g, u, eg, eu = z[:, :384], z[:, 384:], err[:, :384], err[:, 384:]
    s = sigmoid(g)
    eh = np.abs(u) * 1.1 * eg + np.abs(g * s) * eu + eg * eu + np.abs(g * s * u) * ((np.abs(g) + 8) * 2.0 ** -23 + 8 * U)
    mx64.check_rn_abs(h[0].cpu().numpy(), h[1].cpu().numpy(), g * s * u, eh, "h")


def test_outputs_at_every_alignment(pmn):
    """16-byte aligned codes and byte-aligned scales: the wide stores give way to narrow ones, with the same bytes"""
    off = [0, 128, 256]
    fr, br = (problem(256, 2, 384, 512, off, bwd, 41 + bwd) for bwd in (False, True))
    a, b, o = cuda(fr[0]), cuda(fr[1]), torch.from_numpy(fr[3]).cuda()
    c, w, y = cuda(br[0]), cuda(br[1]), br[2].cuda()

    def shifted(rows, cols):
        q = torch.zeros((rows * cols + 64,), dtype=torch.uint8, device="cuda")[16:16 + rows * cols].view(rows, cols)
        sc = torch.zeros((rows * cols // 32 + 8,), dtype=torch.uint8, device="cuda")[1:1 + rows * cols // 32]
        return q, sc.view(rows, cols // 32)

    want = pmn.w1_gemm_swiglu_mxfp8(a, b, o, want_t=True)
    got = pmn.w1_gemm_swiglu_mxfp8(a, b, o, out=shifted(256, 384), out_t=shifted(384, 256))
    wb = pmn.dh_gemm_swiglu_backward_mxfp8(c, w, y, o)
    gb = pmn.dh_gemm_swiglu_backward_mxfp8(c, w, y, o, out=shifted(256, 768), out_t=shifted(768, 256))
    for x, z in zip(want[:2] + wb, got[:2] + gb):
        assert torch.equal(x[0], z[0]) and torch.equal(x[1], z[1])
    assert pmn.get_device_error() == 0


@pytest.mark.parametrize("which", ["serve", "train", "backward"])
def test_a_wait_that_runs_out_is_reported(pmn, which):
    """with no time to wait the call returns, latches the timeout at most, and the next call is right"""
    off = [0, 256, 512]
    a, b, y, o = problem(512, 2, 384, 512, off, which == "backward", 61)
    a, b, o, y = cuda(a), cuda(b), torch.from_numpy(o).cuda(), y.cuda() if which == "backward" else None

    def call():
        if which == "backward":
            return pmn.dh_gemm_swiglu_backward_mxfp8(a, b, y, o)
        r = pmn.w1_gemm_swiglu_mxfp8(a, b, o, want_t=which == "train", want_y=which == "train")
        return r[:2] if which == "train" else r[:1]

    want = call()
    assert pmn.get_device_error() == 0
    limit = pmn.set_wait_limit_ns(0)
    try:
        call()
        torch.cuda.synchronize()
        assert pmn.get_device_error() in (0, pmn.DEVERR_WAIT_TIMEOUT)
    finally:
        pmn.set_wait_limit_ns(limit)
    for x, z in zip(want, call()):
        assert torch.equal(x[0], z[0]) and torch.equal(x[1], z[1])
    assert pmn.get_device_error() == 0


@pytest.mark.parametrize("which", ["serve", "train", "backward"])
def test_a_call_that_runs_out_of_time_says_so(pmn, which):
    """with no time to wait a call either is right or latches the timeout: an incomplete result is never silent"""
    off = [0, 256, 640, 640, 1280]
    a, b, y, o = problem(1280, 4, 384, 1024, off, which == "backward", 62)
    a, b, o, y = cuda(a), cuda(b), torch.from_numpy(o).cuda(), y.cuda() if which == "backward" else None

    def call():
        if which == "backward":
            return pmn.dh_gemm_swiglu_backward_mxfp8(a, b, y, o)
        r = pmn.w1_gemm_swiglu_mxfp8(a, b, o, want_t=which == "train", want_y=which == "train")
        return r[:2] if which == "train" else r[:1]

    want = call()
    assert pmn.get_device_error() == 0
    limit = pmn.set_wait_limit_ns(0)
    try:
        for _ in range(5):
            got = call()
            error = pmn.get_device_error()
            same = all(torch.equal(x[0], z[0]) and torch.equal(x[1], z[1]) for x, z in zip(want, got))
            assert error == pmn.DEVERR_WAIT_TIMEOUT or (error == 0 and same)
    finally:
        pmn.set_wait_limit_ns(limit)
    got = call()
    assert all(torch.equal(x[0], z[0]) and torch.equal(x[1], z[1]) for x, z in zip(want, got))
    assert pmn.get_device_error() == 0


@pytest.mark.parametrize("rows", [1, 4, 48])
@pytest.mark.parametrize("up", [114, 60, -125])
def test_scales_far_apart(pmn, rows, up):
    """operands whose scales are far from 1 and whose products are not: 2^up times 2^-up"""
    a, b, _, off = problem(rows, 1, 128, 512, [0, rows], False, 71)
    a = (a[0], np.full_like(a[1], 127 + up))
    b = (b[0], np.full_like(b[1], 127 - up - 12))
    h, _, _ = pmn.w1_gemm_swiglu_mxfp8(cuda(a), cuda(b), torch.from_numpy(off).cuda())
    z, mass = product(a, b, off)
    err = 512 * U * mass
    g, u, eg, eu = z[:, :128], z[:, 128:], err[:, :128], err[:, 128:]
    s = sigmoid(g)
    eh = np.abs(u) * 1.1 * eg + np.abs(g * s) * eu + eg * eu + np.abs(g * s * u) * ((np.abs(g) + 8) * 2.0 ** -23 + 8 * U)
    mx64.check_rn_abs(h[0].cpu().numpy(), h[1].cpu().numpy(), g * s * u, eh, "h")
    assert pmn.get_device_error() == 0


def test_a_scale_that_is_no_number(pmn):
    """an E8M0 byte of 255 makes its row's results NaN, by every path, and no other row's"""
    for rows in (3, 48):
        a, b, _, off = problem(rows, 1, 128, 512, [0, rows], False, 72)
        a[1][1, 5] = 255
        h, _, _ = pmn.w1_gemm_swiglu_mxfp8(cuda(a), cuda(b), torch.from_numpy(off).cuda())
        nan = (h[0] & 127) == 127
        assert nan[1].all() and not nan[0].any() and not nan[2:].any()


@pytest.mark.parametrize("bwd", [False, True])
def test_a_shared_last_round_changes_no_bit(pmn, bwd):
    """a row's results do not depend on how many tiles the call has, whose last round may be shared among CTA pairs"""
    a, b, y, _ = problem(20480, 1, 384, 512, [0, 20480], bwd, 81)

    def call(n):
        o = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        x = cuda((a[0][:n], a[1][:n]))
        if bwd:
            return pmn.dh_gemm_swiglu_backward_mxfp8(x, cuda(b), y[:n].cuda(), o)
        return pmn.w1_gemm_swiglu_mxfp8(x, cuda(b), o, want_t=True)[:2]

    (q, sc), (qt, sct) = call(20480)
    for n in (256, 2048, 4096, 6144, 8192):
        (r, rs), (rt, rst) = call(n)
        assert torch.equal(r, q[:n]) and torch.equal(rs, sc[:n])
        assert torch.equal(rt, qt[:, :n]) and torch.equal(rst, sct[:, :n // 32])
    assert pmn.get_device_error() == 0


def test_a_few_rows_and_many_agree(pmn):
    """the kernel for a handful of rows and the tiles: their float32 sums differ, their codes by one at most"""
    a, b, _, _ = problem(8, 9, 256, 2048, [0] * 10, False, 51)
    few = np.array([0, 1, 1, 3, 3, 4, 6, 6, 8, 8], np.int32)
    h, _, _ = pmn.w1_gemm_swiglu_mxfp8(cuda(a), cuda(b), torch.from_numpy(few).cuda())
    wide = (np.concatenate([a[0], np.zeros((8, 2048), np.uint8)]), np.concatenate([a[1], np.zeros((8, 64), np.uint8)]))
    many, _, _ = pmn.w1_gemm_swiglu_mxfp8(cuda(wide), cuda(b), torch.from_numpy(few).cuda())
    same = (h[1] == many[1][:8]).cpu().numpy()
    assert same.mean() > 0.99
    d = np.abs(mx64.E4M3[h[0].cpu().numpy()] - mx64.E4M3[many[0][:8].cpu().numpy()])
    v = np.abs(mx64.E4M3[h[0].cpu().numpy()])
    assert (d <= np.maximum(v / 4, 2.0 ** -8))[np.repeat(same, 32, axis=1)].all()
    assert pmn.get_device_error() == 0


def test_long_contraction_and_many_tiles(pmn):
    """K = 4096 and more tiles than SMs, so every CTA runs several and both accumulators come round"""
    off = [0, 640, 640, 1536, 2688]
    check_forward(pmn, problem(2688, 4, 1536, 4096, off, False, 5), True)
    check_backward(pmn, problem(2688, 4, 1536, 4096, off, True, 6))


def test_large_gates(pmn):
    """|gate| far beyond the exponential's range in both signs: silu is 0 or the identity"""
    off = [0, 64, 128]
    check_forward(pmn, problem(128, 2, 128, 512, off, False, 7, big=200.0), True)
    check_backward(pmn, problem(128, 2, 128, 512, off, True, 8, big=200.0))


def test_many_experts(pmn):
    """more experts than the offsets are scanned at a time, most of them empty"""
    rng = np.random.default_rng(3)
    cut = np.sort(rng.integers(0, 4, 99)) * 32
    off = [0] + cut.tolist() + [128]
    check_forward(pmn, problem(128, 100, 128, 512, off, False, 9), True)
    check_backward(pmn, problem(128, 100, 128, 512, off, True, 10))


def test_the_most_experts(pmn):
    """1024 experts, nearly all of them without rows: the same bytes as with the others left out"""
    few = np.array([0, 32, 96, 224, 256], np.int32)
    at = [3, 31, 512, 1023]
    counts = np.zeros(1024, np.int64)
    counts[at] = np.diff(few)
    all_of_them = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    for bwd in (False, True):
        a, b, y, off = problem(256, 4, 128, 512, few, bwd, 91 + bwd)
        a, b, y, off = cuda(a), cuda(b), y.cuda(), torch.from_numpy(off).cuda()
        wide = tuple(torch.full((1024,) + t.shape[1:], 120, dtype=torch.uint8, device="cuda") for t in b)
        for w, t in zip(wide, b):
            w[at] = t
        if bwd:
            want, got = (pmn.dh_gemm_swiglu_backward_mxfp8(a, w, y, o) for w, o in ((b, off), (wide, all_of_them)))
        else:
            want, got = (pmn.w1_gemm_swiglu_mxfp8(a, w, o, want_t=True)[:2] for w, o in ((b, off), (wide, all_of_them)))
        for x, z in zip(want, got):
            assert torch.equal(x[0], z[0]) and torch.equal(x[1], z[1])
    assert pmn.get_device_error() == 0


def test_the_formula_against_differences():
    rng = np.random.default_rng(1)
    g, u, dh, h = rng.standard_normal(50) * 3, rng.standard_normal(50), rng.standard_normal(50), 1e-6
    s = sigmoid(g)

    def f(g, u):
        return g * sigmoid(g) * u
    assert np.allclose((f(g + h, u) - f(g - h, u)) / (2 * h) * dh, dh * u * s * (1 + g * (1 - s)), atol=1e-8)
    assert np.allclose((f(g, u + h) - f(g, u - h)) / (2 * h) * dh, dh * g * s, atol=1e-8)


def test_rows_outside_the_segments_and_guards(pmn):
    """rows before the first and after the last segment stay as they are, and nothing is written outside the outputs"""
    rows, f, d, off, guard = 416, 384, 512, [64, 160, 160, 320], 256
    n = off[-1]
    for bwd in (False, True):
        a, b, y, o = problem(rows, 3, f, d, off, bwd, 11)
        w = 2 * f if bwd else f
        wholes = []

        def buf(*shape, dtype=torch.uint8):
            k = int(np.prod(shape)) * dtype.itemsize
            whole = torch.full((k + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
            wholes.append(whole)
            return whole[guard:guard + k].view(dtype).view(shape)

        out, out_t = (buf(rows, w), buf(rows, w // 32)), (buf(w, rows), buf(w, rows // 32))
        oo = torch.from_numpy(o).cuda()
        if bwd:
            pmn.dh_gemm_swiglu_backward_mxfp8(cuda(a), cuda(b), y.cuda(), oo, out=out, out_t=out_t)
        else:
            yo = buf(rows, 2 * f, dtype=torch.bfloat16)
            pmn.w1_gemm_swiglu_mxfp8(cuda(a), cuda(b), oo, out=out, out_t=out_t, y=yo)
            yb = yo.view(torch.uint8)
            assert (yb[:64] == 0xA5).all() and (yb[n:] == 0xA5).all()
        torch.cuda.synchronize()
        for whole in wholes:
            assert (whole[:guard] == 0xA5).all() and (whole[-guard:] == 0xA5).all()
        assert (out[0][:64] == 0xA5).all() and (out[0][n:] == 0xA5).all()
        assert (out[1][:64] == 0xA5).all() and (out[1][n:] == 0xA5).all()
        assert (out_t[0][:, :64] == 0xA5).all() and (out_t[0][:, n:] == 0xA5).all()
        assert (out_t[1][:, :2] == 0xA5).all() and (out_t[1][:, n // 32:] == 0xA5).all()


def test_bad_offsets_run_nothing(pmn):
    a, b, y, _ = problem(128, 2, 128, 512, [0, 64, 128], False, 12)
    _, w2, _, _ = problem(128, 2, 128, 512, [0, 64, 128], True, 12)
    for off, train in (([0, 130, 128], False), ([0, 64, 129], False), ([-1, 64, 128], False), ([0, 40, 128], True)):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        h = (torch.full((128, 128), 7, dtype=torch.uint8, device="cuda"),
             torch.full((128, 4), 7, dtype=torch.uint8, device="cuda"))
        pmn.w1_gemm_swiglu_mxfp8(cuda(a), cuda(b), o, out=h, want_t=train)
        assert pmn.get_device_error() == pmn.DEVERR_BAD_OFFSETS
        assert (h[0] == 7).all() and (h[1] == 7).all()
    pmn.dh_gemm_swiglu_backward_mxfp8(cuda(a), cuda(w2), y.cuda(), torch.tensor([0, 40, 128], dtype=torch.int32, device="cuda"))
    assert pmn.get_device_error() == pmn.DEVERR_BAD_OFFSETS
    assert pmn.get_device_error() == 0


def test_refusals_and_no_rows(pmn):
    a, b, y, o = problem(64, 2, 128, 512, [0, 32, 64], False)
    _, w2, _, _ = problem(64, 2, 128, 512, [0, 32, 64], True)
    a, b, w2, y, o = cuda(a), cuda(b), cuda(w2), y.cuda(), torch.from_numpy(o).cuda()

    def cut(x, k):
        return x[0][..., :k].contiguous(), x[1][..., :k // 32].contiguous()

    with pytest.raises(pmn.PmnError):
        pmn.w1_gemm_swiglu_mxfp8(cut(a, 384), cut(b, 384), o)                          # k % 512
    with pytest.raises(pmn.PmnError):
        pmn.w1_gemm_swiglu_mxfp8(a, (b[0][:, :128].contiguous(), b[1][:, :128].contiguous()), o)  # f % 128
    with pytest.raises(pmn.PmnError):
        pmn.w1_gemm_swiglu_mxfp8(a, b, o[:2])                                          # offsets' length
    with pytest.raises(pmn.PmnError):
        pmn.w1_gemm_swiglu_mxfp8(a, b, o.long())
    with pytest.raises(pmn.PmnError):
        pmn.w1_gemm_swiglu_mxfp8((a[0][:63], a[1][:63]), b, o, want_t=True)            # rows % 32 with h_t
    with pytest.raises(pmn.PmnError):
        pmn.w1_gemm_swiglu_mxfp8(a, b, o, y=torch.empty((64, 256), device="cuda"))     # y's type
    with pytest.raises(pmn.PmnError):
        pmn.dh_gemm_swiglu_backward_mxfp8(a, w2, y[:, :128], o)
    with pytest.raises(pmn.PmnError):
        pmn.dh_gemm_swiglu_backward_mxfp8((a[0][:48], a[1][:48]), w2, y[:48], o)       # rows % 32
    L = pmn.lib()
    p = 1 << 20
    assert L.pmn_w1_gemm_swiglu_mxfp8(p, p, p, p, p, 2, 64, 128, 512, p, p, p, None, None, None) == pmn.ERR_INVALID_ARG
    assert L.pmn_w1_gemm_swiglu_mxfp8(p + 8, p, p, p, p, 2, 64, 128, 512, p, p, None, None, None, None) == pmn.ERR_INVALID_ARG
    assert L.pmn_w1_gemm_swiglu_mxfp8(p, p, p, p, p, 1025, 64, 128, 512, p, p, None, None, None, None) == pmn.ERR_INVALID_ARG
    none = (a[0][:0], a[1][:0])
    h, _, _ = pmn.w1_gemm_swiglu_mxfp8(none, b, torch.zeros((3,), dtype=torch.int32, device="cuda"))
    assert h[0].shape == (0, 128) and pmn.get_device_error() == 0


def test_reproducible_on_a_side_stream(pmn):
    pr = problem(736, 2, 384, 1024, [0, 256, 736], False, 21)
    br = problem(736, 2, 384, 1024, [0, 256, 736], True, 22)
    a, b, o = cuda(pr[0]), cuda(pr[1]), torch.from_numpy(pr[3]).cuda()
    c, w, y = cuda(br[0]), cuda(br[1]), br[2].cuda()
    want = pmn.w1_gemm_swiglu_mxfp8(a, b, o, want_t=True, want_y=True)
    wb = pmn.dh_gemm_swiglu_backward_mxfp8(c, w, y, o)
    late = torch.zeros_like(a[0])
    lc = torch.zeros_like(c[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(a[0])
        lc.copy_(c[0])
        got = pmn.w1_gemm_swiglu_mxfp8((late, a[1]), b, o, want_t=True, want_y=True)
        gb = pmn.dh_gemm_swiglu_backward_mxfp8((lc, c[1]), w, y, o)
    side.synchronize()
    for x, z in ((want, got), (wb, gb)):
        for i, j in zip(x, z):
            for s, t in zip(i, j) if isinstance(i, tuple) else ((i, j),):
                assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))
    assert pmn.get_device_error(side) == 0


def test_the_same_bits_under_load(pmn):
    """many tiles per CTA, run again and again: the epilogue's buffers are refilled while others are worked on, and a
    copy that overtakes a read shows as a run that differs"""
    off = [0, 640, 640, 1536, 2688]
    fr, br = (problem(2688, 4, 1536, 4096, off, bwd, 31 + bwd) for bwd in (False, True))
    a, b, o = cuda(fr[0]), cuda(fr[1]), torch.from_numpy(fr[3]).cuda()
    c, w, y = cuda(br[0]), cuda(br[1]), br[2].cuda()

    def run():
        h, h_t, yo = pmn.w1_gemm_swiglu_mxfp8(a, b, o, want_t=True, want_y=True)
        d, d_t = pmn.dh_gemm_swiglu_backward_mxfp8(c, w, y, o)
        return [*h, *h_t, yo.view(torch.int16), *d, *d_t]

    first = run()
    for _ in range(40):
        assert all(torch.equal(s, t) for s, t in zip(run(), first))
    assert pmn.get_device_error() == 0


def test_an_odd_number_of_weight_rows_is_refused(pmn):
    """gate and up are halves: with 2 f + 1 rows an expert's weights would be read from the wrong place"""
    a, _, _, o = problem(64, 2, 128, 512, [0, 32, 64], False)
    b = (torch.zeros((2, 257, 512), dtype=torch.uint8, device="cuda"), torch.zeros((2, 257, 16), dtype=torch.uint8, device="cuda"))
    with pytest.raises(pmn.PmnError):
        pmn.w1_gemm_swiglu_mxfp8(cuda(a), b, torch.from_numpy(o).cuda())


@pytest.mark.parametrize("rows", [1, 4, 48])
def test_zeros_under_large_scales(pmn, rows):
    """zero codes whose scales' product leaves float32's range count as 0, by the kernel for few rows and the tiles"""
    a, b, _, off = problem(rows, 1, 128, 512, [0, rows], False, 73)
    a[0][:, 64:128], a[1][:, 2:4] = 0, 230
    b[1][:, :, 2:4] = 240
    h, _, _ = pmn.w1_gemm_swiglu_mxfp8(cuda(a), cuda(b), torch.from_numpy(off).cuda())
    a[1][:, 2:4] = 0
    want, _, _ = pmn.w1_gemm_swiglu_mxfp8(cuda(a), cuda(b), torch.from_numpy(off).cuda())
    assert torch.equal(h[0], want[0]) and torch.equal(h[1], want[1])
    assert ((h[0] & 127) != 127).all() and pmn.get_device_error() == 0
