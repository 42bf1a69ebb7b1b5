"""The bf16 products of ragged experts against plain 64-bit implementations.

Tolerances.  u = 2^-24.  The tensor core adds bf16 products in float32 and truncates: a product of K terms is within
2 K u S of the exact one, S the sum of the terms' magnitudes.  The sigmoid has a relative error of (|g| + 8) 2^-23; the
errors of h and dY1 follow from their derivatives, plus 8 u per formed product.  Rounding to bf16: half a step, 2^-8 of
the value; to float32 2^-24."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def pmn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


def f64(t):
    return t.double().cpu().numpy()


def bf16(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).bfloat16()


def gpu_offsets(o):
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def strided(t):
    """the same rows with a larger pitch, off the allocation's start"""
    wide = torch.full((t.shape[0], t.shape[1] + 24), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, 8:8 + t.shape[1]] = t
    return wide[:, 8:8 + t.shape[1]]


SEGMENTS = [  # rows, offsets
    (1, [0, 1]), (7, [0, 0, 7, 7]), (16, [0, 1, 1, 10, 13, 15]), (17, [0, 17]), (24, [0, 24]), (29, [0, 13, 29]), (31, [1, 2, 9, 9, 31]), (32, [0, 3, 21, 32]), (32, [0, 32]), (33, [0, 32, 33]), (300, [3, 3, 40, 296]), (513, [0, 513]), (777, [0, 256, 257, 770]),
    (640, [0, 31, 62, 95, 129, 130, 130, 131, 400, 640]), (1100, [5, 1029, 1100]),
]


@pytest.mark.parametrize("rows,offsets", SEGMENTS)
@pytest.mark.parametrize("n,k", [(8, 8), (256, 64), (264, 200), (1000, 72), (136, 1000)])
@pytest.mark.parametrize("out,transposed", [("bf16", False), ("f32", False), ("bf16", True), ("f32", True)])
def test_rows_times_weights(pmn, rows, offsets, n, k, out, transposed):
    gen = torch.Generator(device="cuda").manual_seed(rows + n)
    e = len(offsets) - 1
    a, w = bf16(gen, rows, k), bf16(gen, e, n, k, std=k ** -0.5)
    b = w.transpose(1, 2).contiguous() if transposed else w
    o = torch.full((rows, n), 7.0, dtype=TYPES[out], device="cuda")
    got = f64(pmn.grouped_gemm_bf16(strided(a), b, gpu_offsets(offsets), pmn.GROUP_M, b_transposed=transposed, out=o))
    A, W = f64(a), f64(w)
    inside = np.zeros(rows, bool)
    for g in range(e):
        r = slice(offsets[g], offsets[g + 1])
        want, mag = A[r] @ W[g].T, np.abs(A[r]) @ np.abs(W[g].T)
        assert (np.abs(got[r] - want) <= 2 * k * U * mag + HALF[out] * np.abs(want)).all(), g
        inside[r] = True
    assert (got[~inside] == 7).all()
    assert pmn.get_device_error() == 0


@pytest.mark.parametrize("rows,offsets", SEGMENTS)
@pytest.mark.parametrize("m,n", [(8, 8), (264, 72), (72, 520), (600, 256)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_sums_over_rows(pmn, rows, offsets, m, n, out):
    gen = torch.Generator(device="cuda").manual_seed(rows + n)
    a, b = bf16(gen, rows, m), bf16(gen, rows, n)
    got = f64(pmn.grouped_gemm_bf16(strided(a), strided(b), gpu_offsets(offsets), pmn.GROUP_K, out_dtype=TYPES[out]))
    A, B = f64(a), f64(b)
    for g in range(len(offsets) - 1):
        r = slice(offsets[g], offsets[g + 1])
        want, mag = A[r].T @ B[r], np.abs(A[r]).T @ np.abs(B[r])
        assert (np.abs(got[g] - want) <= 2 * (r.stop - r.start) * U * mag + HALF[out] * np.abs(want)).all(), g
    assert pmn.get_device_error() == 0


@pytest.mark.parametrize("form,K", [("rows", 8200), ("one", 32776), ("few", 8200), ("transposed", 4096), ("sums", 16384), ("sums", 1025), ("sums", 511)])
def test_long_sums_keep_float32(pmn, form, K):
    """Positive terms, so that S is the sum itself: the tensor core's 32 additions of a run of 512 truncate (2 u each, with
    those inside an addition 34), the runs' sums are rounded (u each)."""
    gen = torch.Generator(device="cuda").manual_seed(K)

    def positive(*shape):
        return (torch.rand(shape, generator=gen, device="cuda") + 0.5).bfloat16()

    if form == "sums":
        a, b = positive(K, 72), positive(K, 264)
        got = pmn.grouped_gemm_bf16(a, b, gpu_offsets([0, K]), pmn.GROUP_K)[0]
        want = f64(a).T @ f64(b)
    else:
        rows = {"one": 1, "few": 30}.get(form, 40)
        a, b = positive(rows, K), positive(1, 264, K)
        w = b.transpose(1, 2).contiguous() if form == "transposed" else b
        got = pmn.grouped_gemm_bf16(a, w, gpu_offsets([0, rows]), pmn.GROUP_M, b_transposed=form == "transposed", out_dtype=torch.float32)
        want = f64(a) @ f64(b)[0].T
    assert (np.abs(f64(got) - want) <= (2 * 34 + -(-K // 512)) * U * want).all()
    assert pmn.get_device_error() == 0


def test_each_row_count_of_a_tile(pmn):
    """sums over 0 .. 130 rows, one expert each, and rows of 0 .. 130: every length of a last stage and tile"""
    counts = list(range(131))
    offsets = np.concatenate([[0], np.cumsum(counts)]).tolist()
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, b = bf16(gen, offsets[-1], 72), bf16(gen, offsets[-1], 40)
    got = f64(pmn.grouped_gemm_bf16(a, b, gpu_offsets(offsets), pmn.GROUP_K))
    w = bf16(gen, 131, 40, 72)
    rows = f64(pmn.grouped_gemm_bf16(a, w, gpu_offsets(offsets), pmn.GROUP_M, out_dtype=torch.float32))
    A, B, W = f64(a), f64(b), f64(w)
    for g in counts:
        r = slice(offsets[g], offsets[g + 1])
        assert (np.abs(got[g] - A[r].T @ B[r]) <= 2 * g * U * (np.abs(A[r]).T @ np.abs(B[r]))).all(), g
        assert (np.abs(rows[r] - A[r] @ W[g].T) <= 144 * U * (np.abs(A[r]) @ np.abs(W[g].T))).all(), g


@pytest.mark.parametrize("rows,offsets", SEGMENTS)
@pytest.mark.parametrize("f,k", [(16, 8), (128, 64), (144, 200), (528, 72)])
def test_gated_projection_and_its_backward(pmn, rows, offsets, f, k):
    gen = torch.Generator(device="cuda").manual_seed(rows + f)
    e = len(offsets) - 1
    a, w = bf16(gen, rows, k), bf16(gen, e, 2 * f, k, std=2 * k ** -0.5)
    off = gpu_offsets(offsets)
    h0, y0 = torch.full((rows, f), 7.0, device="cuda").bfloat16(), torch.full((rows, 2 * f), 7.0, device="cuda").bfloat16()
    h, y = pmn.w1_gemm_swiglu_bf16(strided(a), w, off, out=h0, y=y0)
    assert torch.equal(pmn.w1_gemm_swiglu_bf16(a, w, off, out=torch.full_like(h, 7.0))[0], h)
    dz, w2 = bf16(gen, rows, k), bf16(gen, e, k, f, std=k ** -0.5)
    dy = pmn.dh_gemm_swiglu_backward_bf16(strided(dz), w2, y, off, out=torch.full_like(y, 7.0))
    A, W, Z, W2, H, Y, DY = (f64(t) for t in (a, w, dz, w2, h, y, dy))
    inside = np.zeros(rows, bool)
    for x in range(e):
        r = slice(offsets[x], offsets[x + 1])
        inside[r] = True
        z, mag = A[r] @ W[x].T, 2 * k * U * (np.abs(A[r]) @ np.abs(W[x].T))
        assert (np.abs(Y[r] - z) <= mag + HALF["bf16"] * np.abs(z)).all()
        g, u, eg, eu = z[:, :f], z[:, f:], mag[:, :f], mag[:, f:]
        s = 1 / (1 + np.exp(-g))
        want = g * s * u
        err = eu * np.abs(g * s) + eg * np.abs(u) * 1.1 + np.abs(want) * ((np.abs(g) + 8) * 2 ** -23 + 16 * U)  # |silu'| < 1.1
        assert (np.abs(H[r] - want) <= err * 1.01 + HALF["bf16"] * np.abs(want) + 1e-38).all()
        d, ed = Z[r] @ W2[x], 2 * k * U * (np.abs(Z[r]) @ np.abs(W2[x]))
        g, u = Y[r][:, :f], Y[r][:, f:]
        s = 1 / (1 + np.exp(-g))
        es = s * (np.abs(g) + 8) * 2 ** -23
        for got, val, ders in ((DY[r][:, f:], g * s, es * np.abs(g)),
                               (DY[r][:, :f], u * s * (1 + g * (1 - s)), es * np.abs(u) * (1 + 3 * np.abs(g)))):
            want = d * val
            err = ed * np.abs(val) + np.abs(d) * (ders + 16 * U * (np.abs(val) + np.abs(u * s * g)))
            assert (np.abs(got - want) <= err * 1.01 + HALF["bf16"] * np.abs(want) + 1e-38).all()
    for t in (H, Y, DY):
        assert (t[~inside] == 7).all()
    assert pmn.get_device_error() == 0


@pytest.mark.parametrize("rows", [13, 24, 50])
def test_gates_far_from_zero(pmn, rows):
    """gate, up and dH given as they are by one-hot products.  The sigmoid's 2^-148 below the normal range reaches h times
    gate and up, which may be large; a product of two that is itself subnormal adds 2^-149 times the third."""
    f, k = 16, 8
    g = torch.linspace(-103, 103, rows).bfloat16()
    x = torch.zeros((rows, k))
    x[:, 0], x[:, 1] = g.float(), torch.tensor([3e30, -1.5, 2e20, 1e-3, 0.0]).repeat(rows)[:rows]
    w = torch.zeros((1, 2 * f, k))
    w[0, :f, 0], w[0, f:, 1] = 1.0, 1.0
    x, w, off = x.bfloat16().cuda(), w.bfloat16().cuda(), gpu_offsets([0, rows])
    h, y = pmn.w1_gemm_swiglu_bf16(x, w, off, want_y=True)
    assert torch.equal(y[:, :f], x[:, :1].expand(-1, f)) and torch.equal(y[:, f:], x[:, 1:2].expand(-1, f))
    X = f64(x)
    G, V = X[:, :1], X[:, 1:2]
    s = 1 / (1 + np.exp(-G))
    tiny, rel = 2.0 ** -148, (np.abs(G) + 8) * 2 ** -23 + 16 * U + HALF["bf16"]
    want = G * s * V
    assert (np.abs(f64(h) - want) <= np.abs(want) * rel + tiny * (np.abs(G) + 1) * np.abs(V) + 2.0 ** -133).all()
    d = torch.zeros((rows, k))
    d[:, 0] = torch.tensor([1e25, -2.0, 1e-2]).repeat(rows)[:rows]
    w2 = torch.zeros((1, k, f))
    w2[0, 0] = 1.0
    d, v = d.bfloat16().cuda(), y.clone()
    v[:, f:] = torch.tensor([-4.0, 1e10, 0.5, 1.0]).repeat(rows)[:rows].bfloat16().cuda()[:, None]
    got, D, V = f64(pmn.dh_gemm_swiglu_backward_bf16(d, w2.bfloat16().cuda(), v, off)), f64(d)[:, :1], f64(v)[:, f:f + 1]
    up, gate = D * G * s, D * V * s * (1 + G * (1 - s))
    mag = np.abs(D * V * s) * (1 + np.abs(G))  # 1 + g (1 - s) cancels near its zero
    assert (np.abs(got[:, f:] - up) <= np.abs(up) * rel + tiny * (np.abs(D) + 1) * (np.abs(G) + 1) + 2.0 ** -133).all()
    assert (np.abs(got[:, :f] - gate) <= np.abs(gate) * rel + mag * (np.abs(G) + 16) * 2 ** -22
            + tiny * (np.abs(D) + 1) * (np.abs(V) + 1) * (1 + np.abs(G)) + 2.0 ** -133).all()


def test_gated_gradient_against_differences(pmn):
    """dY1 against central differences of sum(dz . (h W2^T)) in 64 bits"""
    gen = torch.Generator(device="cuda").manual_seed(5)
    f, d, rows = 16, 24, 5
    y, dz, w2 = bf16(gen, rows, 2 * f), bf16(gen, rows, d), bf16(gen, 1, d, f)
    got = f64(pmn.dh_gemm_swiglu_backward_bf16(dz, w2, y, gpu_offsets([0, rows])))
    Y, Z, W = f64(y), f64(dz), f64(w2)[0]

    def loss(v):
        return (Z * ((v[:, :f] / (1 + np.exp(-v[:, :f])) * v[:, f:]) @ W.T)).sum()

    for i in range(rows):
        for j in range(2 * f):
            hi, lo = Y.copy(), Y.copy()
            hi[i, j] += 1e-5
            lo[i, j] -= 1e-5
            diff = (loss(hi) - loss(lo)) / 2e-5
            assert abs(got[i, j] - diff) <= HALF["bf16"] * abs(diff) + 1e-6


def test_nan_and_infinity_stay_with_their_rows(pmn):
    gen = torch.Generator(device="cuda").manual_seed(2)
    offsets = [0, 5, 70, 71, 141]
    a, b, w = bf16(gen, 150, 64), bf16(gen, 150, 72), bf16(gen, 4, 72, 64)
    clean_rows = pmn.grouped_gemm_bf16(a, w, gpu_offsets(offsets), pmn.GROUP_M, out=torch.zeros((150, 72), device="cuda"))
    clean_sums = pmn.grouped_gemm_bf16(a, b, gpu_offsets(offsets), pmn.GROUP_K)
    for r, v in ((5, float("nan")), (69, float("inf")), (141, float("nan")), (149, float("-inf"))):
        a[r], b[r] = v, v
    rows = pmn.grouped_gemm_bf16(a, w, gpu_offsets(offsets), pmn.GROUP_M, out=torch.zeros((150, 72), device="cuda"))
    sums = pmn.grouped_gemm_bf16(a, b, gpu_offsets(offsets), pmn.GROUP_K)
    keep = torch.ones(150, dtype=torch.bool)
    keep[[5, 69]] = False
    assert torch.equal(rows[keep], clean_rows[keep]) and not torch.isfinite(rows[[5, 69]]).any()
    assert torch.equal(sums[[0, 2, 3]], clean_sums[[0, 2, 3]]) and torch.isnan(sums[1]).all()


@pytest.mark.parametrize("offsets", [[0, 5, 4, 8], [0, 3, 6, 9], [-1, 2, 4, 8]])
def test_bad_offsets_run_nothing_and_are_reported(pmn, offsets):
    gen = torch.Generator(device="cuda").manual_seed(2)
    a, b, w = bf16(gen, 8, 64), bf16(gen, 8, 72), bf16(gen, 3, 72, 64)
    out, sums = torch.full((8, 72), 7.0, device="cuda"), torch.full((3, 64, 72), 7.0, device="cuda")
    pmn.grouped_gemm_bf16(a, w, gpu_offsets(offsets), pmn.GROUP_M, out=out)
    assert pmn.get_device_error() == pmn.DEVERR_BAD_OFFSETS and (out == 7).all()
    pmn.grouped_gemm_bf16(a, b, gpu_offsets(offsets), pmn.GROUP_K, out=sums)
    assert pmn.get_device_error() == pmn.DEVERR_BAD_OFFSETS and (sums == 7).all() and pmn.get_device_error() == 0


def test_no_rows(pmn):
    off = gpu_offsets([0, 0, 0])
    a, w = torch.empty((0, 64), device="cuda").bfloat16(), torch.zeros((2, 32, 64), device="cuda").bfloat16()
    assert pmn.grouped_gemm_bf16(a, w, off, pmn.GROUP_M).shape == (0, 32)
    assert pmn.w1_gemm_swiglu_bf16(a, w, off)[0].shape == (0, 16)
    out = torch.full((2, 64, 64), 7.0, device="cuda")
    assert (pmn.grouped_gemm_bf16(a, a, off, pmn.GROUP_K, out=out) == 0).all()


def test_many_experts_and_wide_rows(pmn):
    """1024 experts, a few with rows; more tiles than CTA pairs; sums of long segments"""
    gen = torch.Generator(device="cuda").manual_seed(9)
    counts = [0] * 1024
    for e, c in ((0, 1), (17, 300), (512, 2), (1023, 700)):
        counts[e] = c
    offsets = np.concatenate([[0], np.cumsum(counts)]).tolist()
    a, w = bf16(gen, 1003, 128), bf16(gen, 1024, 264, 128)
    got = f64(pmn.grouped_gemm_bf16(a, w, gpu_offsets(offsets), pmn.GROUP_M, out_dtype=torch.float32))
    for e in (0, 17, 512, 1023):
        r = slice(offsets[e], offsets[e + 1])
        A, W = f64(a[r]), f64(w[e])
        assert (np.abs(got[r] - A @ W.T) <= 256 * U * (np.abs(A) @ np.abs(W.T))).all()
    a, b = bf16(gen, 4100, 1032), bf16(gen, 4100, 1288)
    got = f64(pmn.grouped_gemm_bf16(a, b, gpu_offsets([0, 2, 4099]), pmn.GROUP_K))
    A, B = f64(a[2:4099]), f64(b[2:4099])
    assert (np.abs(got[1] - A.T @ B) <= 2 * 4097 * U * (np.abs(A).T @ np.abs(B))).all()


@pytest.mark.parametrize("experts,k", [(1024, 264), (257, 1032), (3, 4104)])
def test_few_rows_of_many_experts(pmn, experts, k):
    """the kernel for a few rows: experts found among many, K that ends inside a warp's share, both outputs"""
    gen = torch.Generator(device="cuda").manual_seed(experts)
    counts = [0] * experts
    for e, c in ((0, 2), (experts // 2, 9), (experts - 1, 3)):
        counts[e] = c
    offsets = np.concatenate([[0], np.cumsum(counts)]).tolist()
    a, w = bf16(gen, 14, k), bf16(gen, experts, 32, k, std=k ** -0.5)
    off = gpu_offsets(offsets)
    rows = f64(pmn.grouped_gemm_bf16(a, w, off, pmn.GROUP_M, out_dtype=torch.float32))
    h, y = pmn.w1_gemm_swiglu_bf16(a, w, off, want_y=True)
    for e in (0, experts // 2, experts - 1):
        r = slice(offsets[e], offsets[e + 1])
        A, W = f64(a[r]), f64(w[e])
        want, err = A @ W.T, 2 * k * U * (np.abs(A) @ np.abs(W.T))
        assert (np.abs(rows[r] - want) <= err).all()
        assert (np.abs(f64(y)[r] - want) <= err + HALF["bf16"] * np.abs(want)).all()
        g, u, eg, eu = want[:, :16], want[:, 16:], err[:, :16], err[:, 16:]
        s = 1 / (1 + np.exp(-g))
        tol = eu * np.abs(g * s) + eg * np.abs(u) * 1.1 + np.abs(g * s * u) * ((np.abs(g) + 8) * 2 ** -23 + 16 * U)  # |silu'| < 1.1
        assert (np.abs(f64(h)[r] - g * s * u) <= tol * 1.01 + HALF["bf16"] * np.abs(g * s * u) + 1e-38).all()
    assert pmn.get_device_error() == 0


def test_captured_and_replayed_with_other_rows(pmn):
    gen = torch.Generator(device="cuda").manual_seed(4)
    a, w, w2 = bf16(gen, 400, 64), bf16(gen, 3, 64, 64), bf16(gen, 3, 64, 32)
    off = gpu_offsets([0, 100, 250, 400])

    def chain(s=None):
        h, y = pmn.w1_gemm_swiglu_bf16(a, w, off, want_y=True, stream=s)
        z = pmn.grouped_gemm_bf16(h, w2, off, pmn.GROUP_M, stream=s)
        dy = pmn.dh_gemm_swiglu_backward_bf16(z, w2, y, off, stream=s)
        return h, y, z, dy, pmn.grouped_gemm_bf16(dy, a, off, pmn.GROUP_K, stream=s)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    chain(s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        captured = chain()
    for cut in ([0, 0, 300, 400], [0, 399, 399, 400]):
        off.copy_(gpu_offsets(cut))
        a.copy_(bf16(gen, 400, 64))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(captured, chain()):
            assert torch.equal(x, y)


@pytest.mark.parametrize("which", ["rows", "rows_f32", "transposed", "sums", "gated", "gated_backward"])
def test_a_call_that_runs_out_of_time_says_so(pmn, which):
    """with no time to wait a call either is right or latches the timeout, and the next one is right"""
    gen = torch.Generator(device="cuda").manual_seed(6)
    off = gpu_offsets([0, 300, 300, 333, 900])
    a, b, w, w2, y = bf16(gen, 900, 640), bf16(gen, 900, 256), bf16(gen, 4, 512, 640), bf16(gen, 4, 640, 256), bf16(gen, 900, 512)
    call = {"rows": lambda: pmn.grouped_gemm_bf16(a, w, off, pmn.GROUP_M),
            "rows_f32": lambda: pmn.grouped_gemm_bf16(a, w, off, pmn.GROUP_M, out_dtype=torch.float32),
            "transposed": lambda: pmn.grouped_gemm_bf16(a, w2, off, pmn.GROUP_M, b_transposed=True),
            "sums": lambda: pmn.grouped_gemm_bf16(a, b, off, pmn.GROUP_K),
            "gated": lambda: torch.cat(pmn.w1_gemm_swiglu_bf16(a, w, off, want_y=True), 1),
            "gated_backward": lambda: pmn.dh_gemm_swiglu_backward_bf16(a, w2, y, off)}[which]
    want = call()
    assert pmn.get_device_error() == 0
    limit = pmn.set_wait_limit_ns(0)
    try:
        for _ in range(3):
            got = call()
            error = pmn.get_device_error()
            assert error == pmn.DEVERR_WAIT_TIMEOUT or (error == 0 and torch.equal(got, want))
    finally:
        pmn.set_wait_limit_ns(limit)
    assert torch.equal(call(), want) and pmn.get_device_error() == 0
