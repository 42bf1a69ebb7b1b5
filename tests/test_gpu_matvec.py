"""Rows times NVFP4 weights against a plain 64-bit implementation.

Tolerances.  u = 2^-24.  An activation is a sum of eight octal digits in units of 2^-22 of 2^b, b the exponent of the
largest of its 16: bf16's 8 bits are all there unless it lies below 2^-15 of 2^b, and then rounding leaves half a unit,
2^-23 of 2^b; 16 values below 2^-17 of the row's largest, 2^e, have units of 2^-39 of it and leave 2^-40.  Each digit's sum
of K terms is formed in float32 with truncation, at least 16 terms at a time: K / 16 * 2 u of its magnitude, and the
magnitudes of all digits together are at most 5 times the value's (a digit rounds a remainder r to at most 2 r; what it
leaves is at most r, and from the second on an eighth of that each), so 2 K u S holds with room, S the sum of the terms' magnitudes; the joining of
digits and shares and the expert's scale add 24 u S.  The sigmoid has a relative error of (|g| + 8) 2^-23.  Rounding to bf16:
half a step, 2^-8 of the value; to float32 2^-24."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E2M1 = np.concatenate([E2M1, -E2M1])


@pytest.fixture(scope="module")
def pmn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


def weights(rng, e, n, k, top=0x7E):
    """any codes, scales from 0 up to byte `top`, outer scales of either size"""
    codes = rng.integers(0, 256, (e, n, k // 2), dtype=np.uint8)
    scales = rng.integers(0, top + 1, (e, n, k // 16), dtype=np.uint8)
    outer = (2.0 ** rng.uniform(-20, 2, e)).astype(np.float32)
    return codes, scales, outer


def values(w):
    codes, scales, outer = w
    v = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(codes.shape[:2] + (-1,))
    b = scales.astype(np.int64)
    s = np.where(b >> 3 == 0, (b & 7) * 2.0 ** -9, (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10.0))
    return v * np.repeat(s, 16, -1) * outer.astype(np.float64)[:, None, None]


def cuda(*arrays):
    return tuple(torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays)


def f64(t):
    return t.double().cpu().numpy()


def check(pmn, x, w, offsets, out, swiglu=False, choice=None, k=1, got=None):
    """x: bf16 tensor; compares every row, and that rows outside the segments keep their 7"""
    rows, n = (x.shape[0] if choice is None else len(choice)), w[0].shape[1]
    o = torch.full((rows, n // 2 if swiglu else n), 7.0, dtype=TYPES[out], device="cuda")
    rc = None if choice is None else torch.tensor(choice, dtype=torch.int32, device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    got = f64(pmn.matvec_nvfp4(x, cuda(*w), off, row_choice=rc, k=k, swiglu=swiglu, out=o))
    X, W = f64(x), values(w)
    K = X.shape[1]
    inside = np.zeros(rows, bool)
    for e in range(len(offsets) - 1):
        r = np.arange(offsets[e], offsets[e + 1])
        inside[r] = True
        xr = X[r] if choice is None else np.where((np.array(choice)[r] >= 0)[:, None], X[np.maximum(np.array(choice)[r], 0) // k], 0)
        y, mag = xr @ W[e].T, np.abs(xr) @ np.abs(W[e].T)
        block = np.repeat(np.abs(xr).reshape(len(r), K // 16, 16).max(-1), 16, -1)
        left = np.where(np.abs(xr) < 2.0 ** -14 * block, 2.0 ** -23 * block, 0) + 2.0 ** -40 * np.abs(xr).max(1, initial=0)[:, None]
        err = (2 * K + 24) * U * mag + left @ np.abs(W[e].T)
        if swiglu:
            g, u, eg, eu = y[:, :n // 2], y[:, n // 2:], err[:, :n // 2], err[:, n // 2:]
            s = 1 / (1 + np.exp(-np.clip(g, -700, None)))
            y = g * s * u
            err = eu * np.abs(g * s) + eg * (np.abs(u) + eu) * 1.1 + np.abs(y) * ((np.abs(g) + 8) * 2 ** -23 + 16 * U)  # |silu'| < 1.1
            err += 2.0 ** -148 * (np.abs(g) + 1) * np.abs(u)  # the sigmoid below float32's normal range
        assert (np.abs(got[r] - y) <= err * 1.01 + HALF[out] * np.abs(y) + 1e-37).all(), e
    assert (got[~inside] == 7).all()
    assert pmn.get_device_error() == 0


def activations(rng, tokens, k):
    x = rng.standard_normal((tokens, k)).astype(np.float32)
    x[rng.random(x.shape) < 0.01] *= 1e4
    x *= 2.0 ** rng.integers(-30, 30, (tokens, 1))
    return torch.from_numpy(x).bfloat16().cuda()


SIZES = [(16, 256), (48, 512), (1040, 768), (272, 1024), (32, 1536), (80, 4096), (16, 4352), (48, 8192), (16, 12544)]


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("offsets", [[0, 1], [0, 0, 8, 8], [1, 4, 4, 13, 30, 50]])
def test_rows(pmn, n, k, out, offsets):
    rng = np.random.default_rng(n + k)
    rows = offsets[-1] + (2 if offsets[-1] > 8 else 0)
    w = weights(rng, len(offsets) - 1, n, k)
    check(pmn, activations(rng, rows, k), w, offsets, out)


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,offsets", [(1, [0, 1, 1, 2]), (3, [0, 5, 5, 6]), (9, [0, 17, 26, 27])])
def test_gated_rows_of_tokens(pmn, n, k, out, tokens, offsets):
    """rows that name their tokens, some of them padding"""
    rng = np.random.default_rng(n + k)
    w = weights(rng, len(offsets) - 1, n, k, top=0x40)
    choice = rng.integers(0, tokens * 3, offsets[-1])
    choice[offsets[-1] // 2] = -1
    check(pmn, activations(rng, tokens, k), w, offsets, out, swiglu=True, choice=choice.tolist(), k=3)


def test_every_row_count(pmn):
    rng = np.random.default_rng(1)
    counts = list(range(36))
    offsets = np.concatenate([[0], np.cumsum(counts)]).tolist()
    check(pmn, activations(rng, offsets[-1], 256), weights(rng, 36, 32, 256), offsets, "f32")


def test_many_experts(pmn):
    rng = np.random.default_rng(2)
    counts = np.zeros(1024, int)
    counts[[0, 31, 32, 700, 1023]] = [1, 2, 9, 1, 3]
    check(pmn, activations(rng, 16, 512), weights(rng, 1024, 64, 512), np.concatenate([[0], np.cumsum(counts)]).tolist(), "f32")


def test_the_ends_of_the_range(pmn):
    """activations near bf16's largest and smallest values, one outlier beside small ones, zeros"""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 512)).astype(np.float32)
    x[0] *= 1e37
    x[1] *= 1e-38
    x[2, 5] = 3e38
    x[3] = 0
    x[4] *= 1e-40
    w = weights(rng, 1, 32, 512)
    w = w[0], w[1], np.full(1, 2.0 ** -14, np.float32)
    check(pmn, torch.from_numpy(x).bfloat16().cuda(), w, [0, 6], "f32")


def test_nan_and_infinity_stay_in_their_rows(pmn):
    rng = np.random.default_rng(4)
    x = activations(rng, 12, 768)
    w = weights(rng, 2, 48, 768)
    off = torch.tensor([0, 9, 12], dtype=torch.int32, device="cuda")
    clean = pmn.matvec_nvfp4(x, cuda(*w), off, out_dtype=torch.float32)
    for r, v in ((1, float("nan")), (8, float("inf")), (11, float("-inf"))):
        x[r, 300] = v
    got = pmn.matvec_nvfp4(x, cuda(*w), off, out_dtype=torch.float32)
    keep = torch.ones(12, dtype=torch.bool)
    keep[[1, 8, 11]] = False
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[[8, 11]]).any()
    zero = torch.from_numpy(values(w)[0][:, 300] == 0).cuda()
    assert torch.isnan(got[8][zero]).all() and torch.isinf(got[8][~zero]).all()


def test_strided_activations(pmn):
    rng = np.random.default_rng(5)
    x = activations(rng, 5, 256)
    wide = torch.full((5, 280), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 16:272] = x
    w = cuda(*weights(rng, 1, 48, 256))
    off = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    assert torch.equal(pmn.matvec_nvfp4(wide[:, 16:272], w, off), pmn.matvec_nvfp4(x, w, off))


def test_bad_rows_and_offsets_are_reported(pmn):
    rng = np.random.default_rng(6)
    x, w = activations(rng, 3, 256), cuda(*weights(rng, 2, 32, 256))
    good = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    choice = torch.tensor([0, 5, 6, 1 << 30], dtype=torch.int32, device="cuda")
    out = pmn.matvec_nvfp4(x, w, good, row_choice=choice, k=2, out_dtype=torch.float32)
    assert pmn.get_device_error() == pmn.DEVERR_BAD_OFFSETS
    assert (out[2:] == 0).all() and (out[:2] != 0).any()
    for bad in ([0, 3, 2], [-1, 1, 2], [0, 2, 5]):
        out.fill_(7.0)
        pmn.matvec_nvfp4(x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), row_choice=choice, k=2, out=out)
        assert pmn.get_device_error() == pmn.DEVERR_BAD_OFFSETS and (out == 7).all()
    assert pmn.get_device_error() == 0


def test_no_rows(pmn):
    w = cuda(*weights(np.random.default_rng(7), 2, 32, 256))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert pmn.matvec_nvfp4(torch.empty((0, 256), device="cuda").bfloat16(), w, off).shape == (0, 32)
    out = torch.full((4, 32), 7.0, device="cuda")
    pmn.matvec_nvfp4(torch.zeros((4, 256), device="cuda").bfloat16(), w, off, out=out)
    assert (out == 7).all() and pmn.get_device_error() == 0


def test_weights_of_the_quantiser(pmn):
    """weights as nvfp4_quantize leaves them, against their product in 64 bits"""
    rng = np.random.default_rng(8)
    w = torch.from_numpy(rng.standard_normal((2 * 64, 512)).astype(np.float32)).bfloat16().cuda() * 0.02
    c, s, o = pmn.nvfp4_quantize(w, outer_mode=pmn.OUTER_PER_GROUP, rows_per_group=64)
    w = c.view(2, 64, 256).cpu().numpy(), s.view(2, 64, 32).cpu().numpy(), o.cpu().numpy()
    check(pmn, activations(rng, 20, 512), w, [0, 12, 20], "bf16")
    check(pmn, activations(rng, 20, 512), w, [0, 12, 20], "bf16", swiglu=True)


def test_captured_and_replayed(pmn):
    rng = np.random.default_rng(9)
    x, w = activations(rng, 4, 512), cuda(*weights(rng, 3, 64, 512))
    off = torch.tensor([0, 4, 8, 8], dtype=torch.int32, device="cuda")
    choice = torch.arange(8, dtype=torch.int32, device="cuda")

    def call(s=None):
        return pmn.matvec_nvfp4(x, w, off, row_choice=choice, k=2, swiglu=True, stream=s)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        captured = call()
    off.copy_(torch.tensor([0, 0, 1, 8], dtype=torch.int32))
    x.copy_(activations(rng, 4, 512))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, call())


@pytest.mark.parametrize("rows", [3, 40])
def test_a_call_that_runs_out_of_time_says_so(pmn, rows):
    """with no time to wait a call either is right or latches the timeout, and the next one is right"""
    rng = np.random.default_rng(10)
    x, w = activations(rng, rows, 1024), cuda(*weights(rng, 2, 512, 1024))
    off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
    want = pmn.matvec_nvfp4(x, w, off)
    assert pmn.get_device_error() == 0
    limit = pmn.set_wait_limit_ns(0)
    try:
        for _ in range(3):
            got = pmn.matvec_nvfp4(x, w, off)
            error = pmn.get_device_error()
            assert error == pmn.DEVERR_WAIT_TIMEOUT or (error == 0 and torch.equal(got, want))
    finally:
        pmn.set_wait_limit_ns(limit)
    assert torch.equal(pmn.matvec_nvfp4(x, w, off), want) and pmn.get_device_error() == 0


@pytest.mark.parametrize("experts,rows,n,k", [(2, 52, 4096, 3584), (1, 104, 1536, 4096), (16, 8, 1040, 3584), (2, 52, 272, 8192)])
def test_scales_of_every_step_are_its_own(pmn, experts, rows, n, k):
    """each 256 of K under a scale of its own, many calls: every sum is exact, so a scale taken from another step shows"""
    step = np.arange(k // 16) // 16
    w = (np.full((experts, n, k // 2), 0x22, dtype=np.uint8),
         np.broadcast_to(((1 + step % 14) << 3).astype(np.uint8), (experts, n, k // 16)), np.ones(experts, dtype=np.float32))
    w, x = cuda(*w), torch.ones((experts * rows, k), device="cuda").bfloat16()
    off = torch.arange(experts + 1, dtype=torch.int32, device="cuda") * rows
    want = 16 * (2.0 ** (step % 14 - 6)).sum()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(150):
        wrong += (pmn.matvec_nvfp4(x, w, off, out_dtype=torch.float32) != want).sum()
    assert wrong.item() == 0 and pmn.get_device_error() == 0


def test_the_same_bits_every_time(pmn):
    """tiles that CTAs share are joined in the order of K, whoever comes last"""
    rng = np.random.default_rng(11)
    x, w = activations(rng, 9, 4096), cuda(*weights(rng, 3, 528, 4096))
    off = torch.tensor([0, 1, 3, 9], dtype=torch.int32, device="cuda")
    want = pmn.matvec_nvfp4(x, w, off, out_dtype=torch.float32)
    for _ in range(20):
        assert torch.equal(pmn.matvec_nvfp4(x, w, off, out_dtype=torch.float32), want)
