"""Products over a very long K in bf16 are off by their rounding.

Positive terms, so that a sum is that of its terms' magnitudes; u = 2^-24.  The tensor core's additions of a run, one for
16 of K, truncate, 2 u each, with two more inside an addition; a run is 512 of K where the result is float32, 4096 where
it is bf16 and K is above 16384, and else all of it.  The runs' sums are added rounded, u each; the result's rounding is
2^-8 of it at most.  The weights' rows (the columns of b) are constant, of different sizes, so that the sums fall
everywhere between two bf16 values.  (In one accumulator 2^20 of one sign lose 1.4 u an addition, 5.4e-3 of the sum,
70001 of them 3.6e-4: 2^-8 and 3.2e-5 are allowed.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def pmn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


def allowed(k, run):
    return (2 * (-(-run // 16) + 2) + -(-k // run)) * U


def bf16_run(k):
    return 4096 if k > 16384 else k


@pytest.mark.parametrize("rows", [511, 1025, 16384, 16385, 70001, 1 << 20])
def test_sums_over_very_many_rows(pmn, rows):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    a = (torch.rand((rows, 72), generator=gen, device="cuda") + 0.5).bfloat16()
    b = (1 + torch.arange(136, device="cuda") / 136).bfloat16().repeat(rows, 1)
    off = torch.tensor([0, 0, rows], dtype=torch.int32, device="cuda")
    want = a.double().sum(0)[:, None] * b[0].double()
    for out, half, run in ((torch.bfloat16, 2.0 ** -8, bf16_run(rows)), (torch.float32, U, 512)):
        got = pmn.grouped_gemm_bf16(a, b, off, pmn.GROUP_K, out_dtype=out).double()
        worst = ((got[1] - want).abs() / want).max().item()
        assert worst <= allowed(rows, run) + half, (out, worst)
        assert (got[0] == 0).all()
    assert pmn.get_device_error() == 0


@pytest.mark.parametrize("k", [1000, 16384, 16392, 1 << 19])
@pytest.mark.parametrize("form", ["rows", "transposed", "gated", "gated_backward"])
def test_rows_of_a_very_long_k(pmn, k, form):
    """h = silu(gate) * up of sums so large that the sigmoid is 1; the gradients with gate and up given.  The sigmoid's
    relative error is (|g| + 8) 2^-23, formed products' 16 u."""
    gen = torch.Generator(device="cuda").manual_seed(k)
    rows, n = 40, 64
    a = (torch.rand((rows, k), generator=gen, device="cuda") + 0.5).bfloat16()
    w = (1 + torch.arange(n, device="cuda") / n).bfloat16()[:, None].repeat(1, k)[None]
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    want = a.double().sum(1)[:, None] * w[0, :, 0].double()
    half, err = 2.0 ** -8, allowed(k, bf16_run(k))

    def close(got, want, tol):
        worst = ((got.double() - want).abs() / want).max().item()
        assert worst <= tol, worst

    if form == "gated":
        h, y = pmn.w1_gemm_swiglu_bf16(a, w, off, want_y=True)
        close(y, want, err + half)
        close(h, want[:, :n // 2] * want[:, n // 2:], 2.01 * err + 16 * U + half)
    elif form == "gated_backward":
        y = torch.full((rows, 2 * n), 1.5, device="cuda").bfloat16()
        got = pmn.dh_gemm_swiglu_backward_bf16(a, w.transpose(1, 2).contiguous(), y, off)
        s = 1 / (1 + torch.exp(torch.tensor(-1.5, dtype=torch.float64, device="cuda")))
        tol = err + 9.5 * 2.0 ** -23 * 2 + 16 * U + half
        close(got[:, n:], want * 1.5 * s, tol)
        close(got[:, :n], want * 1.5 * s * (1 + 1.5 * (1 - s)), tol)
    else:
        b = w.transpose(1, 2).contiguous() if form == "transposed" else w
        close(pmn.grouped_gemm_bf16(a, b, off, pmn.GROUP_M, b_transposed=form == "transposed"), want, err + half)
    assert pmn.get_device_error() == 0


@pytest.mark.parametrize("form", ["rows", "transposed", "sums", "gated", "gated_backward"])
def test_a_long_call_that_runs_out_of_time_says_so(pmn, form):
    """with no time to wait a call either is right or latches the timeout, and the next one is right"""
    gen = torch.Generator(device="cuda").manual_seed(8)
    k, off = 16392, torch.tensor([0, 300, 300, 333, 900], dtype=torch.int32, device="cuda")
    a = torch.randn((900, k), generator=gen, device="cuda").bfloat16()
    w = torch.randn((4, 128, k), generator=gen, device="cuda").bfloat16()
    y = torch.randn((900, 256), generator=gen, device="cuda").bfloat16()
    x = torch.randn((k, 264), generator=gen, device="cuda").bfloat16()
    sums = torch.tensor([0, 9001, 9001, 9003, k], dtype=torch.int32, device="cuda")
    call = {"rows": lambda: pmn.grouped_gemm_bf16(a, w, off, pmn.GROUP_M),
            "transposed": lambda: pmn.grouped_gemm_bf16(a, w.view(4, k, 128), off, pmn.GROUP_M, b_transposed=True),
            "sums": lambda: pmn.grouped_gemm_bf16(x, x, sums, pmn.GROUP_K, out_dtype=torch.bfloat16),
            "gated": lambda: torch.cat(pmn.w1_gemm_swiglu_bf16(a, w, off, want_y=True), 1),
            "gated_backward": lambda: pmn.dh_gemm_swiglu_backward_bf16(a, w.view(4, k, 128), y, off)}[form]
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
