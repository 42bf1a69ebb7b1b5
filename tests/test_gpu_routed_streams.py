"""The calls from logits to expert products and back on streams that are not the current one: what they allocate is that
stream's own, and two of them at once get in each other's way nowhere."""
import pytest
import torch

from test_gpu_operator_streams import flat

pytestmark = pytest.mark.gpu
T, E, K, D, F = 200, 6, 2, 512, 256


@pytest.fixture(scope="module")
def pmn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


def calls(pmn, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def bf16(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()

    logits, x, dg = torch.randn((T, E), generator=g, device="cuda"), bf16(T, D), torch.randn((T, K), generator=g, device="cuda")
    r = pmn.route_topk(logits, K, pad=8)
    xr = torch.zeros((r.row_choice.numel(), D), device="cuda").bfloat16()
    pmn.dispatch_rows(x, r.row_index, r.row_choice, out=xr)
    w1, w2 = bf16(E, 2 * F, D, std=0.05), bf16(E, D, F, std=0.05)
    y, h = bf16(xr.shape[0], 2 * F), bf16(xr.shape[0], F)
    c, s, o = pmn.nvfp4_quantize(w1.view(-1, D), outer_mode=pmn.OUTER_PER_GROUP, rows_per_group=2 * F)
    nv = c.view(E, 2 * F, D // 2), s.view(E, 2 * F, D // 16), o
    # every row in a segment, so that whole outputs are written
    full = r.offsets.clone()
    full[-1] = xr.shape[0]
    return {
        "route": lambda **k: tuple(pmn.route_topk(logits, K, pad=8, **k)),
        "route_backward": lambda **k: pmn.route_topk_backward(logits, r.experts, dg, **k),
        "dispatch": lambda **k: pmn.dispatch_rows(x, r.row_index, r.row_choice, **k)[r.row_choice != -2],
        "combine": lambda **k: pmn.combine_rows(xr, r.row_index, r.gates, **k),
        "rows": lambda **k: pmn.grouped_gemm_bf16(xr, w1, full, pmn.GROUP_M, **k),
        "transposed": lambda **k: pmn.grouped_gemm_bf16(xr, w2, full, pmn.GROUP_M, b_transposed=True, **k),
        "sums": lambda **k: pmn.grouped_gemm_bf16(xr, h, full, pmn.GROUP_K, **k),
        "gated": lambda **k: pmn.w1_gemm_swiglu_bf16(xr, w1, full, want_y=True, **k),
        "gated_backward": lambda **k: pmn.dh_gemm_swiglu_backward_bf16(xr, w2, y, full, **k),
        "matvec": lambda **k: pmn.matvec_nvfp4(xr, nv, full, swiglu=True, **k),
    }


NAMES = ["route", "route_backward", "dispatch", "combine", "rows", "transposed", "sums", "gated", "gated_backward", "matvec"]


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream(pmn, name):
    call = calls(pmn, 1)[name]
    want = flat(call())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # the test's own indexing too
        got = flat(call(stream=side))
    side.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert pmn.get_device_error() == 0


@pytest.mark.parametrize("name", [n for n in NAMES if n != "dispatch"])
def test_memory_belongs_to_the_calls_stream(pmn, name):
    call = calls(pmn, 2)[name]
    want = flat(call())
    torch.cuda.synchronize()
    free = [torch.empty_like(t) for t in want for _ in range(3)]  # blocks of the outputs' sizes, free in the current stream's pool
    held = {t.data_ptr() for t in free}
    del free
    side = torch.cuda.Stream()
    got = flat(call(stream=side))
    side.synchronize()
    assert all(g.data_ptr() not in held and torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_two_at_once(pmn, name):
    one, two = calls(pmn, 3)[name], calls(pmn, 4)[name]
    want = flat(one()), flat(two())
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(8):
        for s, f in zip(streams, (one, two)):
            with torch.cuda.stream(s):
                got.append(flat(f()))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))
    assert pmn.get_device_error() == 0
