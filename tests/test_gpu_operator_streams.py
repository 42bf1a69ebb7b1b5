"""The calls around the gated block on a stream that is not the current one: what they allocate is that stream's own
(a block that the current stream's pool would hand out may still be in use there), and the results are the same."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROWS, COLS, F, EXPERTS = 256, 512, 256, 2


@pytest.fixture(scope="module")
def pmn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


def flat(x):
    return [x] if torch.is_tensor(x) else [] if x is None else [t for y in x for t in flat(y)]


def calls(pmn):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def bf16(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def mx(*shape):
        q = [pmn.mxfp8_quantize(m) for m in bf16(*shape).reshape(-1, *shape[-2:])]
        return (torch.stack([a for a, _ in q]).reshape(shape), torch.stack([b for _, b in q]).reshape(*shape[:-1], -1))

    x, r, w = bf16(ROWS, COLS), bf16(ROWS, COLS).float(), bf16(COLS)
    off = torch.tensor([0, 96, ROWS], dtype=torch.int32, device="cuda")
    a, b, c = mx(ROWS, COLS), mx(EXPERTS, 2 * F, COLS), mx(EXPERTS, F, COLS)
    y, dy, rstd = bf16(ROWS, 2 * F), bf16(ROWS, COLS), torch.rand(ROWS, generator=g, device="cuda") + 0.5
    return {
        "norm": lambda **k: pmn.add_rmsnorm_mxfp8(x, r, w, want_y=True, want_rstd=True, **k),
        "norm_backward": lambda **k: pmn.add_rmsnorm_backward(dy, r, rstd, w, want_dx=True, **k),
        "gated": lambda **k: pmn.w1_gemm_swiglu_mxfp8(a, b, off, want_t=True, want_y=True, **k),
        "gated_backward": lambda **k: pmn.dh_gemm_swiglu_backward_mxfp8(a, c, y, off, **k),
    }


@pytest.mark.parametrize("name", ["norm", "norm_backward", "gated", "gated_backward"])
def test_memory_belongs_to_the_calls_stream(pmn, name):
    call = calls(pmn)[name]
    want = flat(call())
    torch.cuda.synchronize()
    # blocks of the outputs' sizes, free in the current stream's pool
    free = [torch.empty_like(t) for t in want for _ in range(3)]
    held = {t.data_ptr() for t in free}
    del free
    side = torch.cuda.Stream()
    got = flat(call(stream=side))
    side.synchronize()
    assert len(got) == len(want)
    for g, w in zip(got, want):
        assert g.data_ptr() not in held
        assert g.dtype == w.dtype and np.array_equal(g.view(torch.uint8).cpu().numpy(), w.view(torch.uint8).cpu().numpy())
    assert pmn.get_device_error() == 0
