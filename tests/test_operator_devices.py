"""The calls around the gated block launch on the current GPU: tensors or a stream of another one are refused before
anything is launched.  No GPU needed: stand-ins for tensors on two GPUs, and a library that records what reaches it."""
import types

import pytest
import torch

from precision_moe_numerics_gb300 import pmn

BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


class OnGpu:
    """a tensor's shape and type with a GPU's number"""
    is_cuda = True

    def __init__(self, gpu, *shape, dtype):
        self.gpu, self.meta = gpu, torch.empty(shape, dtype=dtype, device="meta")

    def get_device(self):
        return self.gpu

    @property
    def device(self):
        return torch.device("cuda", self.gpu)

    def data_ptr(self):
        return 1 << 20

    def __getattr__(self, name):
        return getattr(self.meta, name)


@pytest.fixture
def reached(monkeypatch):
    calls = []
    entry = types.SimpleNamespace(**{n: (lambda *a, n=n: calls.append(n) or 0) for n in pmn.SIGNATURES})
    monkeypatch.setattr(pmn, "lib", lambda: entry)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    return calls


def mx(*shape):
    return [(shape, U8), (shape[:-1] + (shape[-1] // 32,), U8)]


T, D, F, E = 64, 512, 128, 2
# operands as (shape, type), and the call made of them in that order
CALLS = {
    "norm": ([((T, D), BF16), ((T, D), F32), ((D,), BF16), *mx(T, D), ((T, D), F32), ((T, D), BF16), ((T,), F32)],
             lambda t, **k: pmn.add_rmsnorm_mxfp8(t[0], t[1], t[2], out=t[3:5], res_out=t[5], y=t[6], rstd=t[7], **k)),
    "norm_backward": ([((T, D), BF16), ((T, D), F32), ((T,), F32), ((D,), BF16), ((T, D), F32), ((T, D), F32),
                       ((T, D), BF16), ((D,), F32), ((1 << 20,), U8)],
                      lambda t, **k: pmn.add_rmsnorm_backward(t[0], t[1], t[2], t[3], dres=t[4], dr=t[5], dx=t[6], dw=t[7],
                                                              workspace=t[8], **k)),
    "gated": ([*mx(T, D), *mx(E, 2 * F, D), ((E + 1,), I32), *mx(T, F), *mx(F, T), ((T, 2 * F), BF16)],
              lambda t, **k: pmn.w1_gemm_swiglu_mxfp8(t[:2], t[2:4], t[4], out=t[5:7], out_t=t[7:9], y=t[9], **k)),
    "gated_backward": ([*mx(T, D), *mx(E, F, D), ((T, 2 * F), BF16), ((E + 1,), I32), *mx(T, 2 * F), *mx(2 * F, T)],
                       lambda t, **k: pmn.dh_gemm_swiglu_backward_mxfp8(t[:2], t[2:4], t[4], t[5], out=t[6:8], out_t=t[8:10],
                                                                        **k)),
    "adamw": ([((40,), F32), ((9,), F32), ((40,), BF16), ((9,), BF16), ((40,), F32), ((9,), F32), ((40,), F32), ((9,), F32),
               ((40,), BF16), ((9,), BF16), ((1,), F32)],
              lambda t, **k: pmn.adamw_step(pmn.AdamWTensors(t[:2], t[2:4], t[4:6], t[6:8], copies=t[8:10]), 1e-3,
                                            grad_scale=t[10], **k)),
    "adamw_mxfp8": ([((40,), BF16), ((40,), F32), ((40,), U8), ((2,), U8), ((40,), U8), ((2,), U8)],
                    lambda t, **k: pmn.adamw_step(pmn.AdamWTensors(t[:1], t[1:2], [tuple(t[2:4])], [tuple(t[4:6])]), 1e-3, **k)),
}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_gpu_are_refused(reached, name):
    specs, call = CALLS[name]

    def made(where):
        return [OnGpu(where(i), *shape, dtype=dtype) for i, (shape, dtype) in enumerate(specs)]

    call(made(lambda i: 0))
    assert len(reached) == 1
    for other in range(len(specs)):
        with pytest.raises(pmn.PmnError):
            call(made(lambda i: int(i == other)))
    with pytest.raises(pmn.PmnError):
        call(made(lambda i: 1))  # all on one GPU, which is not the current one
    assert len(reached) == 1


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_gpu_is_refused(reached, name):
    specs, call = CALLS[name]
    t = [OnGpu(0, *shape, dtype=dtype) for shape, dtype in specs]
    with pytest.raises(pmn.PmnError):
        call(t, stream=types.SimpleNamespace(device_index=1, cuda_stream=0))
    assert not reached
    call(t, stream=types.SimpleNamespace(device_index=0, cuda_stream=0))
    assert len(reached) == 1


def test_a_step_over_no_tensors(reached):
    pmn.adamw_step(pmn.AdamWTensors([], [], [], []), 1e-3)
    assert len(reached) == 1
