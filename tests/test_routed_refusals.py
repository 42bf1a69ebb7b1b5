"""The calls from logits to expert products and back refuse what their kernels cannot index, before anything is launched.
No GPU needed: stand-ins for tensors, a library that records what reaches it, and the C entry points' own checks."""
import ctypes
import os
import shutil
import types

import pytest
import torch

from precision_moe_numerics_gb300 import pmn
from test_operator_devices import OnGpu

BF16, F32, U8, I32, F16 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.float16
SIZES = {"pmn_route_rows": 300, "pmn_route_topk_workspace_bytes": 64, "pmn_matvec_nvfp4_workspace_bytes": 64}


@pytest.fixture
def reached(monkeypatch):
    calls = []
    entry = {n: (lambda *a, n=n: calls.append(n) or 0) for n in pmn.SIGNATURES}
    entry.update({n: (lambda *a, v=v: v) for n, v in SIZES.items()})
    lib = types.SimpleNamespace(**entry)
    monkeypatch.setattr(pmn, "lib", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    return calls


T, E, K, R, D, F = 64, 8, 2, 300, 512, 64
# operands as (shape, type), and the call made of them in that order
CALLS = {
    "route": ([((T, E), F32), ((E,), F32), ((T, K), I32), ((T, K), F32), ((T, K), I32), ((R,), I32), ((E + 1,), I32), ((64,), U8)],
              lambda t, **k: pmn.route_topk(t[0], K, bias=t[1], out=pmn.Routing(*t[2:7]), workspace=t[7], **k)),
    "route_backward": ([((T, E), BF16), ((T, K), I32), ((T, K), F32), ((T, E), BF16)],
                       lambda t, **k: pmn.route_topk_backward(t[0], t[1], t[2], dlogits=t[3], **k)),
    "dispatch": ([((T, D), F32), ((T, K), I32), ((R,), I32), ((R, D), F32)],
                 lambda t, **k: pmn.dispatch_rows(t[0], t[1], t[2], out=t[3], **k)),
    "combine": ([((R, D), BF16), ((T, K), I32), ((T, K), F32), ((T, D), F32)],
                lambda t, **k: pmn.combine_rows(t[0], t[1], t[2], out=t[3], **k)),
    "combine_backward": ([((T, D), BF16), ((R, D), BF16), ((T, K), I32), ((R,), I32), ((T, K), F32), ((R, D), BF16), ((T, K), F32)],
                         lambda t, **k: pmn.combine_rows_backward(*t[:5], dz=t[5], dgates=t[6], **k)),
    "rows": ([((R, D), BF16), ((E, F, D), BF16), ((E + 1,), I32), ((R, F), F32)],
             lambda t, **k: pmn.grouped_gemm_bf16(t[0], t[1], t[2], pmn.GROUP_M, out=t[3], **k)),
    "rows_transposed": ([((R, F), BF16), ((E, F, D), BF16), ((E + 1,), I32), ((R, D), BF16)],
                        lambda t, **k: pmn.grouped_gemm_bf16(t[0], t[1], t[2], pmn.GROUP_M, b_transposed=True, out=t[3], **k)),
    "sums": ([((R, D), BF16), ((R, F), BF16), ((E + 1,), I32), ((E, D, F), F32)],
             lambda t, **k: pmn.grouped_gemm_bf16(t[0], t[1], t[2], pmn.GROUP_K, out=t[3], **k)),
    "gated": ([((R, D), BF16), ((E, 2 * F, D), BF16), ((E + 1,), I32), ((R, F), BF16), ((R, 2 * F), BF16)],
              lambda t, **k: pmn.w1_gemm_swiglu_bf16(t[0], t[1], t[2], out=t[3], y=t[4], **k)),
    "gated_backward": ([((R, D), BF16), ((E, D, F), BF16), ((R, 2 * F), BF16), ((E + 1,), I32), ((R, 2 * F), BF16)],
                       lambda t, **k: pmn.dh_gemm_swiglu_backward_bf16(t[0], t[1], t[2], t[3], out=t[4], **k)),
    "matvec": ([((T, D), BF16), ((E, F, D // 2), U8), ((E, F, D // 16), U8), ((E,), F32), ((E + 1,), I32), ((R,), I32), ((R, F), F32),
                ((64,), U8)],
               lambda t, **k: pmn.matvec_nvfp4(t[0], t[1:4], t[4], row_choice=t[5], k=K, out=t[6], workspace=t[7], **k)),
}


def made(specs, where=lambda i: 0, shapes={}, types_={}):
    return [OnGpu(where(i), *shapes.get(i, s), dtype=types_.get(i, d)) for i, (s, d) in enumerate(specs)]


@pytest.mark.parametrize("name", CALLS)
def test_tensors_and_streams_of_another_gpu_are_refused(reached, name):
    specs, call = CALLS[name]
    call(made(specs))
    assert len(reached) == 1
    for other in range(len(specs)):
        with pytest.raises(pmn.PmnError):
            call(made(specs, lambda i: int(i == other)))
    with pytest.raises(pmn.PmnError):
        call(made(specs), stream=types.SimpleNamespace(device_index=1, cuda_stream=0))
    assert len(reached) == 1
    call(made(specs), stream=types.SimpleNamespace(device_index=0, cuda_stream=0))
    assert len(reached) == 2


@pytest.mark.parametrize("name", CALLS)
def test_other_types_and_shapes_are_refused(reached, name):
    specs, call = CALLS[name]
    for i, (shape, _) in enumerate(specs):
        if shape == (64,):  # the workspace: any type, its size is the library's to check
            continue
        with pytest.raises(pmn.PmnError):
            call(made(specs, types_={i: F16}))
        with pytest.raises((pmn.PmnError, IndexError, ValueError)):
            call(made(specs, shapes={i: shape + (1,)}))
    # one row less in each but the first, and (where nothing else tells the size) in the first
    for i, (shape, _) in enumerate(specs):
        if shape == (64,) or (name, i) in (("route", 5), ("dispatch", 2), ("matvec", 0), ("combine", 0)):
            continue  # these say themselves how many rows there are
        with pytest.raises(pmn.PmnError):
            call(made(specs, shapes={i: (shape[0] - 1,) + shape[1:]}))
    assert not reached


@pytest.fixture(scope="module")
def L():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from precision_moe_numerics_gb300 import build
    build.build()
    return pmn.lib()


P, Q, W = 1 << 20, 2 << 20, 3 << 20  # aligned addresses that nothing reads: every call below is refused


def test_route_checks_its_arguments(L):
    def rows(tokens=64, experts=8, k=2, pad=1):
        return L.pmn_route_rows(tokens, experts, k, pad)

    assert rows() == 128 and rows(pad=32) == 128 + 8 * 31 // 32 * 32 and rows(tokens=1, pad=32) == 64 and rows(tokens=0) == 0
    assert L.pmn_route_topk_workspace_bytes(256, 384, 8) == 0 and L.pmn_route_topk_workspace_bytes(257, 384, 8) > 0
    for bad in (dict(tokens=-1), dict(experts=0), dict(experts=1025), dict(k=0), dict(k=9), dict(experts=64, k=33), dict(pad=0)):
        assert rows(**bad) == -1

    def call(**k):
        a = dict(logits=P, ldl=8, kind=1, bias=P, tokens=257, experts=8, k=2, score=0, normalize=1, scale=1.0, pad=1, rows=514, chosen=P,
                 gates=P, row_index=P, row_choice=P, offsets=P, ws=P, bytes=1 << 20)
        a.update(k)
        return L.pmn_route_topk(*a.values(), None)

    for bad in (dict(ldl=7), dict(kind=2), dict(score=2), dict(normalize=2), dict(rows=513), dict(rows=1 << 31), dict(k=9), dict(pad=0),
                dict(logits=0), dict(logits=P + 2), dict(bias=P + 1), dict(chosen=0), dict(gates=0), dict(row_index=0), dict(row_choice=0),
                dict(offsets=0), dict(offsets=P + 2), dict(ws=0), dict(ws=P + 8), dict(bytes=15)):
        assert call(**bad) == pmn.ERR_INVALID_ARG, bad
    assert call(tokens=128 * 65504 + 1, rows=(1 << 31) - 1) == pmn.ERR_UNSUPPORTED

    def backward(**k):
        a = dict(logits=P, ldl=8, kind=1, chosen=P, dgates=P, tokens=65, experts=8, k=2, score=0, normalize=1, scale=1.0, dlogits=Q)
        a.update(k)
        return L.pmn_route_topk_backward(*a.values(), None)

    for bad in (dict(ldl=7), dict(kind=3), dict(score=-1), dict(normalize=-1), dict(k=9), dict(logits=0), dict(chosen=P + 1), dict(dgates=0),
                dict(dlogits=0), dict(dlogits=P)):
        assert backward(**bad) == pmn.ERR_INVALID_ARG, bad
    assert backward(tokens=0, logits=0) == pmn.OK


def test_row_calls_check_their_arguments(L):
    def dispatch(**k):
        a = dict(x=P, ldx=64, kind=0, tokens=4, cols=64, index=P, k=2, choice=P, rows=8, out=Q)
        a.update(k)
        return L.pmn_dispatch_rows(*a.values(), None)

    def combine(**k):
        a = dict(z=P, kind=0, rows=8, cols=64, index=P, gates=P, tokens=4, k=2, out_kind=0, out=Q)
        a.update(k)
        return L.pmn_combine_rows(*a.values(), None)

    def backward(**k):
        a = dict(dout=P, z=P, kind=0, rows=8, cols=64, index=P, choice=P, gates=P, tokens=4, k=2, dz=Q, dgates=Q)
        a.update(k)
        return L.pmn_combine_rows_backward(*a.values(), None)

    for call, names in ((dispatch, ("x", "index", "out")), (combine, ("z", "index", "out")), (backward, ("dout", "z", "index", "dz", "dgates"))):
        for bad in [dict(kind=2), dict(cols=60), dict(k=0), dict(k=65), dict(rows=1 << 31), dict(rows=-1), dict(tokens=-1)] + \
                [{n: 0} for n in names] + [{n: P + 2} for n in names]:
            assert call(**bad) == pmn.ERR_INVALID_ARG, (call, bad)
    assert dispatch(ldx=63) == dispatch(ldx=60) == dispatch(ldx=68) == pmn.ERR_INVALID_ARG
    assert dispatch(out=P) == combine(out=P) == backward(dz=P) == backward(dgates=P) == backward(dout=W, z=W, dz=W) == pmn.ERR_INVALID_ARG
    assert combine(out_kind=3) == combine(kind=1, cols=4, out_kind=0) == combine(gates=P + 2) == pmn.ERR_INVALID_ARG
    assert dispatch(rows=0) == combine(tokens=0) == backward(tokens=0, choice=0) == pmn.OK


def test_products_check_their_arguments(L):
    def gemm(**k):
        a = dict(a=P, lda=64, b=P, ldb=0, offsets=P, groups=2, mode=0, bt=0, m=8, n=32, k=64, kind=0, out=Q)
        a.update(k)
        return L.pmn_grouped_gemm_bf16(*a.values(), None)

    for bad in (dict(lda=56), dict(lda=68), dict(groups=0), dict(groups=1025), dict(mode=2), dict(bt=2), dict(m=-1), dict(m=1 << 31),
                dict(n=0), dict(n=36), dict(k=0), dict(k=60), dict(kind=2), dict(a=0), dict(b=0), dict(out=0), dict(offsets=0),
                dict(a=P + 8), dict(b=P + 2), dict(out=P + 4), dict(offsets=P + 2), dict(out=P), dict(a=W, out=W),
                dict(mode=1, ldb=24), dict(mode=1, ldb=36), dict(mode=1, ldb=32, m=12), dict(mode=1, ldb=32, bt=1), dict(mode=1, ldb=32, m=0),
                dict(mode=1, ldb=32, lda=0, m=8)):
        assert gemm(**bad) == pmn.ERR_INVALID_ARG, bad
    assert gemm(m=0) == pmn.OK
    assert gemm(n=(1 << 30) - 512, m=1 << 20) == pmn.ERR_UNSUPPORTED

    def gated(**k):
        a = dict(a=P, lda=64, b=P, offsets=P, experts=2, rows=8, f=32, k=64, out=Q, y=W)
        a.update(k)
        return L.pmn_w1_gemm_swiglu_bf16(*a.values(), None)

    def gated_backward(**k):
        a = dict(a=P, lda=64, b=P, y=P, offsets=P, experts=2, rows=8, f=32, k=64, out=Q)
        a.update(k)
        return L.pmn_dh_gemm_swiglu_backward_bf16(*a.values(), None)

    for call in (gated, gated_backward):
        for bad in (dict(lda=56), dict(experts=0), dict(rows=-1), dict(f=0), dict(f=20), dict(k=60), dict(k=0), dict(a=0), dict(b=P + 4),
                    dict(offsets=0), dict(out=0), dict(out=P + 8), dict(y=P + 8), dict(out=P), dict(y=Q), dict(a=W + 16, out=W + 16)):
            assert call(**bad) == pmn.ERR_INVALID_ARG, (call, bad)
        assert call(rows=0, a=0) == pmn.OK
    assert gated(f=24) == pmn.ERR_INVALID_ARG and gated_backward(y=0) == pmn.ERR_INVALID_ARG

    def matvec(**k):
        a = dict(x=P, ldx=256, tokens=2, codes=P, scales=P, outer=P, offsets=P, experts=2, rows=4, n=32, k=256, choice=P, choices=2,
                 swiglu=0, kind=0, out=Q, ws=W, bytes=1 << 30)
        a.update(k)
        return L.pmn_matvec_nvfp4(*a.values(), None)

    need = L.pmn_matvec_nvfp4_workspace_bytes(4, 256)
    assert need > 4 * 8 * 128 and L.pmn_matvec_nvfp4_workspace_bytes(0, 256) == 0 and L.pmn_matvec_nvfp4_workspace_bytes(4, 128) == -1
    for bad in (dict(ldx=248), dict(ldx=260), dict(tokens=-1), dict(experts=0), dict(experts=1025), dict(rows=-1), dict(rows=1 << 28),
                dict(n=24), dict(n=0), dict(k=128), dict(k=0), dict(choices=0), dict(swiglu=2), dict(kind=2), dict(choice=0), dict(x=0),
                dict(codes=0), dict(scales=P + 8), dict(outer=P + 2), dict(offsets=P + 1), dict(choice=P + 2), dict(out=0), dict(ws=0),
                dict(ws=P + 4), dict(bytes=need - 1), dict(n=1 << 30, experts=2), dict(out=P), dict(out=W)):
        assert matvec(**bad) == pmn.ERR_INVALID_ARG, bad
    assert matvec(rows=0) == pmn.OK
    assert matvec(rows=1 << 20, n=1 << 20, k=1 << 16, ldx=1 << 16, bytes=1 << 60) == pmn.ERR_UNSUPPORTED
