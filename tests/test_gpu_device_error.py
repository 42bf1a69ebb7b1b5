"""pmn_get_device_error: one read takes the bits of all the library's files, each once, in the time of a launch and a copy."""
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pmn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


def calls_with_bad_offsets(pmn):
    """one of each file whose kernels check offsets or rows on the device"""
    off = torch.tensor([0, 9], dtype=torch.int32, device="cuda")  # of 8 rows
    a, w = torch.zeros((8, 256), device="cuda").bfloat16(), torch.zeros((1, 64, 256), device="cuda").bfloat16()
    codes, scales = torch.zeros((1, 64, 128), dtype=torch.uint8, device="cuda"), torch.zeros((1, 64, 16), dtype=torch.uint8, device="cuda")
    index = torch.full((8, 1), 8, dtype=torch.int32, device="cuda")
    q, qs = torch.zeros((128, 512), dtype=torch.uint8, device="cuda"), torch.zeros((128, 16), dtype=torch.uint8, device="cuda")
    far = torch.tensor([0, 256], dtype=torch.int32, device="cuda")  # of 128 rows
    wq, wqs = torch.zeros((1, 256, 512), dtype=torch.uint8, device="cuda"), torch.zeros((1, 256, 16), dtype=torch.uint8, device="cuda")
    return {"gemm_bf16": lambda: pmn.grouped_gemm_bf16(a, w, off, pmn.GROUP_M),
            "matvec": lambda: pmn.matvec_nvfp4(a, (codes, scales, torch.ones(1, device="cuda")), off),
            "route": lambda: pmn.combine_rows(a, index),
            "gated": lambda: pmn.w1_gemm_swiglu_mxfp8((q, qs), (wq, wqs), far)}


@pytest.mark.parametrize("which", ["gemm_bf16", "matvec", "route", "gated"])
def test_each_files_bits_are_taken_once(pmn, which):
    call = calls_with_bad_offsets(pmn)[which]
    assert pmn.get_device_error() == 0
    s = torch.cuda.Stream()
    for stream in (None, s):
        call()
        torch.cuda.synchronize()
        assert pmn.get_device_error(stream) == pmn.DEVERR_BAD_OFFSETS and pmn.get_device_error(stream) == 0


def test_threads_take_a_bit_once_between_them(pmn):
    call = calls_with_bad_offsets(pmn)["route"]
    assert pmn.get_device_error() == 0
    for _ in range(10):
        call()
        torch.cuda.synchronize()
        got = [[] for _ in range(4)]
        start = threading.Barrier(4)

        def take(into):
            s = torch.cuda.Stream()
            start.wait()
            into.extend(pmn.get_device_error(s) for _ in range(20))

        threads = [threading.Thread(target=take, args=(g,)) for g in got]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        bits = sorted(sum(got, []))
        assert bits == [0] * 79 + [pmn.DEVERR_BAD_OFFSETS]


def test_a_read_costs_a_launch_and_a_copy(pmn):
    """against a copy of four bytes that the host waits for; one copy per file took more than six of them"""
    word = torch.zeros(1, dtype=torch.int32, device="cuda")

    def fastest(f):
        took = []
        for _ in range(300):
            t = time.perf_counter()
            f()
            took.append(time.perf_counter() - t)
        return min(took)

    pmn.get_device_error()
    assert fastest(pmn.get_device_error) <= 3.5 * fastest(word.cpu)
