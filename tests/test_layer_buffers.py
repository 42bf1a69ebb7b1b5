"""Rows of the layer's buffers that no call writes (past the last expert's segment) are defined: two steps compare equal
whatever the memory held before.  No GPU needed: the buffers are made on the CPU and no kernel runs."""
import os
import shutil

import pytest
import torch


@pytest.fixture(scope="module")
def layer():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from precision_moe_numerics_gb300 import build, layer as m
    build.build()
    return m


def test_rows_that_no_call_writes(layer, monkeypatch):
    empty = torch.empty

    def used_memory(*shape, **kw):
        t = empty(*shape, **kw)
        t.view(torch.uint8).fill_(0xFF)  # NaN in every floating-point type
        return t

    E, D, F, T = 2, 64, 32, 512
    bf16 = torch.bfloat16
    x, dy, dy1 = torch.zeros((T, D), dtype=bf16), torch.zeros((T, D), dtype=bf16), torch.zeros((T, 2 * F), dtype=bf16)
    w1, w2 = torch.zeros((E, 2 * F, D), dtype=bf16), torch.zeros((E, D, F), dtype=bf16)
    offsets = torch.tensor([0, 128, 256], dtype=torch.int32)
    monkeypatch.setattr(torch, "empty", used_memory)
    step = layer.ExpertLayerStep(x, w1, w2, dy, dy1, offsets, 200, device="cpu")
    for t in (step.h, *step.hq):
        assert torch.equal(t, t.clone()) and not t.any()
