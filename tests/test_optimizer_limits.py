"""adamw_step's limits are checked before anything is launched, so a refused call has updated nothing.  No GPU needed:
the pointers are never used."""
import os
import shutil

import pytest


@pytest.fixture(scope="module")
def pmn():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


def step(pmn, lengths):
    table = (pmn.AdamWTensor * len(lengths))()
    for t, n in zip(table, lengths):
        t.param = t.grad = t.m = t.v = 1 << 20
        t.n = n
    return pmn.lib().pmn_adamw_step(table, len(lengths), pmn.OUT_F32, pmn.OUT_F32, pmn.STATE_F32, 1e-3, 0.9, 0.999, 1e-8,
                                    0.0, 1, None, 0, None)


@pytest.mark.parametrize("lengths", [
    [1 << 43],                                   # 2^31 blocks of 4096 elements in one launch
    [(1 << 63) - 1], [(1 << 63) - 4096],         # where the count of blocks would pass 64 bits
    [1 << 42, 1 << 42],                          # together
    [0] * 440 + [1 << 43],                       # in the second launch of a step
    [0] * 880 + [1 << 42, (1 << 62)],
])
def test_too_many_elements(pmn, lengths):
    assert step(pmn, lengths) == pmn.ERR_UNSUPPORTED


def test_a_negative_length(pmn):
    assert step(pmn, [0] * 500 + [-1]) == pmn.ERR_INVALID_ARG


def test_a_refusal_comes_before_the_first_launch(pmn):
    """the first 440 tensors are small, and would be updated by a launch of their own"""
    assert step(pmn, [4096] * 440 + [1 << 43]) == pmn.ERR_UNSUPPORTED
