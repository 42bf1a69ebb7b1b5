"""The calls from logits to expert products and back refuse an output, or a workspace, at the address of an input or of
another output.  No GPU needed: a call that is not refused could launch nothing here (and is not made where it could)."""
import os
import shutil

import pytest
import torch

from precision_moe_numerics_gb300 import pmn

# operands in the order of the C entry points: a name for an address, "out:" before those that are written, else a number
CALLS = {
    "pmn_route_topk": ["logits", 8, 1, "bias", 257, 8, 2, 0, 1, 1.0, 1, 514, "out:chosen", "out:gates", "out:row_index",
                       "out:row_choice", "out:offsets", "out:workspace", 1 << 20, None],
    "pmn_route_topk_backward": ["logits", 8, 1, "chosen", "dgates", 65, 8, 2, 0, 1, 1.0, "out:dlogits", None],
    "pmn_dispatch_rows": ["x", 64, 0, 4, 64, "row_index", 2, "row_choice", 8, "out:out", None],
    "pmn_combine_rows": ["z", 0, 8, 64, "row_index", "gates", 4, 2, 0, "out:out", None],
    "pmn_combine_rows_backward": ["dout", "z", 0, 8, 64, "row_index", "row_choice", "gates", 4, 2, "out:dz", "out:dgates", None],
    "pmn_grouped_gemm_bf16": ["a", 64, "b", 0, "offsets", 2, 0, 0, 8, 32, 64, 0, "out:out", None],
    "sums": ["a", 64, "b", 32, "offsets", 2, 1, 0, 64, 32, 8, 0, "out:out", None],
    "pmn_w1_gemm_swiglu_bf16": ["a", 64, "b", "offsets", 2, 8, 32, 64, "out:out", "out:y", None],
    "pmn_dh_gemm_swiglu_backward_bf16": ["a", 64, "b", "y", "offsets", 2, 8, 32, 64, "out:out", None],
    "pmn_matvec_nvfp4": ["x", 256, 2, "codes", "scales", "outer", "offsets", 2, 4, 32, 256, "row_choice", 2, 0, 0, "out:out",
                         "out:workspace", 1 << 30, None],
}
PAIRS = [(call, o, n) for call, args in CALLS.items() for o in args if str(o).startswith("out:")
         for n in args if isinstance(n, str) and n != o]


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("addresses that nothing may read")
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from precision_moe_numerics_gb300 import build
    build.build()
    return pmn.lib()


def made(call, same=()):
    at = {n: (i + 1) << 20 for i, n in enumerate(a for a in CALLS[call] if isinstance(a, str))}
    for n in same:
        at[n] = 1 << 30
    return [at.get(a, a) if isinstance(a, str) else a for a in CALLS[call]]


def entry(lib, call, same=()):
    return getattr(lib, "pmn_grouped_gemm_bf16" if call == "sums" else call)(*made(call, same))


@pytest.mark.parametrize("call", CALLS)
def test_addresses_of_their_own_are_not_refused(lib, call):
    assert entry(lib, call) not in (pmn.ERR_INVALID_ARG, pmn.ERR_UNSUPPORTED)  # (but find no GPU)


@pytest.mark.parametrize("call,out,other", PAIRS)
def test_an_output_at_another_operands_address_is_refused(lib, call, out, other):
    assert entry(lib, call, (out, other)) == pmn.ERR_INVALID_ARG
