"""Long sums of matvec_nvfp4 keep float32.

Positive terms, so that their sum is the sum of their magnitudes; activations of 1/2, 1 and 3/2, which one 4-bit digit
holds, so that all of it is in one accumulator.  u = 2^-24.  The tensor core truncates: 2 u an addition, of at least 16
terms, 256 of them in the 4096 of K that an accumulator adds up.  The accumulators' sums are added rounded, u each; the
joining of digits and of CTAs' shares and the scales are within 24 u.  (One accumulator for all of K loses about 0.36 u an
addition of 64 terms, the truncated part of a sum that grows evenly: 1500 u of the longest here, where 600 u are allowed.)"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


@pytest.fixture(scope="module")
def pmn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


@pytest.mark.parametrize("k,rows", [(2048, 3), (4352, 8), (262144, 1), (131072, 12)])
def test_long_sums_keep_float32(pmn, k, rows):
    """as many tiles of 128 weight rows as SMs: each has one tile, and all of K, to itself"""
    rng = np.random.default_rng(k + rows)
    tiles = torch.cuda.get_device_properties(0).multi_processor_count
    codes = rng.integers(1, 8, (128, k // 2), dtype=np.uint8) | (rng.integers(1, 8, (128, k // 2), dtype=np.uint8) << 4)
    scales = rng.integers(1, 0x7F, (128, k // 16), dtype=np.uint8)
    x = rng.choice([0.5, 1.0, 1.5], (rows, k))
    b = scales.astype(np.int64)
    s = np.where(b >> 3 == 0, (b & 7) * 2.0 ** -9, (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10.0))
    want = x @ (np.stack([E2M1[codes & 7], E2M1[codes >> 4]], -1).reshape(128, k) * np.repeat(s, 16, -1)).T
    c, s = (torch.from_numpy(a).cuda().repeat(tiles, 1)[None] for a in (codes, scales))
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    got = pmn.matvec_nvfp4(torch.from_numpy(x).bfloat16().cuda(), (c, s, torch.ones(1, device="cuda")), off, out_dtype=torch.float32)
    got = got.double().cpu().numpy().reshape(rows, tiles, 128)
    worst = (np.abs(got - want[:, None]) / want[:, None]).max() / U
    assert worst <= 2 * 256 + -(-k // 4096) + 24, worst
    assert pmn.get_device_error() == 0
