"""Sigmoid scores far from zero: the gates and their gradient where e^-l or e^l leaves float32's range.

Tolerance: an exponential two ulps of a value that may be below the normal range, 2^-149 each, twice that with the
quotient; relative (64 + 4 |l|) u, u = 2^-24, as for other gates; all of it times the scale."""
import numpy as np
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


@pytest.mark.parametrize("tokens", [7, 300])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_gates_far_below_zero(pmn, tokens, kind):
    scale = 1e30
    x = torch.linspace(-102, -70, tokens * 8, device="cuda").view(tokens, 8).to(kind)
    r = pmn.route_topk(x, 8, score=pmn.SCORE_SIGMOID, normalize=False, scale=scale)
    d = torch.ones((tokens, 8), device="cuda")
    dl = pmn.route_topk_backward(x, r.experts, d, score=pmn.SCORE_SIGMOID, normalize=False, scale=scale).double().cpu().numpy()
    l = x.double().cpu().numpy()
    want = scale / (1 + np.exp(-l))  # its gradient too: 1 - p is 1 to 2^-100
    err = (64 + 4 * np.abs(l)) * U * want + 4 * 2.0 ** -149 * scale
    got = np.empty_like(l)
    np.put_along_axis(got, r.experts.cpu().numpy().astype(np.int64), r.gates.double().cpu().numpy(), 1)
    assert (np.abs(got - want) <= err).all()
    assert (np.abs(dl - want) <= err + (2.0 ** -8 if kind == torch.bfloat16 else U) * want).all()
    assert (got > 0).all() and pmn.get_device_error() == 0


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("tokens", [7, 300])
def test_gradients_far_above_zero(pmn, tokens, normalize):
    """there 1 - p is e^-l, and the divided gates are an eighth each to 2^-100"""
    scale = 1e30
    x = torch.linspace(70, 102, tokens * 8, device="cuda").view(tokens, 8)
    r = pmn.route_topk(x, 8, score=pmn.SCORE_SIGMOID, normalize=normalize, scale=scale)
    d = torch.arange(8, device="cuda").float().repeat(tokens, 1)
    got = pmn.route_topk_backward(x, r.experts, d, score=pmn.SCORE_SIGMOID, normalize=normalize, scale=scale).double().cpu().numpy()
    l, by = x.double().cpu().numpy(), np.zeros((tokens, 8))
    np.put_along_axis(by, r.experts.cpu().numpy().astype(np.int64), d.double().cpu().numpy(), 1)
    part = (by - 3.5) / 8 if normalize else by
    want, mag = scale * part * np.exp(-l), scale * ((by + 3.5) / 8 if normalize else by) * np.exp(-l)
    assert (np.abs(got - want) <= 2 * (64 + 4 * np.abs(l)) * U * mag + 4 * 2.0 ** -149 * scale * np.abs(part)).all()
    assert ((got != 0) == (part != 0)).all() and pmn.get_device_error() == 0
