"""What route_topk ranks first where sums of logit and bias are not finite, against an order of two keys: a NaN before any
number, then the larger number, then the lower expert.

Tolerance of the gates: (64 + 4 max|l|) u, u = 2^-24: a quotient of exponentials of at most 32 terms, see the router's
other tests."""
import numpy as np
import pytest
import torch

import routing64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def pmn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


def ranked(c, k):
    """int [tokens, k]: the experts of the k first of c (float32 sums), -1 where only -inf is left"""
    nan = np.isnan(c)
    v = np.where(nan, 0, c).astype(np.float64)
    e = np.lexsort((-v, ~nan), axis=-1)[:, :k]
    return np.where(np.take_along_axis(v, e, 1) == -np.inf, -1, e)


def check(r, chosen, experts):
    offsets, index, choice = routing64.layout(chosen, experts, 1, r.row_choice.numel())
    for name, want in (("experts", chosen), ("offsets", offsets), ("row_index", index), ("row_choice", choice)):
        assert np.array_equal(getattr(r, name).cpu().numpy(), want), name


@pytest.mark.parametrize("tokens", [31, 256, 257, 300, 16385])
@pytest.mark.parametrize("experts", [24, 128, 200, 256, 384, 500])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_a_bias_of_infinity_or_nan(pmn, tokens, experts, kind):
    """experts that the bias forces or closes for every token.  The logits are the first rows of a larger tensor: a token
    behind the last has an address too."""
    rng = np.random.default_rng(tokens + experts)
    x = torch.from_numpy((rng.standard_normal((tokens + 64, experts)) * 2).astype(np.float32)).to(TYPES[kind]).cuda()[:tokens]
    l = x.float().cpu().numpy()
    for at in ({3: INF}, {5: NAN}, {3: INF, 5: NAN, 11: INF, 17: -INF}):
        b = rng.standard_normal(experts).astype(np.float32)
        for e, v in at.items():
            b[e] = v
        r = pmn.route_topk(x, 6, bias=torch.from_numpy(b).cuda())
        chosen = ranked((l + b).astype(np.float32), 6)
        assert all((chosen == e).any(1).all() == (v != -INF) for e, v in at.items())
        check(r, chosen, experts)
        want = routing64.gates(l.astype(np.float64), chosen, "softmax", True)
        assert (np.abs(r.gates.cpu().numpy() - want) <= (64 + 4 * np.abs(l).max()) * U * want).all()
    assert pmn.get_device_error() == 0


@pytest.mark.parametrize("tokens", [2, 64, 256, 257, 1000])
@pytest.mark.parametrize("experts,k", [(3, 2), (60, 8), (384, 8), (384, 32), (700, 32), (1024, 32)])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_nan_before_infinity_before_numbers(pmn, tokens, experts, k, many, kind):
    """NaN of either sign and both infinities in every row; many: so many equals that they cannot be packed to a lane each"""
    rng = np.random.default_rng(tokens + experts + k)
    l = (rng.standard_normal((tokens, experts)) * 2).astype(np.float32)
    share = 0.3 if many else 1.5 / experts
    for v in (NAN, -NAN, INF, -INF):
        l[rng.random(l.shape) < share] = v
    l[0, :3] = INF, NAN, 1.0
    x = torch.from_numpy(l).to(TYPES[kind]).cuda()
    r = pmn.route_topk(x, k)
    check(r, ranked(x.float().cpu().numpy(), k), experts)
    assert pmn.get_device_error() == 0


def test_a_few_rows_by_hand(pmn):
    x = torch.tensor([[INF, NAN, 1.0, -INF], [1.0, INF, 2.0, INF], [-INF, -INF, NAN, -INF], [INF, -INF, -NAN, NAN]])
    for tokens in (4, 260):
        got = pmn.route_topk(x.repeat(tokens // 4, 1).cuda(), 3).experts.cpu().numpy()
        want = np.array([[1, 0, 2], [1, 3, 2], [2, -1, -1], [2, 3, 0]])
        assert np.array_equal(ranked(x.numpy(), 3), want) and np.array_equal(got, np.tile(want, (tokens // 4, 1)))
