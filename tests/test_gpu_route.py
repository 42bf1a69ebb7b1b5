"""Routing and the moving of rows against plain 64-bit implementations.

Tolerances.  u = 2^-24.  A gate is a quotient of exponentials: the argument's rounding gives |v| u (and the logarithm of
the sigmoid three times that), an exponential two ulps, a sum of n positive terms n u, the quotient and the scale u each:
(64 + 4 max|l|) u covers sums of up to 37 terms in order (1024 experts: 32 in a lane, 5 steps between lanes).  A gradient
is within twice that of the sum of its terms' magnitudes.  combine: k fused sums, k u of the sum of magnitudes; a dot
product of n terms n u; rounding to bf16 half a step, 2^-8 of the value, to float32 2^-24."""
import numpy as np
import pytest
import torch

import routing64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def pmn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


def host(t):
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def problem(tokens, experts, kind, seed=0, masked=False, ties=False):
    rng = np.random.default_rng(seed)
    l = (rng.standard_normal((tokens, experts)) * 2).astype(np.float32)
    if ties:
        l = np.round(l)
        l[rng.random(l.shape) < 0.3] *= -0.0
    if masked:
        l[rng.random(l.shape) < 0.5] = -np.inf
        l[::3] = -np.inf
    return torch.from_numpy(l).to(TYPES[kind]).cuda()


def score_of(pmn, score):
    return pmn.SCORE_SOFTMAX if score == "softmax" else pmn.SCORE_SIGMOID


def check_layout(r, chosen, experts, pad):
    offsets, index, choice = routing64.layout(chosen, experts, pad, r.row_choice.numel())
    for name, want in (("experts", chosen), ("offsets", offsets), ("row_index", index), ("row_choice", choice)):
        assert np.array_equal(host(getattr(r, name)), want), name


ROUTES = [  # tokens, experts, k, pad, kind
    (1, 1, 1, 1, "f32"), (1, 384, 8, 1, "f32"), (3, 2, 2, 128, "bf16"), (64, 384, 8, 1, "f32"), (65, 60, 4, 32, "bf16"),
    (129, 33, 32, 7, "f32"), (200, 100, 5, 1, "f32"), (777, 200, 6, 8, "bf16"), (300, 500, 3, 16, "f32"), (131, 1024, 32, 3, "f32"),
    (4097, 1000, 8, 128, "bf16"), (8193, 384, 8, 128, "f32"), (20011, 24, 2, 512, "f32"),
    (2, 128, 8, 1, "bf16"), (5, 700, 32, 4, "f32"), (9, 256, 8, 1, "bf16"), (17, 60, 4, 8, "f32"), (31, 384, 6, 1, "bf16"),
    (255, 1024, 32, 2, "bf16"), (256, 384, 8, 128, "f32"), (257, 384, 8, 1, "bf16"), (512, 16, 16, 1, "f32"),
    (19457, 128, 8, 1, "bf16"),
]


@pytest.mark.parametrize("tokens,experts,k,pad,kind", ROUTES)
@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_and_its_gradient(pmn, tokens, experts, k, pad, kind, score, normalize):
    bias = tokens % 2 == 0
    x = problem(tokens, experts, kind, tokens, masked=experts % 2 == 0 and tokens > 1, ties=experts == 60)
    b = torch.randn(experts, generator=torch.Generator().manual_seed(1)).cuda() if bias else None
    r = pmn.route_topk(x, k, bias=b, score=score_of(pmn, score), normalize=normalize, scale=2.5, pad=pad)
    l32 = host(x)
    chosen = routing64.choices(l32, None if b is None else host(b), k)
    check_layout(r, chosen, experts, pad)
    l = l32.astype(np.float64)
    rel = (64 + 4 * np.abs(l[np.isfinite(l)]).max(initial=0)) * U
    want = routing64.gates(l, chosen, score, normalize, 2.5)
    assert (np.abs(host(r.gates) - want) <= rel * want + 1e-37).all()
    d = np.random.default_rng(7).standard_normal((tokens, k)).astype(np.float32)
    got = host(pmn.route_topk_backward(x, r.experts, torch.from_numpy(d).cuda(), score=score_of(pmn, score),
                                       normalize=normalize, scale=2.5)).astype(np.float64)
    want, mag = routing64.gates_backward(l, chosen, d.astype(np.float64), score, normalize, 2.5)
    assert (np.abs(got - want) <= 2 * rel * mag + HALF[kind] * np.abs(want) + 1e-37).all()
    assert pmn.get_device_error() == 0


@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_route_gradient_against_differences(pmn, score, normalize):
    x = problem(6, 11, "f32", 3)
    l, d = host(x).astype(np.float64), np.random.default_rng(4).standard_normal((6, 3))
    r = pmn.route_topk(x, 3, score=score_of(pmn, score), normalize=normalize)
    chosen = host(r.experts)
    d32 = torch.from_numpy(d.astype(np.float32)).cuda()
    got = host(pmn.route_topk_backward(x, r.experts, d32, score=score_of(pmn, score), normalize=normalize))
    h = 1e-5
    for t in range(6):
        for e in range(11):
            hi, lo = l.copy(), l.copy()
            hi[t, e] += h
            lo[t, e] -= h
            diff = ((routing64.gates(hi, chosen, score, normalize) - routing64.gates(lo, chosen, score, normalize)) * d).sum() / (2 * h)
            assert abs(got[t, e] - diff) <= 1e-5  # h^2 of the third derivative, 1e-16 / h of the differences, float32


def test_route_names_the_lowest_of_equals_and_drops_what_is_masked(pmn):
    inf = float("inf")
    x = torch.tensor([[0.0, -0.0, 0.0, -0.0], [-inf, 1.0, -inf, 1.0], [-inf] * 4, [-inf, -inf, -3e38, -inf]]).cuda()
    r = pmn.route_topk(x, 3, pad=4)
    assert host(r.experts).tolist() == [[0, 1, 2], [1, 3, -1], [-1, -1, -1], [2, -1, -1]]
    g = host(r.gates)
    assert np.allclose(g, [[1 / 3] * 3, [0.5, 0.5, 0], [0, 0, 0], [1, 0, 0]], rtol=1e-6, atol=0)
    b = torch.tensor([0.0, 0.0, -inf, 1.0]).cuda()  # a bias of -inf closes an expert
    assert host(pmn.route_topk(x, 3, bias=b).experts).tolist() == [[3, 0, 1], [3, 1, -1], [-1, -1, -1], [-1, -1, -1]]


def test_route_with_nan_and_infinity(pmn):
    nan, inf = float("nan"), float("inf")
    x = torch.tensor([[0.0, nan, 2.0, nan], [inf, 0.0, 1.0, 2.0], [0.0, 1.0, 2.0, 3.0]]).cuda()
    for normalize in (True, False):
        for score in ("softmax", "sigmoid"):
            r = pmn.route_topk(x, 2, score=score_of(pmn, score), normalize=normalize)
            assert host(r.experts).tolist() == [[1, 3], [0, 3], [3, 2]]
            assert np.isnan(host(r.gates)[0]).all() and np.isfinite(host(r.gates)[2]).all()
    assert host(pmn.route_topk(x, 2, score=pmn.SCORE_SIGMOID, normalize=False).gates)[1, 0] == 1.0


def test_gates_where_every_score_underflows(pmn):
    x = torch.tensor([[-300.0, -301.0, -400.0]]).cuda()
    r = pmn.route_topk(x, 2, score=pmn.SCORE_SIGMOID)
    want = 1 / (1 + np.exp(-1.0))
    assert np.allclose(host(r.gates), [[want, 1 - want]], rtol=2000 * U, atol=0)


def test_route_of_strided_logits_into_given_tensors(pmn):
    x = problem(150, 40, "bf16", 5)
    wide = torch.full((150, 72), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:48] = x
    rows = pmn.route_rows(150, 40, 4, 32) + 100
    out = pmn.Routing(*[torch.full(s, 77, dtype=t, device="cuda") for s, t in
                        (((150, 4), torch.int32), ((150, 4), torch.float32), ((150, 4), torch.int32), ((rows,), torch.int32),
                         ((41,), torch.int32))])
    ws = torch.empty(pmn.route_topk_workspace_bytes(150, 40, 4), dtype=torch.uint8, device="cuda")
    r = pmn.route_topk(wide[:, 8:48], 4, pad=32, out=out, workspace=ws)
    check_layout(r, routing64.choices(host(x), None, 4), 40, 32)
    d = torch.ones((150, 4), device="cuda")
    assert torch.equal(pmn.route_topk_backward(wide[:, 8:48], r.experts, d), pmn.route_topk_backward(x, r.experts, d))


def test_no_tokens(pmn):
    r = pmn.route_topk(torch.empty((0, 5), device="cuda"), 2, rows=9)
    assert host(r.offsets).tolist() == [0] * 6 and host(r.row_choice).tolist() == [-2] * 9
    assert pmn.route_topk_backward(torch.empty((0, 5), device="cuda"), r.experts, r.gates).shape == (0, 5)
    out = torch.full((9, 8), 3.0, device="cuda")
    pmn.dispatch_rows(torch.empty((0, 8), device="cuda"), r.row_index, r.row_choice, out=out)
    assert (out == 3.0).all()
    assert pmn.combine_rows(out, r.row_index).shape == (0, 8)


def test_a_choice_beyond_the_experts_is_reported(pmn):
    x = problem(4, 5, "f32")
    chosen = torch.tensor([[0, 5], [1, 2], [3, -1], [1000, 4]], dtype=torch.int32, device="cuda")
    d = torch.ones((4, 2), device="cuda")
    got = pmn.route_topk_backward(x, chosen, d, score=pmn.SCORE_SIGMOID, normalize=False)
    assert pmn.get_device_error() == pmn.DEVERR_BAD_OFFSETS and pmn.get_device_error() == 0
    assert (host(got) != 0).sum(1).tolist() == [1, 2, 1, 1]


ROWS = [  # tokens, experts, k, pad, cols, kind
    (1, 1, 1, 1, 8, "bf16"), (1, 8, 8, 16, 4096, "bf16"), (5, 3, 2, 1, 4, "f32"), (64, 30, 8, 1, 4096, "bf16"),
    (65, 7, 5, 32, 1028, "f32"), (333, 24, 9, 128, 2056, "bf16"), (300, 200, 17, 8, 520, "f32"), (1021, 384, 8, 128, 1536, "f32"),
]


@pytest.mark.parametrize("tokens,experts,k,pad,cols,kind", ROWS)
def test_rows_there_and_back(pmn, tokens, experts, k, pad, cols, kind):
    x32 = problem(tokens, experts, "f32", 2, masked=tokens % 2 == 1 and tokens > 1)
    rows = pmn.route_rows(tokens, experts, k, pad) + 5
    r = pmn.route_topk(x32, k, pad=pad, rows=rows)
    choice, index, g = host(r.row_choice), host(r.row_index), host(r.gates).astype(np.float64)
    gen = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn((tokens, cols + 16), generator=gen, device="cuda").to(TYPES[kind])
    x = wide[:, 8:8 + cols]  # a strided view
    z = torch.randn((rows, cols), generator=gen, device="cuda").to(TYPES[kind])
    z[r.row_choice < 0] = float("nan")  # rows that no choice names are not read
    xs, zs = host(x).astype(np.float64), host(z).astype(np.float64)
    live, pads, tail = choice >= 0, choice == -1, choice == -2

    out = torch.full((rows, cols), 7.0, dtype=TYPES[kind], device="cuda")
    got = host(pmn.dispatch_rows(x, r.row_index, r.row_choice, out=out))
    assert np.array_equal(got[live], xs[choice[live] // k]) and (got[pads] == 0).all() and (got[tail] == 7).all()

    for gates in (r.gates, None):
        want, mag = np.zeros((2, tokens, cols))
        for i in range(k):
            on = index[:, i] >= 0
            w = g[on, i:i + 1] if gates is not None else 1.0
            want[on] += w * zs[index[on, i]]
            mag[on] += np.abs(w * zs[index[on, i]])
        for o in ("bf16", "f32"):
            if cols % (8 if o == "bf16" else 4) == 0:
                got = host(pmn.combine_rows(z, r.row_index, gates, out_dtype=TYPES[o])).astype(np.float64)
                assert (np.abs(got - want) <= k * U * mag * 1.01 + HALF[o] * np.abs(want)).all()

        dz0 = torch.full((rows, cols), 7.0, dtype=TYPES[kind], device="cuda")
        dout = x.contiguous()
        dz, dg = pmn.combine_rows_backward(dout, z, r.row_index, r.row_choice, gates, dz=dz0)
        dz, dg = host(dz).astype(np.float64), host(dg).astype(np.float64)
        w = g.reshape(-1)[choice[live], None] if gates is not None else 1.0
        want = w * xs[choice[live] // k]
        assert (np.abs(dz[live] - want) <= HALF[kind] * np.abs(want)).all()
        assert (dz[pads] == 0).all() and (dz[tail] == 7).all()
        want, mag = np.zeros((2, tokens, k))
        for i in range(k):
            on = index[:, i] >= 0
            want[on, i] = (xs[on] * zs[index[on, i]]).sum(1)
            mag[on, i] = np.abs(xs[on] * zs[index[on, i]]).sum(1)
        assert (np.abs(dg - want) <= (cols + 2) * U * mag).all()
    assert pmn.get_device_error() == 0


def test_a_row_named_twice_is_summed_twice(pmn):
    z = torch.randn((3, 8), device="cuda")
    idx = torch.tensor([[1, 1, -1], [2, 0, 2]], dtype=torch.int32, device="cuda")
    got = pmn.combine_rows(z, idx)
    assert torch.equal(got[0], z[1] + z[1]) and torch.equal(got[1], (z[2] + z[0]) + z[2])


def test_rows_beyond_the_tensor_are_skipped_and_reported(pmn):
    z, x = torch.ones((4, 8), device="cuda"), torch.ones((2, 8), device="cuda")
    idx = torch.tensor([[0, 4], [1 << 30, 3]], dtype=torch.int32, device="cuda")
    choice = torch.tensor([0, -1, -2, 3], dtype=torch.int32, device="cuda")
    out = torch.full((4, 8), 5.0, device="cuda")
    pmn.dispatch_rows(x, idx, choice, out=out)
    assert out[:, 0].tolist() == [1, 0, 5, 1]
    assert pmn.get_device_error() == pmn.DEVERR_BAD_OFFSETS
    assert pmn.combine_rows(z, idx)[:, 0].tolist() == [1, 1]
    assert pmn.get_device_error() == pmn.DEVERR_BAD_OFFSETS
    dz, dg = pmn.combine_rows_backward(x, z, idx, choice, dz=out.fill_(5.0))
    assert dz[:, 0].tolist() == [1, 0, 5, 1] and dg.tolist() == [[8, 0], [0, 8]]
    assert pmn.get_device_error() == pmn.DEVERR_BAD_OFFSETS and pmn.get_device_error() == 0


def test_captured_and_on_another_stream(pmn):
    """the whole way there and back in a graph on a stream of its own, replayed on other inputs"""
    tokens, experts, k, cols = 257, 50, 6, 264
    x, l = torch.randn((tokens, cols), device="cuda").bfloat16(), problem(tokens, experts, "f32", 1)

    def chain(s=None):
        r = pmn.route_topk(l, k, pad=16, stream=s)
        rows = pmn.dispatch_rows(x, r.row_index, r.row_choice, stream=s)
        out = pmn.combine_rows(rows, r.row_index, r.gates, stream=s)
        _, dg = pmn.combine_rows_backward(x, rows, r.row_index, r.row_choice, r.gates, stream=s)
        return out, pmn.route_topk_backward(l, r.experts, dg, stream=s)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    chain(s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        captured = chain()
    for seed in (2, 3):
        l.copy_(problem(tokens, experts, "f32", seed))
        x.copy_(torch.randn((tokens, cols), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, chain()):
            assert torch.equal(a, b)
