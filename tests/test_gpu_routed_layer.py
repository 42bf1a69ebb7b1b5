"""layer.RoutedExpertsStep and layer.RoutedDecode: the router, the rows and the products together, and the device's routing
in front of the calls that took it from the host.

Tolerances.  Along any path from an input to an output at most seven tensors are rounded to bf16 (xr is a copy; y, h, z, out
forward; dz, dY1, dX rows and dx back), each element by at most 2^-8 of itself: 7 * 2^-8 = 2.7 % of the norm.  Router gradients
pass through dgates in float32: the same bound.  NVFP4 weights are taken as the numbers they stand for."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
TOL = 7 * 2.0 ** -8


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, layer as m
    build.build()
    return m


def draw(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def close(got, want, what):
    err = (got.double() - want).norm() / want.norm()
    assert err <= TOL, (what, float(err))


def reference(x, logits, w1, w2, chosen, gates_of):
    """the layer in float64, choice by choice, with torch's own differentiation"""
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    gates = gates_of(logits)
    for t in range(x.shape[0]):
        for i, e in enumerate(chosen[t].tolist()):
            if e >= 0:
                g, u = (w1[e] @ x[t]).chunk(2)
                out[t] = out[t] + gates[t, i] * (w2[e] @ (torch.nn.functional.silu(g) * u))
    return out


@pytest.mark.parametrize("tokens,E,k,D,F,pad,score,normalize", [
    (40, 6, 2, 64, 48, 1, "softmax", True), (67, 9, 3, 72, 32, 32, "sigmoid", True), (70, 5, 5, 128, 16, 8, "softmax", False),
])
def test_routed_experts_and_their_gradients(layer, tokens, E, k, D, F, pad, score, normalize):
    from precision_moe_numerics_gb300 import pmn
    g = torch.Generator(device="cuda").manual_seed(tokens)
    w1, w2 = draw(g, E, 2 * F, D, std=2 * D ** -0.5), draw(g, E, D, F, std=F ** -0.5)
    x, logits, dout = draw(g, tokens, D), torch.randn((tokens, E), generator=g, device="cuda"), draw(g, tokens, D)
    logits[3] = -float("inf")  # a padding token
    step = layer.RoutedExpertsStep(tokens, w1, w2, k, score=getattr(pmn, "SCORE_" + score.upper()), normalize=normalize, pad=pad)
    for _ in range(2):  # the second time over used buffers
        out = step.forward(x, logits)
        dx, dlogits, dw1, dw2 = step.backward(dout)
    chosen = step.routing.experts.long()

    def gates_of(l):
        at = chosen.clamp(min=0)
        p = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
        q = torch.gather(torch.where(torch.isinf(l), torch.zeros_like(p), p), 1, at) * (chosen >= 0)
        return q / q.sum(1, keepdim=True).clamp(min=1e-30) if normalize else q

    xd, w1d, w2d = (t.double().requires_grad_() for t in (x, w1, w2))
    ld = logits.double().nan_to_num(neginf=-1e9).requires_grad_()
    want = reference(xd, ld, w1d, w2d, chosen, gates_of)
    (want * dout.double()).sum().backward()
    for a, b, what in ((out, want.detach(), "out"), (dx, xd.grad, "dx"), (dlogits, ld.grad, "dlogits"), (dw1, w1d.grad, "dw1"),
                       (dw2, w2d.grad, "dw2")):
        close(a, b, what)
    assert not out[3].any() and not dx[3].any() and not dlogits[3].any()
    assert pmn.get_device_error() == 0


def test_a_captured_step(layer):
    g = torch.Generator(device="cuda").manual_seed(1)
    w1, w2 = draw(g, 4, 64, 64, std=0.2), draw(g, 4, 64, 32, std=0.2)
    x, logits, dout = draw(g, 100, 64), torch.randn((100, 4), generator=g, device="cuda"), draw(g, 100, 64)
    step = layer.RoutedExpertsStep(100, w1, w2, 2)

    def whole():
        return [step.forward(x, logits), *step.backward(dout)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        whole()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        captured = whole()
    x.copy_(draw(g, 100, 64))
    logits.copy_(torch.randn((100, 4), generator=g, device="cuda"))
    want = [t.clone() for t in whole()]
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("tokens,k", [(1, 3), (5, 2), (40, 3)])
def test_routed_decode(layer, tokens, k):
    from precision_moe_numerics_gb300 import pmn
    g = torch.Generator(device="cuda").manual_seed(tokens)
    E, D, F = 7, 512, 256
    q1 = pmn.nvfp4_quantize(draw(g, E * 2 * F, D, std=0.1), outer_mode=pmn.OUTER_PER_GROUP, rows_per_group=2 * F)
    q2 = pmn.nvfp4_quantize(draw(g, E * D, F, std=0.1), outer_mode=pmn.OUTER_PER_GROUP, rows_per_group=D)
    w1 = q1[0].view(E, 2 * F, D // 2), q1[1].view(E, 2 * F, D // 16), q1[2]
    w2 = q2[0].view(E, D, F // 2), q2[1].view(E, D, F // 16), q2[2]
    x, logits = draw(g, tokens, D), torch.randn((tokens, E), generator=g, device="cuda")
    step = layer.RoutedDecode(tokens, w1, w2, k)
    out = step.forward(x, logits)
    from test_gpu_matvec import values
    v1, v2 = (torch.from_numpy(values([t.cpu().numpy() for t in w])).cuda() for w in (w1, w2))
    chosen = step.routing.experts.long()
    want = reference(x.double(), logits.double(), v1, v2, chosen, lambda l: torch.softmax(torch.gather(l, 1, chosen), 1))
    close(out, want, "out")
    assert pmn.get_device_error() == 0


def test_routing_made_here_is_the_hosts(layer):
    """the same layout as the host's routing, and the NVFP4 decode path and its combine on top of it"""
    from precision_moe_numerics_gb300 import pmn, workloads as W
    rng = np.random.default_rng(3)
    for tokens, experts, k, pad in ((64, 384, 8, 1), (500, 24, 4, 128)):
        logits = rng.standard_normal((tokens, experts), dtype=np.float32)
        want = W.route_topk(logits, k, pad)
        r = pmn.route_topk(torch.from_numpy(logits).cuda(), k, pad=pad)
        choice = r.row_choice.cpu().numpy()[:want.rows]
        assert np.array_equal(r.offsets.cpu().numpy(), want.offsets) and np.array_equal(r.experts.cpu().numpy(), want.topk)
        assert np.array_equal(np.where(choice >= 0, choice // k, -1), want.row_token)
        assert np.array_equal(r.row_index.cpu().numpy(), want.token_rows())
        assert np.allclose(r.gates.cpu().numpy(), want.gates, rtol=1e-5, atol=0)
    D, F, E, k, tokens = 512, 256, 6, 2, 33
    g = torch.Generator(device="cuda").manual_seed(5)
    q1 = pmn.nvfp4_quantize(draw(g, E * 2 * F, D, std=0.1), outer_mode=pmn.OUTER_PER_GROUP, rows_per_group=2 * F)
    q2 = pmn.nvfp4_quantize(draw(g, E * D, F, std=0.1), outer_mode=pmn.OUTER_PER_GROUP, rows_per_group=D)
    w1 = q1[0].view(E, 2 * F, D // 2), q1[1].view(E, 2 * F, D // 16), q1[2]
    w2 = q2[0].view(E, D, F // 2), q2[1].view(E, D, F // 16), q2[2]
    x, logits = draw(g, tokens, D), torch.randn((tokens, E), generator=g, device="cuda")
    r = pmn.route_topk(logits, k)
    rows = pmn.dispatch_rows(x, r.row_index, r.row_choice)
    decode = layer.DecodeForward(rows, w1, w2, r.offsets)
    decode.forward()
    out = pmn.combine_receive_s2f6(decode.z, decode.seed, r.row_index, r.gates)
    want = layer.RoutedDecode(tokens, w1, w2, k).forward(x, logits).double()
    # 4-bit activations twice (their E2M1 step is a quarter of a value at most, 2^-3 in the mean square of a uniform error of
    # half a step) and 6 bits of payload: within a third of the norm
    assert (out.double() - want).norm() / want.norm() <= 1 / 3
    assert pmn.get_device_error() == 0
