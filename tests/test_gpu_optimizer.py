"""adamw_step against a plain 64-bit implementation.

Tolerances.  u = 2^-24.  m and v: three roundings each, <= 4 u of the terms' magnitudes.  The step's quotient has
a relative error of at most 8 u beside m's, and p's update rounds twice: |p error| <= 2 u (|p| + |step|) + 12 u *
lr1 * M / d, with M the magnitude of m's terms.  Stochastic roundings compare the 16-bit fraction with 16 random
bits: a value with a relative error of 16 u moves its fraction by at most 16 * 16 u * 65536 < 1 unit (at most 16
E4M3 steps, 2^8 bf16 places of 2^-8: below 1 unit too), so the rounding is fixed wherever fraction + bits is
2 units or more from the carry; elsewhere either neighbour is right.  The sums of m and p may cancel, so their
relative errors against 64 bits have no such bound: the values that are rounded are the definition's float32 m and
p, formed here by the same float32 products, quotient and sums (and checked against 64 bits themselves)."""
import numpy as np
import pytest
import torch

import mx64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HP = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=7)
SIZES = [1, 7, 31, 32, 33, 511, 512, 513, 4095, 4096, 4097, 10001]


@pytest.fixture(scope="module")
def pmn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from precision_moe_numerics_gb300 import build, pmn as p
    build.build()
    return p


def f64(t):
    return t.double().cpu().numpy()


def test_philox_known_answers():
    w = mx64.philox([np.zeros(1, np.uint64)] * 4, 0)
    assert [int(x[0]) for x in w] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = np.full(1, 0xFFFFFFFF, np.uint64)
    w = mx64.philox([ones] * 4, 0xFFFFFFFFFFFFFFFF)
    assert [int(x[0]) for x in w] == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def make(sizes, pk, gk, eight, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def draw(n, std):
        return torch.randn((n,), generator=g, device="cuda") * std

    p = [draw(n, 0.05).to(pk) for n in sizes]
    gr = [draw(n, 1e-2).to(gk) for n in sizes]
    if not eight:
        return p, gr, [draw(n, 3e-3) for n in sizes], [draw(n, 1e-2).square() for n in sizes]

    def state(n, root):
        q = torch.randint(0, 127, (n,), generator=g, device="cuda", dtype=torch.uint8)
        if not root:
            q = q | (torch.randint(0, 2, (n,), generator=g, device="cuda", dtype=torch.uint8) << 7)
        return q, torch.randint(108, 115, ((n + 31) // 32,), generator=g, device="cuda", dtype=torch.uint8)

    return p, gr, [state(n, False) for n in sizes], [state(n, True) for n in sizes]


def values(x):
    return mx64.decode(x[0].cpu().numpy(), x[1].cpu().numpy()) if isinstance(x, tuple) else f64(x)


def rn(x):
    """float64 -> float32 -> float64; a fused product and sum of float32 values is rounded by one call"""
    return np.asarray(x, np.float32).astype(np.float64)


def m_and_p_in_float32(p, g, m, v, gs, root, lr, beta1, beta2, eps, weight_decay, step):
    g, m, v = rn(f64(g) * gs), values(m), values(v)
    v = rn(v * v) if root else v
    m = rn(rn(beta1) * m + rn(rn(1 - beta1) * g))
    v = rn(rn(beta2) * v + rn(rn(1 - beta2) * rn(g * g)))
    d = rn(m / rn(rn(np.sqrt(v)) * rn(1 / np.sqrt(1 - beta2 ** step)) + rn(eps)))
    return m, rn(-rn(lr / (1 - beta1 ** step)) * d + rn(f64(p) * rn(1 - lr * weight_decay)))


def clone(xs):
    return [tuple(t.clone() for t in x) if isinstance(x, tuple) else x.clone() for x in xs]


def reference(p, g, m, v, gs, root, lr, beta1, beta2, eps, weight_decay, step):
    g = f64(g) * gs
    m, v = values(m), values(v)
    v = v * v if root else v
    mass = beta1 * np.abs(m) + (1 - beta1) * np.abs(g)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    d = np.sqrt(v) / np.sqrt(1 - beta2 ** step) + eps
    lr1 = lr / (1 - beta1 ** step)
    new = f64(p) * (1 - lr * weight_decay) - lr1 * m / d
    tol = 2 * U * (np.abs(f64(p)) + np.abs(new)) + 16 * U * lr1 * mass / d
    return new, m, v, mass, tol


def check_sr(got, x, step_of, bits, what, least=0.0):
    """got: x rounded stochastically to multiples of step_of by `bits`"""
    t = np.abs(x) / step_of
    low = np.floor(t)
    f = (t - low) * 65536
    sure = np.abs(f + bits - 65536) >= 2
    want = (low + (np.floor(f) + bits >= 65536)) * step_of
    lowest = np.where((want == 0) & (x != 0), least, want) if np.any(least) else want
    err = np.abs(np.abs(got) - lowest)
    assert (err[sure] <= 1e-12 * np.abs(lowest[sure])).all(), "%s: %d wrong roundings" % (what, (err[sure] > 1e-12 * np.abs(lowest[sure])).sum())
    assert (np.abs(np.abs(got) - np.abs(x)) <= np.maximum(step_of, np.asarray(least)) * 1.001).all(), what
    assert ((np.sign(got) == np.sign(x)) | (got == 0)).all(), what


def check_mx_sr(q, sc, x, bits, what, keep):
    """MXFP8 of the float32-accurate x, E4M3 rounded stochastically; blocks whose maximum is within 2^-18 of a scale
    boundary may take either scale"""
    e = sc.cpu().numpy().astype(np.int64) - 127
    amax = np.abs(mx64.blocks(x)).max(-1)
    assert ((e >= mx64.exponent(amax * (1 - 2.0 ** -18))) & (e <= mx64.exponent(amax * (1 + 2.0 ** -18)))).all(), what
    s = np.repeat(np.ldexp(1.0, e), 32)[:x.size]
    y = np.abs(x) / s
    step = np.ldexp(1.0, np.maximum(np.frexp(np.maximum(y, 1e-300))[1] - 1, -6) - 3) * s
    got = mx64.decode(q.cpu().numpy(), sc.cpu().numpy())
    check_sr(got, x, step, bits, what, least=s * 2.0 ** -9 if keep else 0.0)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("gk", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pk", [torch.bfloat16, torch.float32])
def test_step(pmn, pk, gk, eight):
    p, g, m, v = make(SIZES, pk, gk, eight)
    copies = [torch.empty_like(x, dtype=torch.bfloat16) for x in p] if pk == torch.float32 else None
    gs = torch.full((1,), 0.3, device="cuda")
    old = [clone(x) for x in (p, m, v)]
    pmn.adamw_step(pmn.AdamWTensors(p, g, m, v, copies=copies), seed=12345678901, grad_scale=gs, **HP)
    for i, n in enumerate(SIZES):
        new, m64, v64, mass, tol = reference(old[0][i], g[i], old[1][i], old[2][i], float(gs.double()), eight, **HP)
        what = "n = %d" % n
        mf, pf = m_and_p_in_float32(old[0][i], g[i], old[1][i], old[2][i], float(gs.double()), eight, **HP)
        assert (np.abs(mf - m64) <= 4 * U * mass).all() and (np.abs(pf - new) <= tol).all(), what
        if pk == torch.float32:
            assert (np.abs(f64(p[i]) - new) <= tol).all(), what
            assert torch.equal(copies[i], p[i].to(torch.bfloat16)), what
        else:
            place = np.ldexp(1.0, np.frexp(np.maximum(np.abs(pf), 1e-300))[1] - 8)
            check_sr(f64(p[i]), pf, place, mx64.random_bits(n, 12345678901, 4 * i, HP["step"]), what)
        if eight:
            for k, (x, x64) in enumerate(((m[i], mf), (v[i], np.sqrt(v64)))):
                check_mx_sr(x[0], x[1], x64, mx64.random_bits(n, 12345678901, 4 * i + 1 + k, HP["step"]), what, k == 1)
        else:
            assert (np.abs(f64(m[i]) - m64) <= 4 * U * mass).all(), what
            assert (np.abs(f64(v[i]) - v64) <= 6 * U * v64).all(), what


def test_many_tensors_empty_ones_among_them(pmn):
    """more tensors than one launch holds, and the table of a single launch at each of its two sizes"""
    for count in (47, 48, 49, 441, 1000):
        sizes = [(i * 37) % 131 for i in range(count)]
        p, g, m, v = make(sizes, torch.float32, torch.float32, False, count)
        old = [clone(x) for x in (p, m, v)]
        pmn.adamw_step(pmn.AdamWTensors(p, g, m, v), **HP)
        P, G, M, V = [torch.cat(x) for x in (old[0], g, old[1], old[2])]
        new, m64, v64, mass, tol = reference(P, G, M, V, 1.0, False, **HP)
        assert (np.abs(f64(torch.cat(p)) - new) <= tol).all()
        assert (np.abs(f64(torch.cat(m)) - m64) <= 4 * U * mass).all()
    pmn.adamw_step(pmn.AdamWTensors([], [], [], []), **HP)


def test_a_tensor_past_32_bit_bytes(pmn):
    """the last elements of a tensor whose arrays are longer than 2^32 bytes"""
    n = (1 << 30) + 4099
    p = torch.zeros((n,), device="cuda")
    g = torch.zeros((n,), device="cuda")
    m, v = torch.zeros((n,), device="cuda"), torch.zeros((n,), device="cuda")
    g[-5000:] = torch.linspace(-1, 1, 5000, device="cuda")
    pmn.adamw_step(pmn.AdamWTensors([p], [g], [m], [v]), **HP)
    k = slice(n - 5000, n)
    zero = torch.zeros((5000,), device="cuda")
    new, m64, v64, mass, tol = reference(zero, g[k], zero, zero, 1.0, False, **HP)
    assert (np.abs(f64(p[k]) - new) <= tol).all() and (np.abs(f64(m[k]) - m64) <= 4 * U * mass).all()
    assert not p[:-5000].any()


def test_zero_states_zero_gradients(pmn):
    p = [torch.full((100,), 2.0, device="cuda")]
    g = [torch.zeros((100,), device="cuda")]
    m, v = pmn.adamw_states(p, mxfp8=True)
    pmn.adamw_step(pmn.AdamWTensors(p, g, m, v), **HP)
    assert (np.abs(f64(p[0]) - 2.0 * (1 - 1e-3)) <= 4 * U).all()
    assert not m[0][0].any() and not v[0][0].any() and not m[0][1].any() and not v[0][1].any()


def test_the_root_of_v_is_never_lost(pmn):
    """one large and 31 tiny gradients in a block: the tiny ones' second moments are below half the smallest code"""
    g = torch.full((32,), 1e-7, device="cuda")
    g[0] = 10.0
    p = [torch.zeros((32,), device="cuda")]
    m, v = pmn.adamw_states(p, mxfp8=True)
    pmn.adamw_step(pmn.AdamWTensors(p, [g], m, v), **HP)
    assert (v[0][0][1:] == 1).all()


def test_gradients_that_are_not_finite(pmn):
    for pk in (torch.bfloat16, torch.float32):
        for eight in (False, True):
            p, g, m, v = make([64], pk, torch.float32, eight, 3)
            g[0][5], g[0][40] = float("nan"), float("inf")
            pmn.adamw_step(pmn.AdamWTensors(p, g, m, v), **HP)
            bad = ~torch.isfinite(p[0])
            assert bad[5] and bad.sum() <= 2 and torch.isnan(p[0][5])


@pytest.mark.parametrize("pk", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan"), 3e19])
def test_neighbours_of_a_gradient_that_is_not_finite(pmn, bad, pk):
    """MXFP8 states: the 31 elements under the scale of one whose gradient is not finite (or overflows when squared)
    keep their states and train on, as in a run where that element's gradient is 0"""
    runs = []
    for value in (bad, 0.0):
        p, g, m, v = make([96], pk, torch.float32, True, 13)
        m[0][0][37] = v[0][0][37] = 0  # no part in its block's scale without the gradient
        g[0][37] = value
        h = pmn.AdamWTensors(p, g, m, v)
        pmn.adamw_step(h, **HP)
        first = clone(p) + clone(m) + clone(v)
        g[0][37] = 1e-2
        pmn.adamw_step(h, **{**HP, "step": 8})
        runs.append((first, p + m + v))
    others = torch.arange(96, device="cuda") != 37
    (first, second), (first0, second0) = runs
    finite_m = abs(bad) < float("inf")  # a large finite m raises its block's scale
    for x, y, keeps in zip(first, first0, (True, not finite_m, True)):
        x, y = (x, y) if isinstance(x, tuple) else ((x,), (y,))
        assert torch.equal(x[0][others], y[0][others]) or not keeps
        assert not keeps or all(torch.equal(a, b) for a, b in zip(x[1:], y[1:]))
    assert (first[2][0][37] & 127) == 127 and ((first[1][0][37] & 127) == 127 or finite_m)
    assert torch.isnan(second[0][37]) and torch.isfinite(second[0][others]).all()
    assert torch.isfinite(torch.from_numpy(values(second[2]) ** 2).float()[others.cpu()]).all()
    if not finite_m:
        assert torch.equal(second[0][others], second0[0][others])
    assert (second[0][others] != first[0][others]).float().mean() > 0.5


def one_step(pmn, p, g, m, v, **hp):
    """params after a step of float32 tensors whose factors are exact: beta1 = beta2 = 1/2, lr1 = 1, no decay"""
    t = [torch.tensor(np.asarray(x, np.float32), device="cuda") for x in (p, g, m, v)]
    pmn.adamw_step(pmn.AdamWTensors(*([x] for x in t)), **{**dict(lr=1.0, beta1=0.5, beta2=0.5, weight_decay=0.0, step=200), **hp})
    return f64(t[0])


def test_quotients_outside_float32s_range(pmn):
    """an infinite stored m, a quotient that overflows, a denominator whose reciprocal is subnormal"""
    # m and v are halved by the step, so that m / (sqrt(v) + eps) is as the comments say
    m, v = np.zeros(64), np.zeros(64)
    m[3], v[3] = np.inf, 2.0                # inf / 1
    m[9], v[9] = -np.inf, 0.0               # -inf / eps
    m[17], v[17] = 2e31, 0.0                # 1e31 / 1e-8: overflows
    m[33], v[33] = 2.0, 2.0                 # 1 / 1
    p = one_step(pmn, np.zeros(64), np.zeros(64), m, v, eps=1e-8)
    assert p[3] == -np.inf and p[9] == np.inf and p[17] == -np.inf and abs(p[33] + 1) <= 2e-7
    rest = np.delete(p, [3, 9, 17, 33])
    assert (rest == 0).all()
    m = np.full(64, 2e38)
    for eps in (2.0 ** 126, 1.5 * 2.0 ** 126, 3e38):
        p = one_step(pmn, np.zeros(64), np.zeros(64), m, np.zeros(64), eps=eps)
        want = rn(1e38) / rn(eps)
        assert (np.abs(p + want) <= 2.0 ** -22 * want).all()


def test_roots_and_quotients_of_one_newton_step(pmn):
    """p = -m / (sqrt(v) + eps) over the range of normal v and of m with its subnormals.

    The kernel's root and quotient are within one place of the correctly rounded ones, so within 1.5 places of the
    exact ones, a place being at most 2^-23 of the value (2^-149 below the normal range): 3 u each, u = 2^-24.  With
    eps = 2^-126 beside a root of 2^-63 and more the denominator is the root; with v = 0 it is eps."""
    rng = np.random.default_rng(17)
    n = 1 << 20
    v = np.exp2(rng.uniform(-125, 127.9, n)).astype(np.float32).astype(np.float64)
    v[:8] = 2.0 ** -125, 2.0 ** 127, 2.0, 8.0, np.float32(3.3e38), np.nextafter(np.float32(2) ** -125, np.float32(1)), 4.5, 2.0 ** -124
    m = np.where(np.arange(n) % 2 == 0, 2.0, np.exp2(rng.uniform(-20, 20, n)).astype(np.float32).astype(np.float64))
    p = one_step(pmn, np.zeros(n), np.zeros(n), m, v, eps=2.0 ** -126)
    want = m / 2 / np.sqrt(v / 2)
    assert (np.abs(-p / want - 1) <= 6.1 * U).all()
    for eps in (2.0 ** -126, 1e-30, 1e-8, 1.0, 3e7, 1e25, 2.0 ** 100):
        lo, hi = max(-148.0, np.log2(eps) - 124), min(127.9, np.log2(eps) + 126)
        m = np.exp2(rng.uniform(lo, hi, n)).astype(np.float32).astype(np.float64) * rng.choice([-1.0, 1.0], n)
        half = rn(m / 2)
        p = one_step(pmn, np.zeros(n), np.zeros(n), m, np.zeros(n), eps=eps)
        want = half / rn(eps)
        assert (np.abs(p + want) <= np.maximum(3 * U * np.abs(want), 1.5 * 2.0 ** -149)).all(), eps


def plain_step(p, g, m, v, seed, index, lr, beta1, beta2, eps, weight_decay, step):
    """one step in float32 torch operations, each rounded by itself; MXFP8 states, coded from their float32 values"""
    def value(x):
        return torch.from_numpy(values(x)).float().cuda()  # exact: 4 bits times a power of two

    m, v = value(m), value(v).square()  # (the square of 4 bits is exact too)
    g = g.float()
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * (g * g)
    p = p * (1.0 - lr * weight_decay) - lr / (1 - beta1 ** step) * m / (torch.sqrt(v) / (1 - beta2 ** step) ** 0.5 + eps)

    def coded(x, stream, keep):
        x = f64(x)
        e = mx64.exponent(np.abs(mx64.blocks(x)).max(-1))
        y = np.abs(x) / np.repeat(np.ldexp(1.0, e), 32)[:x.size]
        place = np.ldexp(1.0, np.maximum(np.frexp(np.maximum(y, 1e-300))[1] - 1, -6) - 3)
        low = np.floor(y / place)
        up = np.floor((y / place - low) * 65536) + mx64.random_bits(x.size, seed, 4 * index + stream, step) >= 65536
        q = np.minimum((low + up) * place, 448.0)
        if keep:
            q = np.where((q == 0) & (y > 0), 2.0 ** -9, q)
        return torch.from_numpy(np.copysign(q, x)).float().to(torch.float8_e4m3fn).view(torch.uint8), torch.from_numpy((e + 127).astype(np.uint8))

    return p, coded(m, 1, False), coded(torch.sqrt(v), 2, True)


@pytest.mark.parametrize("gk", [torch.bfloat16, torch.float32])
def test_float32_parameters_keep_the_states_of_plain_float32(pmn, gk):
    """the stochastic roundings are those of the formulas evaluated one operation at a time: two steps, a million
    elements, every code and scale equal, so that p stays within its roundings of plain float32"""
    sizes, seed = [1 << 20, 33, 70001], 77
    p, g, m, v = make(sizes, torch.float32, gk, True, 19)
    hp = dict(HP)
    for step in (7, 8):
        hp["step"] = step
        want = [plain_step(p[i], g[i], m[i], v[i], seed, i, **hp) for i in range(3)]
        old = clone(p)
        pmn.adamw_step(pmn.AdamWTensors(p, g, m, v), seed=seed, **hp)
        for i in range(3):
            for got, ref in ((m[i], want[i][1]), (v[i], want[i][2])):
                assert torch.equal(got[0].cpu(), ref[0]) and torch.equal(got[1].cpu(), ref[1])
            moved = (want[i][0] - old[i]).abs().double()
            err = (p[i].double() - want[i][0].double()).abs()
            assert (err <= 4 * U * (want[i][0].abs() + old[i].abs()).double() + 16 * U * moved).all()


def test_small_changes_of_v_are_kept_on_average(pmn):
    """beta2 = 0.99 moves v by at most 1 % a step, far below half a step of E4M3: rounding to nearest would leave it
    where it starts.  Stochastic rounding settles between the two neighbouring codes; their mean square is within
    (q2^2 - q1^2) / 4 * (q2 / q1 - 1) <= 0.9 % of v, plus 0.05 % of sampling over 65536 elements."""
    n, c = 65536, 0.37
    p, g = [torch.zeros((n,), device="cuda")], [torch.full((n,), c, device="cuda")]
    m, v = pmn.adamw_states(p, mxfp8=True)
    v[0][0].fill_(0x38)  # 1.0
    v[0][1].fill_(127)
    h = pmn.AdamWTensors(p, g, m, v)
    for t in range(1, 601):
        pmn.adamw_step(h, 1e-3, 0.9, 0.99, 1e-8, 0.0, t, seed=5)
    true = 0.99 ** 600 + (1 - 0.99 ** 600) * c * c
    assert abs((values(v[0]) ** 2).mean() / true - 1) < 0.02
    assert abs(values(m[0]).mean() / c - 1) < 0.005


def test_determinism_and_seeds(pmn):
    def once(seed):
        p, g, m, v = make([1000], torch.bfloat16, torch.bfloat16, True, 8)
        pmn.adamw_step(pmn.AdamWTensors(p, g, m, v), seed=seed, **HP)
        return p[0], m[0][0], v[0][0]
    a, b, c = once(1), once(1), once(2)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and not torch.equal(a[1], c[1])


def test_side_stream(pmn):
    p, g, m, v = make([5000], torch.float32, torch.float32, False, 4)
    q = clone(p) + clone(m) + clone(v)
    pmn.adamw_step(pmn.AdamWTensors([q[0]], g, [q[1]], [q[2]]), **HP)
    late = torch.zeros_like(g[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(g[0])
        pmn.adamw_step(pmn.AdamWTensors(p, [late], m, v), **HP)
    side.synchronize()
    assert torch.equal(p[0], q[0]) and torch.equal(m[0], q[1])


def test_refusals(pmn):
    p, g, m, v = make([64, 32], torch.float32, torch.float32, False)
    T = pmn.AdamWTensors
    bad = [dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(step=0),
           dict(weight_decay=float("inf"))]
    for b in bad:
        with pytest.raises(pmn.PmnError):
            pmn.adamw_step(T(p, g, m, v), **{**HP, **b})
    with pytest.raises(pmn.PmnError):
        T(p, g[:1], m, v)
    with pytest.raises(pmn.PmnError):
        T(p, [g[0], g[1].bfloat16()], m, v)                 # mixed gradient types
    with pytest.raises(pmn.PmnError):
        T(p, g, [m[0][:63], m[1]], v)                       # a short state
    with pytest.raises(pmn.PmnError):
        T([x.bfloat16() for x in p], g, m, v, copies=[x.bfloat16() for x in p])
    with pytest.raises(pmn.PmnError):
        T([x.cpu() for x in p], g, m, v)
    with pytest.raises(pmn.PmnError):
        pmn.adamw_step(T([torch.zeros((65,), device="cuda")[1:]], [g[0]], [m[0]], [v[0]]), **HP)  # alignment
    with pytest.raises(pmn.PmnError):
        pmn.adamw_step(T(p, g, m, v), grad_scale=torch.ones((2,), device="cuda"), **HP)
    assert pmn.get_device_error() == 0
