"""Measured cases of the operators around the MXFP8 gated feed-forward block: add + RMS norm to MXFP8 and
its backward, the gated projection and its backward, and the AdamW step.

Where `own` is false, run() computes the operators in float32 with elementary torch operations, rounded once
at the end; where it is true it calls the framework.  MXFP8 tensors are returned as their E4M3 values and
their E8M0 scale values (float8 views of the bytes, no copy).
"""
import math

import numpy as np
import torch

own = False

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
TYPES = {"bf16": BF16, "f32": F32}
EPS = 1e-6                                               # of the norm
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP = 3e-4, 0.9, 0.95, 1e-8, 0.1, 100
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of a serving loop: the call's latency
        dict(name="norm_1x4096", op="norm", rows=1, cols=4096, residual="bf16", train=False),
        # the layer's 16384 tokens, residual stream in bf16, with what the backward pass needs
        dict(name="norm_16384x4096_train", op="norm", rows=16384, cols=4096, residual="bf16", train=True),
        # a ragged last micro-batch on a float32 residual stream
        dict(name="norm_bwd_1021x1536_f32", op="norm_bwd", rows=1021, cols=1536, residual="f32"),
        # the layer's tokens
        dict(name="norm_bwd_16384x4096", op="norm_bwd", rows=16384, cols=4096, residual="bf16"),
        # one token through one (shared) expert while serving: the weights' bytes
        dict(name="gate_1_token", op="gate", experts=1, rows=1, d=4096, f=1536, train=False),
        # a serving batch of 64 tokens, top-8 over 24 experts: short ragged segments, not padded
        dict(name="gate_512_rows_24_experts", op="gate", experts=24, rows=512, d=4096, f=1536, train=False),
        # training: 1024 tokens top-8 over 24 experts, segments padded to 128 rows, both orientations of h kept
        dict(name="gate_8192_rows_train", op="gate", experts=24, rows=8192, d=4096, f=1536, train=True),
        # its backward: dH and SwiGLU's gradient, both orientations
        dict(name="gate_bwd_8192_rows", op="gate_bwd", experts=24, rows=8192, d=4096, f=1536),
        # all tokens through one shared expert
        dict(name="gate_bwd_16384_rows", op="gate_bwd", experts=1, rows=16384, d=4096, f=1536),
        # the norms, biases and router of a few layers: many small odd tensors, float32 everything
        dict(name="adamw_f32_130_small", op="adamw", param="f32", grad="f32", state="f32", tensors=130, numel=700001),
        # four experts' w1 and w2: float32 masters with bf16 copies
        dict(name="adamw_f32_75M", op="adamw", param="f32", grad="f32", state="f32", tensors=8, numel=75497472),
        # the same weights in bf16 without masters, states in 8 bits
        dict(name="adamw_mxfp8_75M", op="adamw", param="bf16", grad="bf16", state="mxfp8", tensors=8, numel=75497472),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gate", "gate_bwd", "adamw", "adamw"])
    if op in ("norm", "norm_bwd"):
        cols = 32 * _log(rng, 2, 256)
        case = dict(op=op, cols=cols, rows=_log(rng, 1, min(16384, 60_000_000 // cols)))
        case["residual"] = rng.choice(["bf16", "f32"] if op == "norm_bwd" else ["bf16", "f32", "none"])
        if op == "norm":
            case["train"] = rng.random() < 0.5
        return case
    if op == "adamw":
        tensors = _log(rng, 1, 200)
        return dict(op=op, param=rng.choice(["f32", "bf16"]), grad=rng.choice(["f32", "bf16"]),
                    state=rng.choice(["f32", "mxfp8"]), tensors=tensors, numel=_log(rng, max(1000, 40 * tensors), 60_000_000))
    d, f, experts = 512 * rng.randint(1, 8), 128 * rng.randint(1, 12), _log(rng, 1, 24)
    train = op == "gate_bwd" or rng.random() < 0.5
    rows = 128 * _log(rng, 1, 64) if train else _log(rng, 1, 8192)
    case = dict(op=op, experts=experts, rows=rows, d=d, f=f)
    if op == "gate":
        case["train"] = train
    return case


def sizes(case):
    """The tensors' lengths: unequal, most of them odd, `numel` in all."""
    k, left = case["tensors"], case["numel"]
    share = [1 + (i * 40503) % 97 for i in range(k)]
    got = [max(1, left * s // sum(share)) for s in share]
    got[0] += left - sum(got)
    return got


def segments(case, rng):
    """Row offsets of the experts: random shares, whole 128-row pads where the case trains."""
    unit = 128 if case.get("train", True) else 1
    cut = np.sort(rng.integers(0, case["rows"] // unit + 1, case["experts"] - 1)) * unit
    return np.concatenate([[0], cut, [case["rows"]]]).astype(np.int32)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, b = case["rows"] * case["cols"], {"bf16": 2, "f32": 4, "none": 0}[case["residual"]]
        if op == "norm":
            by = n * (2 + 2 * b + 33 / 32 + (2 if case["train"] else 0)) + case["cols"] * 2 + case["rows"] * 4
            return {"bytes": by, "flops": 7.0 * n}
        return {"bytes": n * (2 + 3 * b + (2 if b == 4 else 0)) + case["cols"] * 6 + case["rows"] * 4, "flops": 10.0 * n}
    if op == "adamw":
        p = {"f32": 10, "bf16": 4}[case["param"]]                       # read, written (and the bf16 copy)
        s = {"f32": 16, "mxfp8": 4 * 33 / 32}[case["state"]]
        return {"bytes": case["numel"] * (p + {"f32": 4, "bf16": 2}[case["grad"]] + s), "flops": 16.0 * case["numel"]}
    t, d, f, e, mx = case["rows"], case["d"], case["f"], min(case["experts"], case["rows"]), 33 / 32
    if op == "gate":
        out = t * f * mx * (2 if case["train"] else 1) + (t * 2 * f * 2 if case["train"] else 0)
        return {"bytes": (t * d + e * 2 * f * d) * mx + out, "flops": 4.0 * t * d * f}
    return {"bytes": (t * d + e * f * d) * mx + t * 2 * f * (2 + 2 * mx), "flops": 2.0 * t * d * f}


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, std=1.0, outliers=False):
    """bf16 ~ N(0, std^2); with outliers 0.1 % of the values are 30 times larger, as in a transformer's activations"""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=F32) * std
    if outliers:
        x = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.001, x * 30, x)
    return x.to(BF16)


def _empty(*shape, dtype=U8):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case, seed=seed)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        t, c = case["rows"], case["cols"]
        kind = TYPES.get(case["residual"])
        s["weight"] = (1.0 + 0.1 * torch.randn((c,), generator=gen, device="cuda")).to(BF16)
        if op == "norm":
            s["x"] = _normal(gen, (t, c), 0.5)
            s["residual_in"] = None if kind is None else _normal(gen, (t, c), 2.0, True).to(kind)
            s["res_out"] = None if kind is None else _empty(t, c, dtype=kind)
            s["out"] = (_empty(t, c), _empty(t, c // 32))
            s["y"] = _empty(t, c, dtype=BF16) if case["train"] else None
            s["rstd"] = _empty(t, dtype=F32) if case["train"] else None
        else:
            s["dy"] = _normal(gen, (t, c), 1e-3)
            s["r"] = _normal(gen, (t, c), 2.0, True).to(kind)
            s["rstd"] = torch.rsqrt(s["r"].double().square().mean(1) + EPS).to(F32)
            s["dres"] = _normal(gen, (t, c), 1e-3).to(kind)
            s["dr"] = _empty(t, c, dtype=kind)
            s["dx"] = _empty(t, c, dtype=BF16) if kind == F32 else None
            s["dw"] = _empty(c, dtype=F32)
            if own:
                from precision_moe_numerics_gb300 import pmn
                s["workspace"] = _empty(pmn.add_rmsnorm_backward_workspace_bytes(t, c))
    elif op == "adamw":
        # each tensor is a piece of one buffer per kind, as a program that reserves its memory at start-up has them
        n = sizes(case)
        pk, gk, eight = TYPES[case["param"]], TYPES[case["grad"]], case["state"] == "mxfp8"
        at = np.concatenate([[0], np.cumsum([k + -k % 32 for k in n])])
        live = torch.cat([torch.nn.functional.pad(torch.ones(k, dtype=torch.bool, device="cuda"), (0, -k % 32)) for k in n])
        s["lengths"], s["starts"] = n, at
        s["p"] = (_normal(gen, live.shape, 0.02) * live).to(pk)
        s["g"] = (_normal(gen, live.shape, 1e-3, True) * live).to(gk)
        s["copy"] = s["p"].to(BF16) if pk == F32 else None
        m = (_normal(gen, live.shape, 3e-4) * live).float()
        root = (_normal(gen, live.shape, 1e-3).float().abs() + 1e-5) * live
        s["m"], s["v"] = (mx_quantize(m), mx_quantize(root)) if eight else (m, root * root)
        s["grad_scale"] = torch.full((1,), 0.75, dtype=F32, device="cuda")  # a clipping factor, made on the device
        if own:  # the handle that a program builds once for its tensors
            from precision_moe_numerics_gb300 import pmn

            def pieces(x, unit=1):
                return [x[i // unit:-(-(i + k) // unit)] for i, k in zip(at.tolist(), n)]

            states = [list(zip(pieces(x[0]), pieces(x[1], 32))) if eight else pieces(x) for x in (s["m"], s["v"])]
            s["handle"] = pmn.AdamWTensors(pieces(s["p"]), pieces(s["g"]), *states,
                                           copies=pieces(s["copy"]) if pk == F32 else None)
    else:
        e, t, d, f = case["experts"], case["rows"], case["d"], case["f"]
        s["offsets"] = torch.from_numpy(segments(case, np.random.default_rng(seed))).cuda()
        if op == "gate":
            s["a"] = mx_quantize(_normal(gen, (t, d), 1.0, True).float())
            s["b"] = mx_quantize(_normal(gen, (e, 2 * f, d), 0.02).float())
            s["out"] = (_empty(t, f), _empty(t, f // 32))
            s["out_t"] = (_empty(f, t), _empty(f, t // 32)) if case["train"] else None
            s["y"] = _empty(t, 2 * f, dtype=BF16) if case["train"] else None
        else:
            s["a"] = mx_quantize(_normal(gen, (t, d), 1e-3, True).float())
            s["b"] = mx_quantize(_normal(gen, (e, f, d), 0.02).float())
            s["y"] = _normal(gen, (t, 2 * f), 1.3)
            s["out"] = (_empty(t, 2 * f), _empty(t, 2 * f // 32))
            s["out_t"] = (_empty(2 * f, t), _empty(2 * f, t // 32))
    return s


# ------------------------------------------------------------------ one pass
def _values(q):
    """an MXFP8 tensor's bytes as the values they stand for"""
    return q[0].view(F8), q[1].view(E8)


def run(state):
    if not own:
        return PLAIN[state["op"]](state)
    from precision_moe_numerics_gb300 import pmn
    s, op = state, state["op"]
    if op == "norm":
        pmn.add_rmsnorm_mxfp8(s["x"], s["residual_in"], s["weight"], EPS, out=s["out"], res_out=s["res_out"],
                              y=s["y"], rstd=s["rstd"])
        return dict(out=_values(s["out"]), r=s["res_out"], y=s["y"], rstd=s["rstd"])
    if op == "norm_bwd":
        pmn.add_rmsnorm_backward(s["dy"], s["r"], s["rstd"], s["weight"], dres=s["dres"], dr=s["dr"], dx=s["dx"],
                                 dw=s["dw"], workspace=s["workspace"])
        return dict(dr=s["dr"], dx=s["dx"], dw=s["dw"])
    if op == "gate":
        pmn.w1_gemm_swiglu_mxfp8(s["a"], s["b"], s["offsets"], out=s["out"], out_t=s["out_t"], y=s["y"])
        return dict(h=_values(s["out"]), h_t=_values(s["out_t"]) if s["out_t"] else None, y=s["y"])
    if op == "gate_bwd":
        pmn.dh_gemm_swiglu_backward_mxfp8(s["a"], s["b"], s["y"], s["offsets"], out=s["out"], out_t=s["out_t"])
        return dict(dy1=_values(s["out"]), dy1_t=_values(s["out_t"]))
    pmn.adamw_step(s["handle"], LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP, seed=s["seed"], grad_scale=s["grad_scale"])
    return _adamw_outputs(s)


def _adamw_outputs(s):
    eight = s["state"] == "mxfp8"
    return dict(p=s["p"], copy=s["copy"], m=_values(s["m"]) if eight else s["m"], v=_values(s["v"]) if eight else s["v"])


# ------------------------------------------------------------------ plain forms, float32
def _exponent(amax):
    """smallest e in [-127, 127] with amax <= 448 * 2^e; -127 for 0"""
    m, x = torch.frexp(amax)                      # amax = m * 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax == 0, torch.full_like(e, -127), e.clamp(-127, 127))


def mx_quantize(v):
    """float32 [..., C] -> MXFP8 along the last axis, round to nearest even: (E4M3 bytes, E8M0 bytes)"""
    b = v.reshape(*v.shape[:-1], -1, 32)
    e = _exponent(b.abs().amax(-1))
    q = (b * torch.ldexp(torch.ones_like(b[..., :1]), -e[..., None])).to(F8).view(U8)
    return q.reshape(v.shape), (e + 127).to(U8)


def mx_values(q, sc):
    return (q.view(F8).float().reshape(*sc.shape, 32) * sc.view(E8).float()[..., None]).reshape(q.shape)


def mx_flat_values(q):
    return mx_values(q[0].reshape(-1, 32), q[1][:, None]).reshape(-1)


def _plain_norm(s):
    x, res, w = s["x"].float(), s["residual_in"], s["weight"].float()
    r = x if res is None else (x + res.float()).to(res.dtype)
    rf = r.float()
    rstd = 1.0 / torch.sqrt((rf * rf).mean(1) + EPS)
    y = rf * rstd[:, None] * w
    return dict(out=_values(mx_quantize(y)), r=None if res is None else r, y=y.to(BF16) if s["train"] else None,
                rstd=rstd if s["train"] else None)


def _plain_norm_bwd(s):
    dy, r, rstd, w = s["dy"].float(), s["r"].float(), s["rstd"][:, None], s["weight"].float()
    xhat, g = r * rstd, dy * w
    dr = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True)) + s["dres"].float()
    return dict(dr=dr.to(s["r"].dtype), dx=dr.to(BF16) if s["dx"] is not None else None, dw=(dy * xhat).sum(0))


def _grouped_product(a, b, offsets):
    """a [T, K] times b[e]^T for the rows of each expert, in blocks of 128 rows"""
    if b.shape[0] == 1:
        return a @ b[0].t()
    t, e = a.shape[0], b.shape[0]
    o = offsets.long()
    ends = torch.cumsum((o[1:] - o[:-1] + 127) // 128, 0)
    blk = torch.arange(t // 128 + e, device=a.device)
    g = torch.searchsorted(ends, blk, right=True).clamp(max=e - 1)
    first = torch.cat([ends.new_zeros(1), ends[:-1]])[g]
    row = (o[g] + (blk - first) * 128)[:, None] + torch.arange(128, device=a.device)
    row = torch.where(row < o[g + 1][:, None], row, t)
    wide = torch.cat([a, a.new_zeros(1, a.shape[1])])
    out = a.new_empty(t + 1, b.shape[1])
    out[row] = wide[row] @ b[g].transpose(1, 2)
    return out[:t]


def _plain_gate(s):
    f = s["f"]
    y = _grouped_product(mx_values(*s["a"]), mx_values(*s["b"]), s["offsets"])
    g, u = y[:, :f], y[:, f:]
    h = g / (1.0 + torch.exp(-g)) * u
    return dict(h=_values(mx_quantize(h)), h_t=_values(mx_quantize(h.t().contiguous())) if s["train"] else None,
                y=y.to(BF16) if s["train"] else None)


def _plain_gate_bwd(s):
    f = s["f"]
    dh = _grouped_product(mx_values(*s["a"]), mx_values(*s["b"]), s["offsets"])
    g, u = s["y"][:, :f].float(), s["y"][:, f:].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    dy1 = torch.cat([dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg], 1)
    return dict(dy1=_values(mx_quantize(dy1)), dy1_t=_values(mx_quantize(dy1.t().contiguous())))


def _mulhilo(a, b):
    """high and low 32 bits of a * b for a constant and an int64 tensor of 32-bit values"""
    low = a * (b & 0xFFFF)
    mid = a * (b >> 16) + (low >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)


def random_bits(s, stream):
    """The 16 random bits of each element of the tensors laid end to end: Philox4x32-10, key = seed, counter (i / 16 lo,
    hi, 4 * tensor + stream, step) for element i of a tensor; word (i / 4) % 4 serves four elements: its low half, the
    low half reversed, its high half, the high half reversed."""
    starts = torch.from_numpy(s["starts"] // 16).cuda()
    j = torch.arange(int(s["starts"][-1]) // 16, device="cuda", dtype=torch.int64)
    which = torch.searchsorted(starts, j, right=True) - 1
    j = j - starts[which]
    c = [j & M32, j >> 32, 4 * which + stream, torch.full_like(j, STEP)]
    k0, k1 = s["seed"] & M32, (s["seed"] >> 32) & M32

    def ten_rounds(c, k0, k1, left):
        h0, l0 = _mulhilo(0xD2511F53, c[0])
        h1, l1 = _mulhilo(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        return c if left == 1 else ten_rounds(c, (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32, left - 1)

    w = torch.stack(ten_rounds(c, k0, k1, 10), 1)
    low, high = w & 0xFFFF, w >> 16
    return torch.stack([low, _reverse16(low), high, _reverse16(high)], 2).reshape(-1)


def _reverse16(x):
    x = ((x & 0x5555) << 1) | ((x >> 1) & 0x5555)
    x = ((x & 0x3333) << 2) | ((x >> 2) & 0x3333)
    x = ((x & 0x0F0F) << 4) | ((x >> 4) & 0x0F0F)
    return ((x & 0xFF) << 8) | (x >> 8)


def _stochastic_bf16(p, bits):
    """the 16 bits are added below bf16's last place, and a carry rounds away from zero"""
    raw = p.view(torch.int32).long() & M32
    return ((raw + bits) & 0xFFFF0000).to(torch.int32).view(F32).to(BF16)


def _stochastic_mx(v, bits, keep):
    """MXFP8 of a flat float32 tensor, E4M3 rounded stochastically; `keep`: a nonzero value takes the smallest
    code instead of 0"""
    b = v.reshape(-1, 32)
    e = _exponent(b.abs().amax(1))
    y = b.abs() * torch.ldexp(torch.ones_like(b[:, :1]), -e[:, None])
    ulp = torch.ldexp(torch.ones_like(y), (torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
    t = y / ulp
    q = torch.floor(t)
    up = torch.floor((t - q) * 65536.0).long() + bits.reshape(-1, 32) >= 65536
    q = ((q + up) * ulp).clamp(max=448.0)
    if keep:
        q = torch.where((q == 0) & (b != 0), torch.full_like(q, 2.0 ** -9), q)
    return torch.copysign(q, b).to(F8).view(U8).reshape(-1), (e + 127).to(U8)


def _plain_adamw(s):
    p, g, eight = s["p"], s["g"].float() * s["grad_scale"], s["state"] == "mxfp8"
    m, v = (mx_flat_values(s["m"]), mx_flat_values(s["v"]).square()) if eight else (s["m"], s["v"])
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * (g * g)
    bc1, bc2 = 1.0 - BETA1 ** STEP, 1.0 - BETA2 ** STEP
    new = p.float() * (1.0 - LR * DECAY) - (LR / bc1) * m / (torch.sqrt(v) / math.sqrt(bc2) + ADAM_EPS)
    if p.dtype == F32:
        p.copy_(new)
        s["copy"].copy_(new)
    else:
        p.copy_(_stochastic_bf16(new, random_bits(s, 0)))
    if eight:
        m = _stochastic_mx(m, random_bits(s, 1), False)
        v = _stochastic_mx(torch.sqrt(v), random_bits(s, 2), True)
        s["m"][0].copy_(m[0]), s["m"][1].copy_(m[1]), s["v"][0].copy_(v[0]), s["v"][1].copy_(v[1])
    else:
        s["m"].copy_(m), s["v"].copy_(v)
    return _adamw_outputs(s)


PLAIN = dict(norm=_plain_norm, norm_bwd=_plain_norm_bwd, gate=_plain_gate, gate_bwd=_plain_gate_bwd, adamw=_plain_adamw)


# ------------------------------------------------------------------ the definitions in 64 bits
def _double(q, sc):
    """an MXFP8 tensor's values from its bytes: sign, 4 exponent bits of bias 7, 3 mantissa bits"""
    b = q.to(torch.int64)
    exp, man = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(exp == 0, man * 2.0 ** -9, (8.0 + man) * torch.pow(2.0, (exp - 10).double()))
    val = torch.where(b >= 128, -mag, mag)
    rep = torch.pow(2.0, sc.double() - 127.0).repeat_interleave(32, dim=-1)
    return val * rep[..., :val.shape[-1]]


def _round_mx64(v, bits=None, keep=False):
    """(element values, scale values) of MXFP8 along the last axis, in doubles; the last block may be short"""
    n = v.shape[-1]
    blocks = torch.nn.functional.pad(v, (0, -n % 32)).unflatten(-1, (-1, 32))
    top = blocks.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0))
    e = torch.where(top > 448.0 * torch.pow(2.0, e), e + 1, e)          # log2's own rounding
    e = torch.where(top <= 448.0 * torch.pow(2.0, e - 1), e - 1, e)
    e = torch.where(top == 0, torch.full_like(e, -127.0), e.clamp(-127, 127))
    y = blocks / torch.pow(2.0, e)
    lsb = torch.pow(2.0, torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    lsb = torch.where(y.abs() >= 16 * lsb, 2 * lsb, torch.where((y.abs() < 8 * lsb) & (lsb > 2.0 ** -9), lsb / 2, lsb))
    if bits is None:
        q = torch.round(y / lsb) * lsb
    else:
        steps = (y / lsb).abs()
        low = torch.floor(steps)
        r = torch.nn.functional.pad(bits, (0, -n % 32)).unflatten(-1, (-1, 32))
        q = (low + (torch.floor((steps - low) * 65536) + r >= 65536)) * lsb
        if keep:
            q = torch.where((q == 0) & (blocks != 0), torch.full_like(q, 2.0 ** -9), q)
        q = q.clamp(max=448.0) * torch.sign(blocks)
    return q.flatten(-2)[..., :n], torch.pow(2.0, e).squeeze(-1)


def _rows64(a, b, o):
    """the grouped product, expert by expert"""
    return torch.cat([a[o[i]:o[i + 1]] @ _double(b[0][i], b[1][i]).t() for i in range(len(o) - 1)])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        r = s["x"].double()
        if s["residual_in"] is not None:  # the definition rounds the stream to its type
            r = (r + s["residual_in"].double()).to(s["residual_in"].dtype).double()
        rstd = (r.square().mean(1) + EPS).rsqrt()
        y = r * rstd[:, None] * s["weight"].double()
        return dict(out=_round_mx64(y), r=None if s["residual_in"] is None else r, y=y if case["train"] else None,
                    rstd=rstd if case["train"] else None)
    if op == "norm_bwd":
        dy, r, rs, w = (s[k].double() for k in ("dy", "r", "rstd", "weight"))
        n = r * rs[:, None]
        dr = rs[:, None] * (dy * w - n * (dy * w * n).sum(1, keepdim=True) / n.shape[1]) + s["dres"].double()
        return dict(dr=dr, dx=dr if s["dx"] is not None else None, dw=(dy * n).sum(0))
    if op in ("gate", "gate_bwd"):
        f = case["f"]
        z = _rows64(_double(*s["a"]), s["b"], s["offsets"].tolist())
        if op == "gate":
            h = z[:, :f] * torch.sigmoid(z[:, :f]) * z[:, f:]
            return dict(h=_round_mx64(h), h_t=_round_mx64(h.t().contiguous()) if case["train"] else None,
                        y=z if case["train"] else None)
        g, u = s["y"].double().split(f, 1)
        sg = torch.sigmoid(g)
        d = torch.cat([z * u * (sg + g * sg * (1 - sg)), z * g * sg], 1)
        return dict(dy1=_round_mx64(d), dy1_t=_round_mx64(d.t().contiguous()))
    eight = case["state"] == "mxfp8"
    c1, c2 = 1 - BETA1 ** STEP, 1 - BETA2 ** STEP
    p, g = s["p"].double(), s["g"].double() * s["grad_scale"].double()
    m, v = (_double(*s["m"]), _double(*s["v"]).square()) if eight else (s["m"].double(), s["v"].double())
    m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g * g
    p = p - LR * (DECAY * p + (m / c1) / ((v / c2).sqrt() + ADAM_EPS))
    if case["param"] == "bf16":  # rounded by the element's random bits
        q = torch.pow(2.0, torch.floor(torch.log2(p.abs().clamp(min=1e-30))) - 7)
        k = torch.floor(p.abs() / q)
        p = (k + (torch.floor((p.abs() / q - k) * 65536) + random_bits(s, 0) >= 65536)) * q * torch.sign(p)
    if eight:
        m, v = _round_mx64(m, random_bits(s, 1)), _round_mx64(v.sqrt(), random_bits(s, 2), True)
    return dict(p=p, copy=p if s["copy"] is not None else None, m=m, v=v)
