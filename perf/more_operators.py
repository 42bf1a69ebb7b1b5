"""Measured cases of the operators that carry tokens through an expert layer: the router, the moving of
rows into expert order and back, the bf16 products grouped by expert, and the products of a few rows with
4-bit weights.

Where `own` is false, run() computes the operators in float32 with elementary torch operations, rounded once
at the end; where it is true it calls the framework.
"""
import math

import numpy as np
import torch

own = False

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
TYPES = {"bf16": BF16, "f32": F32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode batch of 64 tokens over the layer's 384 experts: the call's latency
        dict(name="route_64x384_serve", op="route", tokens=64, experts=384, k=8, pad=1, logits="f32", score="softmax",
             normalize=True, bias=False, masked=False, train=False),
        # the layer's training batch: segments padded for the gradient GEMMs, and the logits' gradient
        dict(name="route_16384x384_train", op="route", tokens=16384, experts=384, k=8, pad=128, logits="f32",
             score="softmax", normalize=True, bias=False, masked=False, train=True),
        # the same batch's rows into expert order, and the gradient of its tokens
        dict(name="dispatch_16384x4096_train", op="rows", form="dispatch", tokens=16384, experts=384, k=8, pad=128,
             cols=4096, kind="bf16", masked=False, train=True),
        # a ragged last micro-batch in float32 whose padding tokens are not routed: the sum and its gradients
        dict(name="combine_1021x1536_f32_train", op="rows", form="combine", tokens=1021, experts=24, k=8, pad=32,
             cols=1536, kind="f32", masked=True, train=True),
        # the decode batch's sum over eight experts
        dict(name="combine_64x4096_serve", op="rows", form="combine", tokens=64, experts=384, k=8, pad=1, cols=4096,
             kind="bf16", masked=False, train=False),
        # the serving batch of 64 tokens, top-8 over 24 experts: the weights' bytes
        dict(name="w2_512_rows_24_experts", op="gemm", form="rows", experts=24, rows=512, d=4096, f=1536, out="bf16"),
        # training: 1024 tokens, top-8 over 24 experts, ragged segments; the pre-activations are kept
        dict(name="w1_8192_rows_24_experts_train", op="gemm", form="w1", experts=24, rows=8192, d=4096, f=1536, out="bf16"),
        # its input gradient, with the weights as they are stored
        dict(name="dx_8192_rows_24_experts", op="gemm", form="dx", experts=24, rows=8192, d=4096, f=1536, out="bf16"),
        # its weight gradients: sums over each expert's ragged rows
        dict(name="dw1_8192_rows_24_experts", op="gemm", form="dw", experts=24, rows=8192, d=4096, f=1536, out="f32"),
        # all tokens through one shared expert: the gradient of h and of its activation
        dict(name="dh_16384_rows_1_expert", op="gemm", form="dh", experts=1, rows=16384, d=4096, f=1536, out="bf16"),
        # one new token through its eight experts' gated projection, weights in 4 bits
        dict(name="matvec_w1_1_token", op="matvec", form="w1", tokens=1, experts=64, k=8, d=4096, f=1536, out="bf16"),
        # the decode batch through the second projections of the experts it hits
        dict(name="matvec_w2_64_tokens", op="matvec", form="w2", tokens=64, experts=384, k=8, d=4096, f=1536, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "rows", "rows", "gemm", "gemm", "gemm", "matvec", "matvec"])
    if op in ("route", "rows"):
        experts = _log(rng, 2, 512)
        case = dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, k=rng.randint(1, min(16, experts)),
                    pad=rng.choice([1, 8, 32, 128]), masked=rng.random() < 0.4, train=rng.random() < 0.6)
        if op == "route":
            case["experts"] = min(experts, 384)
            case["k"] = min(case["k"], 8)
            return dict(case, logits=rng.choice(["f32", "bf16"]), score=rng.choice(["softmax", "sigmoid"]),
                        normalize=rng.random() < 0.6, bias=rng.random() < 0.4)
        kind = rng.choice(["bf16", "f32"])
        cols = (8 if kind == "bf16" else 4) * _log(rng, 4, 512 if kind == "bf16" else 1024)
        limit = 16384 * 8 * 4096 * 2 // 2 // (case["k"] * cols * (2 if kind == "bf16" else 4))
        return dict(case, form=rng.choice(["dispatch", "combine"]), kind=kind, cols=cols,
                    tokens=max(1, min(case["tokens"], limit)))
    if op == "gemm":
        form = rng.choice(["rows", "w1", "dx", "dw", "dh"])
        case = dict(op=op, form=form, experts=_log(rng, 1, 48), rows=_log(rng, 1, 8192), d=8 * _log(rng, 8, 512),
                    f=16 * _log(rng, 4, 96))
        return dict(case, out="bf16" if form in ("w1", "dh") else rng.choice(["bf16", "f32"]))
    experts = _log(rng, 1, 256)
    return dict(op=op, form=rng.choice(["w1", "w2"]), tokens=_log(rng, 1, 64), experts=experts, k=rng.randint(1, min(8, experts)),
                d=256 * rng.randint(1, 16), f=256 * rng.randint(1, 6), out=rng.choice(["bf16", "f32"]))


def capacity(case):
    """rows that hold every choice whatever the experts' counts are"""
    n = case["tokens"] * case["k"]
    return (n + min(case["experts"], n) * (case["pad"] - 1)) // case["pad"] * case["pad"]


def segments(case, rng):
    """Row offsets of the experts: random shares of all rows, ragged, some of them empty."""
    cut = np.sort(rng.integers(0, case["rows"] + 1, case["experts"] - 1))
    return np.concatenate([[0], cut, [case["rows"]]]).astype(np.int32)


def dims(case):
    """(n, k) of the product's weights [experts, n, k] as they are stored"""
    d, f = case["d"], case["f"]
    return {"rows": (d, f), "w1": (2 * f, d), "dx": (2 * f, d), "dw": (2 * f, d), "dh": (d, f), "w2": (d, f)}[case["form"]]


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k, b = case["tokens"], case["experts"], case["k"], {"f32": 4, "bf16": 2}[case["logits"]]
        by = t * e * b + t * k * 12 + t * k * 4 + e * 4
        if case["train"]:  # the gradient needs the chosen logits, or all of them, and fills the whole matrix
            by += t * k * 8 + t * e * b + (t * e * b if case["score"] == "softmax" and not case["normalize"] else 0)
        return {"bytes": by, "flops": 4.0 * t * e}
    if op == "rows":
        t, k, c, b = case["tokens"], case["k"], case["cols"], {"f32": 4, "bf16": 2}[case["kind"]]
        by = (t + t * k) * c * b + t * k * 8
        if case["train"]:
            by += (t + t * k * (2 if case["form"] == "combine" else 1)) * c * b + t * k * 8
        return {"bytes": by, "flops": (4.0 if case["train"] else 2.0) * t * k * c}
    if op == "gemm":
        t, (n, k), b = case["rows"], dims(case), {"f32": 4, "bf16": 2}[case["out"]]
        e, f = min(case["experts"], t), case["f"]
        moved = {"rows": t * k * 2 + t * n * b, "w1": t * k * 2 + t * (n + f) * 2, "dx": t * n * 2 + t * k * b,
                 "dh": t * n * 2 + t * 4 * f * 2, "dw": t * (n + k) * 2}[case["form"]]
        weights = case["experts"] * n * k * b if case["form"] == "dw" else e * n * k * 2
        return {"bytes": moved + weights, "flops": 2.0 * t * n * k}
    t, (n, k), b = case["tokens"], dims(case), {"f32": 4, "bf16": 2}[case["out"]]
    rows = t * case["k"]
    hit = case["experts"] * (1.0 - (1.0 - case["k"] / case["experts"]) ** t)  # experts that some token chooses
    act = rows * (n // 2 if case["form"] == "w1" else n) * b + (t if case["form"] == "w1" else rows) * k * 2
    return {"bytes": hit * n * k * 9 / 16 + act, "flops": 2.0 * rows * n * k}


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, std=1.0, outliers=False):
    """N(0, std^2); with outliers 0.1 % of the values are 30 times larger, as in a transformer's activations"""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=F32) * std
    if outliers:
        x = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.001, x * 30, x)
    return x


def _zeros(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _logits(case, gen):
    """router logits, some experts more popular than others; masked: a tenth of the tokens are padding, which is
    routed nowhere, and each token is kept from a tenth of the experts"""
    t, e = case["tokens"], case["experts"]
    x = _normal(gen, (t, e), 1.5) + _normal(gen, (e,), 0.5)
    if case["masked"]:
        off = torch.rand((t, e), generator=gen, device="cuda") < 0.1
        off |= torch.rand((t, 1), generator=gen, device="cuda") < 0.1
        x = torch.where(off, torch.full_like(x, -math.inf), x)
    return x


def _nvfp4(gen, experts, n, k):
    """4-bit weights as a quantiser leaves them: E2M1 codes of normal values under an E4M3 scale per 16 and one
    float32 scale per expert, made a few experts at a time"""
    codes, scales = _zeros(experts, n, k // 2, dtype=U8), _zeros(experts, n, k // 16, dtype=U8)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (1 << 26) // (n * k))
    for e in range(0, experts, step):
        w = torch.randn((min(step, experts - e), n, k // 16, 16), generator=gen, device="cuda")
        s = (w.abs().amax(-1, keepdim=True) * 16).to(torch.float8_e4m3fn)
        q = torch.bucketize(w.abs() * 96 / s.float(), edges, out_int32=True).to(U8) + (w < 0).to(U8) * 8
        q = q.view(w.shape[0], n, k // 2, 2)
        codes[e:e + step] = q[..., 0] | (q[..., 1] << 4)
        scales[e:e + step] = s[..., 0].view(U8)
    outer = torch.rand((experts,), generator=gen, device="cuda") * 1e-4 + 2e-4
    return codes, scales, outer


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        s["x"] = _logits(case, gen).to(TYPES[case["logits"]])
        s["b"] = _normal(gen, (e,), 0.3) if case["bias"] else None
        s["dgates"] = _normal(gen, (t, k), 1e-2)
        s["capacity"] = capacity(case)
        if own:
            from precision_moe_numerics_gb300 import pmn
            s["out"] = pmn.Routing(_zeros(t, k, dtype=I32), _zeros(t, k, dtype=F32), _zeros(t, k, dtype=I32),
                                   _zeros(s["capacity"], dtype=I32), _zeros(e + 1, dtype=I32))
            s["workspace"] = _zeros(pmn.route_topk_workspace_bytes(t, e, k), dtype=U8)
            s["dlogits"] = torch.empty_like(s["x"])
    elif op == "rows":
        t, k, c, kind = case["tokens"], case["k"], case["cols"], TYPES[case["kind"]]
        r = capacity(case)
        route = _route(_logits(case, gen), None, k, case["pad"], r, "softmax", True)
        s.update(row_index=route["row_index"], row_choice=route["row_choice"], gates=route["gates"])
        s["token_rows"], s["routed_rows"] = _zeros(t, c, dtype=kind), _zeros(r, c, dtype=kind)
        if case["form"] == "dispatch" or case["train"]:
            s["x"] = _normal(gen, (t, c), 1.0, True).to(kind)           # tokens, or the gradient of their sums
        if case["form"] == "combine" or case["train"]:
            s["z"] = _normal(gen, (r, c), 0.5).to(kind)                 # routed rows, or their gradient
        s["dgates"] = _zeros(t, k, dtype=F32)
    elif op == "gemm":
        t, e, d, f, form = case["rows"], case["experts"], case["d"], case["f"], case["form"]
        n, k = dims(case)
        s["segments"] = segments(case, np.random.default_rng(seed)).tolist()
        s["offsets"] = torch.tensor(s["segments"], dtype=I32, device="cuda")
        a = {"rows": f, "w1": d, "dx": 2 * f, "dw": 2 * f, "dh": d}[form]
        s["a"] = _normal(gen, (t, a), 1.0 if form in ("rows", "w1") else 1e-2, form == "w1").to(BF16)
        if form == "dw":
            s["x"] = _normal(gen, (t, d), 1.0, True).to(BF16)
            s["out_rows"] = _zeros(e, n, k, dtype=TYPES[case["out"]])
        else:
            s["w"] = torch.randn((e, n, k), generator=gen, device="cuda", dtype=BF16) * 0.02
            s["out_rows"] = _zeros(t, {"rows": d, "w1": f, "dx": d, "dh": 2 * f}[form], dtype=TYPES[case["out"]])
        s["y"] = {"w1": lambda: _zeros(t, 2 * f), "dh": lambda: _normal(gen, (t, 2 * f), 1.3).to(BF16)}.get(form, lambda: None)()
    else:
        t, e, k = case["tokens"], case["experts"], case["k"]
        n, width = dims(case)
        lay = dict(tokens=t, experts=e, k=k, pad=1, masked=False)
        route = _route(_logits(lay, gen), None, k, 1, t * k, "softmax", True)
        s["offsets"], s["row_choice"] = route["offsets"], route["row_choice"]
        s["segments"] = s["offsets"].tolist()
        s["w"] = _nvfp4(gen, e, n, width)
        s["x"] = _normal(gen, (t if case["form"] == "w1" else t * k, width), 1.0, True).to(BF16)
        s["out_rows"] = _zeros(t * k, n // 2 if case["form"] == "w1" else n, dtype=TYPES[case["out"]])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if not own:
        return PLAIN[state["op"]](state)
    from precision_moe_numerics_gb300 import pmn
    s, op, form = state, state["op"], state.get("form")
    if op == "route":
        score = pmn.SCORE_SOFTMAX if s["score"] == "softmax" else pmn.SCORE_SIGMOID
        r = pmn.route_topk(s["x"], s["k"], bias=s["b"], score=score, normalize=s["normalize"], pad=s["pad"], out=s["out"],
                           workspace=s["workspace"])
        out = dict(experts=r.experts, gates=r.gates, row_index=r.row_index, row_choice=r.row_choice, offsets=r.offsets)
        if s["train"]:
            out["dlogits"] = pmn.route_topk_backward(s["x"], r.experts, s["dgates"], score=score, normalize=s["normalize"],
                                                     dlogits=s["dlogits"])
        return out
    if op == "rows" and form == "dispatch":
        out = dict(rows=pmn.dispatch_rows(s["x"], s["row_index"], s["row_choice"], out=s["routed_rows"]))
        if s["train"]:
            out["dx"] = pmn.combine_rows(s["z"], s["row_index"], out=s["token_rows"])
        return out
    if op == "rows":
        out = dict(out=pmn.combine_rows(s["z"], s["row_index"], s["gates"], out=s["token_rows"]))
        if s["train"]:
            out["dz"], out["dgates"] = pmn.combine_rows_backward(s["x"], s["z"], s["row_index"], s["row_choice"], s["gates"],
                                                                 dz=s["routed_rows"], dgates=s["dgates"])
        return out
    if op == "gemm":
        if form == "w1":
            h, y = pmn.w1_gemm_swiglu_bf16(s["a"], s["w"], s["offsets"], out=s["out_rows"], y=s["y"])
            return dict(h=h, y=y)
        if form == "dh":
            return dict(dy1=pmn.dh_gemm_swiglu_backward_bf16(s["a"], s["w"], s["y"], s["offsets"], out=s["out_rows"]))
        if form == "dw":
            return dict(dw=pmn.grouped_gemm_bf16(s["a"], s["x"], s["offsets"], pmn.GROUP_K, out=s["out_rows"]))
        return dict(out=pmn.grouped_gemm_bf16(s["a"], s["w"], s["offsets"], pmn.GROUP_M, b_transposed=form == "dx",
                                              out=s["out_rows"]))
    gated = form == "w1"
    return dict(out=pmn.matvec_nvfp4(s["x"], s["w"], s["offsets"], row_choice=s["row_choice"] if gated else None,
                                     k=s["k"] if gated else 1, swiglu=gated, out=s["out_rows"]))


# ------------------------------------------------------------------ plain forms, float32
def _route(logits, bias, k, pad, rows, score, normalize):
    x = logits.float()
    t, e = x.shape
    order, expert = torch.sort(x if bias is None else x + bias, dim=1, descending=True, stable=True)
    kept = order[:, :k] > -math.inf
    expert = torch.where(kept, expert[:, :k], e)
    l = torch.where(kept, torch.gather(x, 1, expert.clamp(max=e - 1)), torch.full_like(order[:, :k], -math.inf))
    if score == "sigmoid" and normalize:
        v = torch.where(kept, torch.clamp(l, max=0.0) - torch.log1p(torch.exp(-l.abs())), l)  # log of the sigmoid
        p = _softmax(v, v)
    elif score == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        p = _softmax(l, l if normalize else x)
    gates = torch.where(kept, p, torch.zeros_like(p))
    flat = expert.reshape(-1)
    by_expert = torch.sort(flat, stable=True)[1]  # rows of an expert in the order of their tokens
    count = torch.zeros(e + 1, dtype=torch.int64, device=x.device).index_add_(0, flat, torch.ones_like(flat))
    ends = torch.cumsum((count[:e] + pad - 1) // pad * pad, 0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    first = torch.cumsum(count, 0) - count
    at = flat[by_expert]
    row = torch.arange(t * k, device=x.device) - first[at] + offsets[at.clamp(max=e - 1)]
    row = torch.where(at < e, row, rows)
    row_index = torch.empty_like(flat)
    row_index[by_expert] = torch.where(at < e, row, -1)
    row_choice = torch.where(torch.arange(rows + 1, device=x.device) < offsets[e], -1, -2)
    row_choice[row] = by_expert
    return dict(experts=torch.where(kept, expert, -1).to(I32), gates=gates, row_index=row_index.view(t, k).to(I32),
                row_choice=row_choice[:rows].to(I32), offsets=offsets.to(I32))


def _softmax(v, among):
    """e^v over the sum of e^among along the rows; 0 where a row holds nothing"""
    top = among.amax(1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    total = torch.exp(among - top).sum(1, keepdim=True)
    return torch.exp(v - top) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_route(s):
    out = _route(s["x"], s["b"], s["k"], s["pad"], s["capacity"], s["score"], s["normalize"])
    if s["train"]:
        x, e, d = s["x"].float(), out["experts"].long(), s["dgates"]
        kept, g = e >= 0, out["gates"]
        dot = (d * g).sum(1, keepdim=True)
        if s["score"] == "softmax":
            inner = g * (d - dot)
        else:
            sg = 1.0 / (1.0 + torch.exp(-torch.gather(x, 1, e.clamp(min=0))))
            inner = g * (d - dot) * (1.0 - sg) if s["normalize"] else d * g * (1.0 - sg)
        full = torch.zeros_like(x)
        if s["score"] == "softmax" and not s["normalize"]:
            full -= _softmax(x, x) * dot
            inner = g * d
        full.scatter_add_(1, e.clamp(min=0), torch.where(kept, inner, torch.zeros_like(inner)))
        out["dlogits"] = full.to(s["x"].dtype)
    return out


def _gathered(z, row_index):
    """the rows of every token's choices [tokens, k, cols], zeros for a dropped one"""
    wide = torch.cat([z, z.new_zeros(1, z.shape[1])])
    return wide[row_index.long()]  # -1 is the last row


def _plain_rows(s):
    c, k = s["row_choice"].long(), s["k"]
    live, pad = (c >= 0)[:, None], (c == -1)[:, None]

    def rows_of(tokens, weights=None):
        r = tokens[c.clamp(min=0) // k]
        r = r if weights is None else r.float() * weights.reshape(-1)[c.clamp(min=0)][:, None]
        return torch.where(live, r, torch.zeros_like(r)).to(s["routed_rows"].dtype)

    if s["form"] == "dispatch":
        out = dict(rows=torch.where(live | pad, rows_of(s["x"]), s["routed_rows"]))
        if s["train"]:
            dx = torch.zeros(s["x"].shape, device=c.device)
            for i in range(k):
                dx += _gathered(s["z"], s["row_index"][:, i]).float()
            out["dx"] = dx.to(s["x"].dtype)
        return out
    total = torch.zeros(s["token_rows"].shape, device=c.device)
    for i in range(k):
        total += s["gates"][:, i:i + 1] * _gathered(s["z"], s["row_index"][:, i]).float()
    out = dict(out=total.to(s["token_rows"].dtype))
    if s["train"]:
        out["dz"] = torch.where(live | pad, rows_of(s["x"], s["gates"]), s["routed_rows"])
        out["dgates"] = torch.stack([(s["x"].float() * _gathered(s["z"], s["row_index"][:, i]).float()).sum(1)
                                     for i in range(k)], 1)
    return out


def _plain_gemm(s):
    o, form, f = s["segments"], s["form"], s["f"]
    out = torch.zeros_like(s["out_rows"])
    y = s["y"] if form == "dh" else torch.zeros_like(s["y"]) if form == "w1" else None
    for e in range(len(o) - 1):
        r = slice(o[e], o[e + 1])
        a = s["a"][r].float()
        if form == "dw":
            out[e] = a.t() @ s["x"][r].float()
        elif a.shape[0] == 0:
            continue
        elif form == "rows":
            out[r] = (a @ s["w"][e].float().t()).to(out.dtype)
        elif form == "dx":
            out[r] = (a @ s["w"][e].float()).to(out.dtype)
        elif form == "w1":
            z = a @ s["w"][e].float().t()
            y[r] = z.to(BF16)
            out[r] = (z[:, :f] / (1.0 + torch.exp(-z[:, :f])) * z[:, f:]).to(BF16)
        else:
            dh = a @ s["w"][e].float()
            g, u = y[r, :f].float(), y[r, f:].float()
            sg = 1.0 / (1.0 + torch.exp(-g))
            out[r] = torch.cat([dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg], 1).to(BF16)
    if form == "w1":
        return dict(h=out, y=y)
    return {"dh": dict(dy1=out), "dw": dict(dw=out)}.get(form, dict(out=out))


def _weights(w, e, dtype=F32):
    """expert e's 4-bit weights as numbers [n, k], without the expert's own scale"""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=dtype, device="cuda")
    q = w[0][e].to(I32)
    v = torch.stack([table[q & 15], table[q >> 4]], -1).reshape(q.shape[0], -1, 16)
    return (v * w[1][e].view(torch.float8_e4m3fn).to(dtype)[..., None]).reshape(q.shape[0], -1)


def _rows_in(s, r):
    return s["x"][s["row_choice"][r].long() // s["k"]] if s["form"] == "w1" else s["x"][r]


def _plain_matvec(s):
    o, out = s["segments"], torch.zeros_like(s["out_rows"])
    for e in range(len(o) - 1):
        r = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            continue
        y = _rows_in(s, r).float() @ (_weights(s["w"], e) * s["w"][2][e]).t()
        if s["form"] == "w1":
            g, u = y.split(s["f"], 1)
            y = g / (1.0 + torch.exp(-g)) * u
        out[r] = y.to(out.dtype)
    return dict(out=out)


PLAIN = dict(route=_plain_route, rows=_plain_rows, gemm=_plain_gemm, matvec=_plain_matvec)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_route(case, s):
    x32 = s["x"].float().cpu().numpy()
    choose = x32 if s["b"] is None else x32 + s["b"].cpu().numpy()  # the choice is by this float32 sum
    t, k = case["tokens"], case["k"]
    experts = np.argsort(-choose, axis=1, kind="stable")[:, :k]
    experts[np.take_along_axis(choose, experts, 1) == -np.inf] = -1
    counts = np.array([(experts == e).sum() for e in range(case["experts"])])
    offsets = np.concatenate([[0], np.cumsum(-(-counts // case["pad"]) * case["pad"])])
    choice = np.full(s["capacity"], -2)
    choice[:offsets[-1]] = -1
    index = np.full(t * k, -1)
    for e in range(case["experts"]):
        mine = np.flatnonzero(experts.reshape(-1) == e)
        choice[offsets[e]:offsets[e] + len(mine)] = mine
        index[mine] = offsets[e] + np.arange(len(mine))
    out = dict(experts=experts, row_index=index.reshape(t, k), row_choice=choice, offsets=offsets)
    out = {n: torch.from_numpy(v).to(I32).cuda() for n, v in out.items()}
    x = s["x"].double().requires_grad_()
    p = torch.softmax(x.nan_to_num(neginf=-1e300), 1) if case["score"] == "softmax" else torch.sigmoid(x)
    p = p * (x > -math.inf)
    chosen = torch.gather(p, 1, out["experts"].long().clamp(min=0)) * (out["experts"] >= 0)
    if case["normalize"]:
        if case["score"] == "softmax":  # the same quotients from shares that cannot all vanish
            l = torch.gather(x, 1, out["experts"].long().clamp(min=0))
            chosen = torch.softmax(torch.where(out["experts"] >= 0, l, torch.full_like(l, -1e300)), 1) * (out["experts"] >= 0)
        else:
            chosen = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-300)
    out["gates"] = chosen.detach()
    if case["train"]:
        (chosen * s["dgates"].double()).sum().backward()
        out["dlogits"] = torch.where(x.detach() > -math.inf, x.grad, torch.zeros_like(x.grad))
    return out


def _exact_rows(case, s):
    c, k = s["row_choice"].long(), case["k"]
    index, gates = s["row_index"].long(), s["gates"].double()
    at = torch.nonzero(c >= 0)[:, 0]
    token = c[at] // k

    def summed(weights):
        out = torch.zeros(s["token_rows"].shape, dtype=torch.float64, device="cuda")
        for i in range(k):
            t = torch.nonzero(index[:, i] >= 0)[:, 0]
            out[t] += weights[t, i, None] * s["z"][index[t, i]].double()
        return out

    if case["form"] == "dispatch":
        rows = torch.zeros(s["routed_rows"].shape, dtype=torch.float64, device="cuda")
        rows[at] = s["x"][token].double()
        return dict(rows=rows, dx=summed(torch.ones_like(gates))) if case["train"] else dict(rows=rows)
    out = dict(out=summed(gates))
    if case["train"]:
        dz = torch.zeros(s["routed_rows"].shape, dtype=torch.float64, device="cuda")
        dz[at] = gates.reshape(-1)[c[at], None] * s["x"][token].double()
        dg = torch.zeros(gates.numel(), dtype=torch.float64, device="cuda")
        for i in range(0, len(at), 8192):
            r, t = at[i:i + 8192], token[i:i + 8192]
            dg[c[r]] = torch.einsum("rc,rc->r", s["x"][t].double(), s["z"][r].double())
        out.update(dz=dz, dgates=dg.view(gates.shape))
    return out


def _exact_gemm(case, s):
    o, form, f = s["segments"], case["form"], case["f"]
    out = torch.zeros(s["out_rows"].shape, dtype=torch.float64, device="cuda")
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda") if form == "w1" else None
    for e, (lo, hi) in enumerate(zip(o[:-1], o[1:])):
        a = s["a"][lo:hi].double()
        if form == "dw":
            out[e] = torch.einsum("tn,tk->nk", a, s["x"][lo:hi].double())
            continue
        z = torch.einsum("tk,nk->tn" if form in ("rows", "w1") else "tn,nk->tk", a, s["w"][e].double())
        if form == "w1":
            y[lo:hi] = z
            z = z[:, :f] * torch.sigmoid(z[:, :f]) * z[:, f:]
        elif form == "dh":
            g, u = s["y"][lo:hi].double().split(f, 1)
            sg = torch.sigmoid(g)
            z = torch.cat([z * u * (sg + g * sg * (1 - sg)), z * g * sg], 1)
        out[lo:hi] = z
    if form == "w1":
        return dict(h=out, y=y)
    return dict(dy1=out) if form == "dh" else dict(dw=out) if form == "dw" else dict(out=out)


def _exact_matvec(case, s):
    out = torch.zeros(s["out_rows"].shape, dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(zip(s["segments"][:-1], s["segments"][1:])):
        if lo == hi:
            continue
        y = torch.einsum("rk,nk->rn", _rows_in(s, slice(lo, hi)).double(), _weights(s["w"], e, torch.float64))
        y = y * s["w"][2][e].double()
        if case["form"] == "w1":
            y = y[:, :case["f"]] * torch.sigmoid(y[:, :case["f"]]) * y[:, case["f"]:]
        out[lo:hi] = y
    return dict(out=out)


def exact(case, seed):
    return dict(route=_exact_route, rows=_exact_rows, gemm=_exact_gemm, matvec=_exact_matvec)[case["op"]](case, prepare(case, seed))
