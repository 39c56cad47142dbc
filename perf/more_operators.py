"""The dense side of a feed-forward block and the step that follows its gradients, as cases to be
timed and compared: a linear layer with bias, activation and residual in its epilogue and its
backward, the gated feed-forward block and its backward, and the AdamW step over many tensors with
states in 32 or in 8 bits.

``own`` picks the side: the library's entry points, or the plain form in elementary torch
operations in 32 bits. ``exact`` gives the definition's values in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
# AdamW: a step in the middle of a run
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.95, 1e-8, 0.1, 1000
BLOCK = 256                                    # elements that share a scale of the 8-bit states
TINY = 2.0 ** -126                             # the smallest scale


# ------------------------------------------------------------------------------------ cases


def _linear(name, T, K, N, kind, layout, act, bias, residual):
    return dict(name=name, op="linear", T=T, K=K, N=N, type=kind, layout=layout, act=act, bias=bias, residual=residual)


def _linear_back(name, T, K, N, kind, layout, act, bias):
    return dict(name=name, op="linear_back", T=T, K=K, N=N, type=kind, layout=layout, act=act, bias=bias)


def listed():
    return [
        # The up projection of one decoded token (the decode workload's layer, dense).
        _linear("linear_token", 1, 4096, 14336, "bf16", "nk", "silu", True, False),
        # The down projection of a decode batch into the residual stream, the weights in the layout
        # of the sparse layer's down projection.
        _linear("linear_decode_down", 64, 14336, 4096, "bf16", "kn", "none", False, True),
        # The up projection of the prefill workload.
        _linear("linear_prefill", 4096, 2048, 8192, "bf16", "nk", "gelu", True, False),
        # Its backward, for a batch of an odd number of tokens.
        _linear_back("linear_back", 4093, 2048, 8192, "bf16", "nk", "gelu", True),
        # The backward of the small fp32 layer.
        _linear_back("linear_back_small", 128, 256, 1024, "f32", "kn", "relu", True),
        # The gated block of one decoded token.
        dict(name="gated_token", op="gated", T=1, d=4096, f=14336, type="bf16", act="silu", bias=False, residual=True,
             saved=False),
        # The gated block of a prefill batch.
        dict(name="gated_prefill", op="gated", T=4096, d=2048, f=8192, type="bf16", act="silu", bias=False,
             residual=True, saved=False),
        # An fp32 training forward of odd sizes, with biases.
        dict(name="gated_odd", op="gated", T=997, d=1000, f=2728, type="f32", act="gelu_tanh", bias=True,
             residual=False, saved=True),
        # The backward of the training workload's block.
        dict(name="gated_train_back", op="gated_back", T=16384, d=4096, f=14336, type="bf16", act="silu", bias=False),
        # The step of one small fp32 layer.
        dict(name="adamw_small", op="adamw", layers=1, d=256, f=1024, V=0, grad="f32", states=32, copy=False, clip=False),
        # Two layers of the prefill workload: fp32 master weights with bf16 copies, clipped.
        dict(name="adamw_layers", op="adamw", layers=2, d=2048, f=8192, V=0, grad="f32", states=32, copy=True, clip=True),
        # Two layers of the training workload and a head of 32000 rows, 8-bit states, bf16 gradients.
        dict(name="adamw8_large", op="adamw", layers=2, d=4096, f=14336, V=32000, grad="bf16", states=8, copy=True, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear_back", "gated", "gated_back", "adamw"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    # no dearer than the largest listed case (an fp32 product costs several bf16 ones)
    most = 16384 * 4096 * 14336 // (1 if kind == "bf16" else 32)
    if op in ("linear", "linear_back"):
        c = dict(op=op, T=_log(rng, 1, 16384), K=8 * _log(rng, 8, 1792), N=8 * _log(rng, 8, 1792), type=kind,
                 layout=rng.choice(["nk", "nk", "kn"]), act=rng.choice(ACTS), bias=rng.random() < 0.5)
        c["T"] = max(1, min(c["T"], most // (c["K"] * c["N"])))
        if op == "linear":
            c["residual"] = rng.random() < 0.5
        return c
    if op in ("gated", "gated_back"):
        c = dict(op=op, T=_log(rng, 1, 16384), d=8 * _log(rng, 8, 512), f=8 * _log(rng, 16, 1792), type=kind,
                 act=rng.choice(ACTS), bias=rng.random() < 0.3)
        c["T"] = max(1, min(c["T"], most // (c["d"] * c["f"])))
        if op == "gated":
            c.update(residual=rng.random() < 0.5, saved=rng.random() < 0.5)
        return c
    c = dict(op=op, layers=rng.randint(1, 3), d=8 * _log(rng, 8, 512), f=8 * _log(rng, 32, 1792),
             V=rng.choice([0, _log(rng, 500, 32000)]), grad=rng.choice(["f32", "bf16"]), states=rng.choice([32, 8]),
             copy=rng.random() < 0.5, clip=rng.random() < 0.5)
    c["layers"] = max(1, min(c["layers"], 2 * 4096 * 14336 // (c["d"] * c["f"])))
    return c


# ----------------------------------------------------------------------------------- inputs


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _weight(g, rows, cols, fan_in, t):
    return (_randn(g, rows, cols) / math.sqrt(fan_in)).to(t)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] in ("linear", "linear_back"):
        T, K, N, t = case["T"], case["K"], case["N"], TYPES[case["type"]]
        # normalised hidden states, and weights that keep their spread
        st = dict(op=case["op"], act=case["act"], layout=case["layout"], x=_randn(g, T, K).to(t),
                  w=_weight(g, N, K, K, t) if case["layout"] == "nk" else _weight(g, K, N, K, t))
        if case["op"] == "linear":
            st["b"] = 0.5 * _randn(g, N) if case["bias"] else None
            st["r"] = _randn(g, T, N).to(t) if case["residual"] else None
        else:
            st["bias"] = case["bias"]
            st["pre"] = _randn(g, T, N).to(t) if case["act"] != "none" else None
            st["dy"] = (_randn(g, T, N) / T).to(t)         # of a mean over the tokens
        return st
    if case["op"] in ("gated", "gated_back"):
        T, d, f, t = case["T"], case["d"], case["f"], TYPES[case["type"]]
        st = dict(op=case["op"], act=case["act"], x=_randn(g, T, d).to(t), wg=_weight(g, f, d, d, t),
                  wu=_weight(g, f, d, d, t), w2=_weight(g, f, d, f, t))
        if case["op"] == "gated":
            st["bg"] = 0.5 * _randn(g, f) if case["bias"] else None
            st["bu"] = 0.5 * _randn(g, f) if case["bias"] else None
            st["r"] = _randn(g, T, d).to(t) if case["residual"] else None
            st["saved"] = case["saved"]
        else:
            # the pre-activations that the forward saved
            st["g"], st["u"] = _randn(g, T, f).to(t), _randn(g, T, f).to(t)
            st["dy"] = (_randn(g, T, d) / T).to(t)
            st["bias"] = case["bias"]
        return st
    d, f = case["d"], case["f"]
    shapes = [(f, d), (f, d), (f,), (d,), (d,)] * case["layers"] + ([(case["V"], d)] if case["V"] else [])
    st = dict(op="adamw", states=case["states"], p=[], g=[], m=[], v=[], decay=[])
    for k, shape in enumerate(shapes):
        # gradients of a scale of their own per tensor and row, a step's noise on a mean
        size = 10.0 ** (-2 - k % 3) * torch.exp(_randn(g, shape[0]))
        size = size[:, None] if len(shape) == 2 else size
        st["p"].append(_randn(g, *shape) / math.sqrt(d))
        st["g"].append((size * _randn(g, *shape)).to(TYPES[case["grad"]]))
        st["m"].append(0.3 * size * _randn(g, *shape))
        st["v"].append((size * (0.1 + _randn(g, *shape).abs())).square())
        st["decay"].append(DECAY if len(shape) == 2 else 0.0)
    total = sum(t.double().square().sum() for t in st["g"])
    st["norm"] = total.sqrt().float() if case["clip"] else None
    st["max_norm"] = 1.0
    st["copy"] = [p.to(torch.bfloat16) for p in st["p"]] if case["copy"] else None
    if case["states"] == 8:
        packed = [_pack(m, v) for m, v in zip(st["m"], st["v"])]
        st["m"], st["ms"], st["v"], st["vs"] = (list(x) for x in zip(*packed))
    return st


# ------------------------------------------------------------------------------ plain forms


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _dact(z, act):
    """The activation's derivative."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(s):
    w = s["w"].float()
    z = s["x"].float() @ (w.t() if s["layout"] == "nk" else w)
    z = z if s["b"] is None else z + s["b"]
    y = _act(z, s["act"])
    return dict(y=(y if s["r"] is None else y + s["r"].float()).to(s["x"].dtype))


def _plain_linear_back(s):
    x, w, t = s["x"].float(), s["w"].float(), s["x"].dtype
    dz = s["dy"].float()
    dz = dz if s["pre"] is None else dz * _dact(s["pre"].float(), s["act"])
    nk = s["layout"] == "nk"
    out = dict(dx=(dz @ (w if nk else w.t())).to(t), dw=(dz.t() @ x if nk else x.t() @ dz).to(t))
    if s["bias"]:
        out["db"] = dz.sum(0)
    return out


def _plain_gated(s):
    x, t = s["x"].float(), s["x"].dtype
    g, u = x @ s["wg"].float().t(), x @ s["wu"].float().t()
    if s["bg"] is not None:
        g, u = g + s["bg"], u + s["bu"]
    y = (_act(g, s["act"]) * u) @ s["w2"].float()
    out = dict(y=(y if s["r"] is None else y + s["r"].float()).to(t))
    if s["saved"]:
        out["g"], out["u"] = g.to(t), u.to(t)
    return out


def _plain_gated_back(s):
    x, dy, g, u, t = s["x"].float(), s["dy"].float(), s["g"].float(), s["u"].float(), s["x"].dtype
    a = _act(g, s["act"])
    dh = dy @ s["w2"].float().t()
    dg, du = dh * u * _dact(g, s["act"]), dh * a
    out = dict(dx=(dg @ s["wg"].float() + du @ s["wu"].float()).to(t), dwg=(dg.t() @ x).to(t), dwu=(du.t() @ x).to(t),
               dw2=((a * u).t() @ dy).to(t))
    if s["bias"]:
        out["dbg"], out["dbu"] = dg.sum(0), du.sum(0)
    return out


# The 8-bit states. A block of 256 elements shares a scale s; m is q |q| s with q in -127 .. 127, v is
# q^4 s with q in 0 .. 255, and a v above zero takes q = 1 at least.


def _blocks(t):
    t = t.reshape(-1)
    return torch.nn.functional.pad(t, (0, -t.numel() % BLOCK)).view(-1, BLOCK)


def _unblock(b, like):
    return b.reshape(-1)[: like.numel()].view(like.shape)


def _scale(b, steps):
    return torch.clamp(b.abs().amax(1, keepdim=True) * (1 / steps), min=TINY)


def _pack(m, v):
    """(codes of m, scales of m, codes of v, scales of v)"""
    bm, bv = _blocks(m), _blocks(v)
    sm, sv = _scale(bm, 127.0 ** 2), _scale(bv, 255.0 ** 4)
    qm = torch.clamp(torch.round(torch.sqrt(bm.abs() * torch.reciprocal(sm))), max=127)
    qm = torch.where(bm < 0, -qm, qm)
    qv = torch.clamp(torch.round(torch.sqrt(torch.sqrt(bv * torch.reciprocal(sv)))), max=255)
    qv = torch.where(bv > 0, torch.clamp(qv, min=1), qv)
    return _unblock(qm, m).to(torch.int8), sm[:, 0], _unblock(qv, v).to(torch.uint8), sv[:, 0]


def _unpack(qm, sm, qv, sv):
    bm, bv = _blocks(qm.to(sm.dtype)), _blocks(qv.to(sv.dtype))
    bv = bv * bv
    return _unblock(bm * bm.abs() * sm[:, None], qm), _unblock(bv * bv * sv[:, None], qv)


def _adamw(p, g, m, v, decay, c):
    """(p, m, v) after the step; c: the clipping factor, None without one."""
    g = g.float()
    g = g if c is None else g * c
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    step = m / (torch.sqrt(v) * (1 / math.sqrt(1 - BETA2 ** STEP)) + EPS)
    return p * (1 - LR * decay) - step * (LR / (1 - BETA1 ** STEP)), m, v


def _keep(t, new):
    return t.copy_(new)


def _plain_adamw(s):
    c = None if s["norm"] is None else torch.clamp(s["max_norm"] / (s["norm"] + 1e-6), max=1.0)
    if s["states"] == 8:
        old = [_unpack(*q) for q in zip(s["m"], s["ms"], s["v"], s["vs"])]
    else:
        old = list(zip(s["m"], s["v"]))
    new = [_adamw(p, g, m, v, k, c) for p, g, (m, v), k in zip(s["p"], s["g"], old, s["decay"])]
    out = dict(p=[_keep(p, n[0]) for p, n in zip(s["p"], new)])
    if s["copy"] is not None:
        out["copy"] = [_keep(b, n[0]) for b, n in zip(s["copy"], new)]
    if s["states"] == 8:
        packed = [_pack(n[1], n[2]) for n in new]
        s["m"], s["ms"], s["v"], s["vs"] = (list(x) for x in zip(*packed))
        values = [_unpack(*q) for q in packed]
        out["m"], out["v"] = [x[0].bfloat16() for x in values], [x[1].bfloat16() for x in values]
    else:
        out["m"] = [_keep(t, n[1]) for t, n in zip(s["m"], new)]
        out["v"] = [_keep(t, n[2]) for t, n in zip(s["v"], new)]
    return out


# -------------------------------------------------------------------------------- one pass


def _own_run(s):
    import activation_sparse_transformer_up_amd as tw
    if s["op"] == "linear":
        y, _ = tw.linear_fwd(s["x"], s["w"], bias=s["b"], residual=s["r"], act=s["act"], w_layout=s["layout"])
        return dict(y=y)
    if s["op"] == "linear_back":
        dx, dw, db = tw.linear_bwd(s["dy"], s["x"], s["w"], pre=s["pre"], act=s["act"], w_layout=s["layout"],
                                   want_bias=s["bias"])
        return dict(dx=dx, dw=dw, db=db) if s["bias"] else dict(dx=dx, dw=dw)
    if s["op"] == "gated":
        y, g, u = tw.ffn_gated_dense_fwd(s["x"], s["wg"], s["wu"], s["w2"], bg=s["bg"], bu=s["bu"], residual=s["r"],
                                         act=s["act"], want_saved=s["saved"])
        return dict(y=y, g=g, u=u) if s["saved"] else dict(y=y)
    if s["op"] == "gated_back":
        dx, dwg, dwu, dw2, dbg, dbu = tw.ffn_gated_dense_bwd(s["dy"], s["x"], s["wg"], s["wu"], s["w2"], s["g"], s["u"],
                                                             act=s["act"], want_bias=s["bias"])
        out = dict(dx=dx, dwg=dwg, dwu=dwu, dw2=dw2)
        return dict(out, dbg=dbg, dbu=dbu) if s["bias"] else out
    eight = s["states"] == 8
    tw.adamw_step(s["p"], s["g"], s["m"], s["v"], lr=LR, step=STEP, betas=(BETA1, BETA2), eps=EPS, weight_decay=s["decay"],
                  norm=s["norm"], max_norm=s["max_norm"], copies=s["copy"], m_scales=s["ms"] if eight else None,
                  v_scales=s["vs"] if eight else None)
    m, v = s["m"], s["v"]
    if eight:
        values = tw.adamw8_values(m + v, s["ms"] + s["vs"], dtype=torch.bfloat16)
        m, v = values[: len(m)], values[len(m):]
    out = dict(p=s["p"], m=m, v=v)
    return out if s["copy"] is None else dict(out, copy=s["copy"])


def run(state):
    if own:
        return _own_run(state)
    return {"linear": _plain_linear, "linear_back": _plain_linear_back, "gated": _plain_gated,
            "gated_back": _plain_gated_back, "adamw": _plain_adamw}[state["op"]](state)


# ------------------------------------------------------------------------- needs and truth


def work(case):
    if case["op"] in ("linear", "linear_back"):
        T, K, N, e = case["T"], case["K"], case["N"], SIZE[case["type"]]
        if case["op"] == "linear":
            return {"bytes": e * (T * K + K * N + T * N * (2 if case["residual"] else 1)) + 4 * N * case["bias"],
                    "flops": 2 * T * K * N}
        return {"bytes": e * (2 * T * K + 2 * K * N + T * N * (1 if case["act"] == "none" else 2)) + 4 * N * case["bias"],
                "flops": 4 * T * K * N}
    if case["op"] in ("gated", "gated_back"):
        T, d, f, e = case["T"], case["d"], case["f"], SIZE[case["type"]]
        if case["op"] == "gated":
            return {"bytes": e * (3 * d * f + T * d * (3 if case["residual"] else 2) + 2 * T * f * case["saved"]) +
                    8 * f * case["bias"], "flops": 6 * T * d * f}
        return {"bytes": e * (6 * d * f + 3 * T * d + 2 * T * f) + 8 * f * case["bias"], "flops": 12 * T * d * f}
    n = case["layers"] * (2 * case["f"] * case["d"] + case["f"] + 2 * case["d"]) + case["V"] * case["d"]
    # states in and out; in 8 bits their values, in bf16, come back too
    states = 16 if case["states"] == 32 else 4 + 4
    return {"bytes": n * (8 + SIZE[case["grad"]] + states + 2 * case["copy"]), "flops": 16 * n}


def _f64(t):
    return None if t is None else t.to(torch.float64)


def _unit64(z, act):
    """(activation, derivative), from other forms than the plain ones."""
    if act == "relu":
        return torch.clamp(z, min=0), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, torch.addcmul(s, z, s * torch.sigmoid(-z))
    if act == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, torch.addcmul(phi, z, torch.exp(-z.square() / 2), value=1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        # (1 + tanh a) / 2 = sigmoid(2 a)
        a2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3))
        s = torch.sigmoid(a2)
        return z * s, s + z * s * torch.sigmoid(-a2) * (2 * math.sqrt(2 / math.pi)) * (1 + 0.134145 * z.square())
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "linear":
        w, r, b = _f64(s["w"]), _f64(s["r"]), _f64(s["b"])
        z = torch.mm(_f64(s["x"]), w.t() if s["layout"] == "nk" else w)
        y = _unit64(z if b is None else z.add_(b), s["act"])[0]
        return dict(y=y if r is None else y + r)
    if s["op"] == "linear_back":
        x, w, dz = _f64(s["x"]), _f64(s["w"]), _f64(s["dy"])
        if s["pre"] is not None:
            dz = dz * _unit64(_f64(s["pre"]), s["act"])[1]
        if s["layout"] == "nk":
            out = dict(dx=torch.mm(dz, w), dw=torch.mm(x.t(), dz).t())
        else:
            out = dict(dx=torch.mm(w, dz.t()).t(), dw=torch.mm(dz.t(), x).t())
        if s["bias"]:
            out["db"] = torch.mv(dz.t(), torch.ones(case["T"], dtype=dz.dtype, device=dz.device))
        return out
    if s["op"] == "gated":
        x, w2 = _f64(s["x"]), _f64(s["w2"])
        g, u = torch.mm(_f64(s["wg"]), x.t()).t(), torch.mm(_f64(s["wu"]), x.t()).t()
        if s["bg"] is not None:
            g, u = g + _f64(s["bg"])[None, :], u + _f64(s["bu"])[None, :]
        y = torch.mm(_unit64(g, s["act"])[0] * u, w2)
        out = dict(y=y if s["r"] is None else y + _f64(s["r"]))
        return dict(out, g=g, u=u) if s["saved"] else out
    if s["op"] == "gated_back":
        x, dy, u = _f64(s["x"]), _f64(s["dy"]), _f64(s["u"])
        a, da = _unit64(_f64(s["g"]), s["act"])
        du = torch.mm(_f64(s["w2"]), dy.t()).t()           # dh for now
        out = dict(dw2=torch.mm(dy.t(), a * u).t())
        dg = du * da * u
        du = du * a
        out.update(dx=torch.addmm(torch.mm(dg, _f64(s["wg"])), du, _f64(s["wu"])), dwg=torch.mm(x.t(), dg).t(),
                   dwu=torch.mm(x.t(), du).t())
        if s["bias"]:
            one = torch.ones(case["T"], dtype=dg.dtype, device=dg.device)
            out.update(dbg=torch.mv(dg.t(), one), dbu=torch.mv(du.t(), one))
        return out
    c = 1.0 if s["norm"] is None else min(1.0, s["max_norm"] / (float(s["norm"]) + 1e-6))
    out = dict(p=[], m=[], v=[], copy=[])
    for k, (p, g) in enumerate(zip(s["p"], s["g"])):
        p, g = _f64(p), _f64(g) * c
        if s["states"] == 8:
            m, v = _values64(s["m"][k], s["ms"][k]), _values64(s["v"][k], s["vs"][k])
        else:
            m, v = _f64(s["m"][k]), _f64(s["v"][k])
        m, v = torch.lerp(g, m, BETA1), torch.lerp(g.square(), v, BETA2)
        hat = (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)).sqrt() + EPS)
        p = p - LR * (hat + s["decay"][k] * p)
        if s["states"] == 8:
            m, v = _codes64(m, 127, 2), _codes64(v, 255, 4)
        for name, t in (("p", p), ("m", m), ("v", v), ("copy", p)):
            out[name].append(t)
    if s["copy"] is None:
        del out["copy"]
    return out


def _values64(q, scale):
    power = 2 if q.dtype == torch.int8 else 4
    each = _f64(scale).repeat_interleave(BLOCK)[: q.numel()].view(q.shape)
    q = _f64(q)
    return torch.sign(q) * q.abs().pow(power) * each


def _codes64(t, top, power):
    """The values that t's codes stand for: in every block the nearest code in the power's root."""
    flat = t.reshape(-1)
    pad = torch.zeros(-flat.numel() % BLOCK, dtype=flat.dtype, device=flat.device)
    b = torch.cat([flat, pad]).view(-1, BLOCK)
    scale = (b.abs().max(1).values / float(top) ** power).clamp(min=TINY)[:, None]
    q = (b.abs() / scale).pow(1.0 / power).round()
    if power == 4:
        q = torch.where((b > 0) & (q == 0), torch.ones_like(q), q)
    return (torch.sign(b) * q.pow(power) * scale).view(-1)[: flat.numel()].view(t.shape)
