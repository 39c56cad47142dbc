"""The operators that stand around the sparse feed-forward layer in a training or scoring step,
as cases to be timed and compared: layer norm (with the residual add) forward and backward, the
softmax cross entropy of a large vocabulary straight from hidden states and head weights, and
the global gradient norm with clipping.

``own`` picks the side: the library's entry points, or the plain form in elementary torch
operations in 32 bits. ``exact`` gives the definition's values in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS_LN = 1e-5
EPS_CLIP = 1e-6


# ------------------------------------------------------------------------------------ cases


def listed():
    return [
        # One token between two layers of a decode loop (the d of the decode workload).
        dict(name="norm_token", op="norm", T=1, d=4096, type="bf16", residual=True),
        # The pre-norm of a prefill batch, with the residual stream updated on the way.
        dict(name="norm_prefill", op="norm", T=4096, d=2048, type="bf16", residual=True),
        # The norm's backward in the training workload: the layer's backward hands over fp32 dy.
        dict(name="norm_train_back", op="norm_back", T=16384, d=4096, type="bf16", dy="f32", residual=True),
        # An fp32 layer of odd sizes, without a residual.
        dict(name="norm_back_odd", op="norm_back", T=997, d=1000, type="f32", dy="f32", residual=False),
        # The log-probability of one token during decoding.
        dict(name="xent_token", op="xent", T=1, d=4096, V=32000, type="bf16", ignored=0),
        # Scoring a short text, an odd vocabulary, the prompt's part without targets.
        dict(name="xent_score", op="xent", T=333, d=2048, V=50021, type="bf16", ignored=90),
        # A small fp32 model's loss and gradients (the fp32 workload's width).
        dict(name="xent_train_small", op="xent_back", T=128, d=256, V=1009, type="f32", ignored=16),
        # A training batch of the prefill workload's width.
        dict(name="xent_train", op="xent_back", T=4096, d=2048, V=32000, type="bf16", ignored=400),
        # A training batch at the training workload's width with a large vocabulary.
        dict(name="xent_train_large", op="xent_back", T=8192, d=4096, V=128000, type="bf16", ignored=0),
        # Gradients of one small fp32 layer.
        dict(name="clip_small", op="clip", layers=1, d=256, f=1024, V=0, max_norm=1.0),
        # Gradients of four layers of the prefill workload's shape, norm below the limit.
        dict(name="clip_layers", op="clip", layers=4, d=2048, f=8192, V=0, max_norm=1e9),
        # Two layers of the training workload and the bf16 head, clipped.
        dict(name="clip_large", op="clip", layers=2, d=4096, f=14336, V=128000, max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "xent", "xent_back", "clip"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_back"):
        c = dict(op=op, T=_log(rng, 1, 16384), d=8 * _log(rng, 8, 1024), type=kind, residual=rng.random() < 0.5)
        c["T"] = min(c["T"], 16384 * 4096 // c["d"] // (1 if kind == "bf16" else 2))
        if op == "norm_back":
            c["dy"] = rng.choice(["f32", kind])
        return c
    if op in ("xent", "xent_back"):
        c = dict(op=op, T=_log(rng, 1, 8192), d=8 * _log(rng, 8, 512), V=_log(rng, 500, 128000), type=kind)
        # no dearer than the largest listed case (an fp32 product costs several bf16 ones)
        most = 8192 * 4096 * 128000 // (1 if kind == "bf16" else 16)
        c["T"] = max(1, min(c["T"], most // (c["d"] * c["V"])))
        c["ignored"] = int(c["T"] * rng.choice([0, 0, 0.1, 0.5]))
        return c
    c = dict(op=op, layers=rng.randint(1, 8), d=8 * _log(rng, 8, 512), f=64 * _log(rng, 4, 224),
             V=rng.choice([0, _log(rng, 500, 128000)]), max_norm=rng.choice([1.0, 1e9]))
    c["layers"] = max(1, min(c["layers"], 4 * 4096 * 14336 // (2 * c["d"] * c["f"])))
    return c


# ----------------------------------------------------------------------------------- inputs


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] == "norm":
        T, d, t = case["T"], case["d"], TYPES[case["type"]]
        # a residual stream: unit spread, an offset of its own per token, a few large channels
        x = _randn(g, T, d) + 0.3 * _randn(g, T, 1)
        x[:, :: max(1, d // 8)] *= 8
        return dict(op="norm", x=x.to(t), r=_randn(g, T, d).to(t) if case["residual"] else None,
                    w=1 + 0.1 * _randn(g, d), b=0.1 * _randn(g, d))
    if case["op"] == "norm_back":
        T, d, t = case["T"], case["d"], TYPES[case["type"]]
        s = _randn(g, T, d) + 0.3 * _randn(g, T, 1)
        s[:, :: max(1, d // 8)] *= 8
        s = s.to(t)
        mean = s.double().mean(1)
        rstd = (s.double().var(1, unbiased=False) + EPS_LN).rsqrt()
        return dict(op="norm_back", s=s, dy=_randn(g, T, d).to(TYPES[case["dy"]]), w=1 + 0.1 * _randn(g, d),
                    mean=mean.float(), rstd=rstd.float(), dres=_randn(g, T, d).to(t) if case["residual"] else None)
    if case["op"] in ("xent", "xent_back"):
        T, d, V, t = case["T"], case["d"], case["V"], TYPES[case["type"]]
        w = (_randn(g, V, d) / math.sqrt(d)).to(t)
        y = torch.randint(0, V, (T,), generator=g, device=DEV)
        # hidden states of unit spread that lean towards their target by 0 to 16 units: from
        # tokens that the model cannot guess to tokens that it is sure of
        lean = 16 * torch.rand(T, 1, generator=g, device=DEV)
        x = (_randn(g, T, d) + lean * w[y].float()).to(t)
        y[torch.randperm(T, generator=g, device=DEV)[: case["ignored"]]] = -100
        n = T - case["ignored"]
        dloss = (0.5 + torch.rand(T, generator=g, device=DEV)) / max(1, n)
        st = dict(op=case["op"], x=x, w=w, y=y)
        if case["op"] == "xent_back":
            st["dloss"] = dloss
        return st
    grads = []
    d, f = case["d"], case["f"]
    for _ in range(case["layers"]):
        for k, shape in enumerate([(f, d), (f, d), (f,), (d,), (d,)]):
            grads.append(_randn(g, *shape) * 10.0 ** (-1 - k % 3))
    if case["V"]:
        grads.append((_randn(g, case["V"], d) * 1e-3).to(torch.bfloat16))
    return dict(op="clip", grads=grads, out=[torch.empty_like(t) for t in grads], max_norm=case["max_norm"])


# -------------------------------------------------------------------------------- one pass


def _plain_norm(s):
    x, t = s["x"].float(), s["x"].dtype
    if s["r"] is not None:
        x = (x + s["r"].float()).to(t).float()         # the residual stream is kept in its type
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS_LN)
    y = (xc * rstd * s["w"] + s["b"]).to(t)
    out = dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0])
    if s["r"] is not None:
        out["s"] = x.to(t)
    return out


def _plain_norm_back(s):
    x, dy = s["s"].float(), s["dy"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["w"]
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dict(dx=dx.to(s["s"].dtype), dw=(dy * xh).sum(0), db=dy.sum(0))


def _plain_xent(s):
    active = s["y"] >= 0
    x, w = s["x"].float(), s["w"].float()
    x = torch.where(active[:, None], x, torch.zeros_like(x))
    y = torch.where(active, s["y"], torch.zeros_like(s["y"]))[:, None]
    z = x @ w.t()
    m = z.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    zero = torch.zeros_like(m)
    out = dict(loss=torch.where(active[:, None], lse - z.gather(1, y), zero)[:, 0],
               lse=torch.where(active[:, None], lse, zero)[:, 0])
    if s["op"] == "xent_back":
        p = torch.exp(z - lse)
        p.scatter_add_(1, y, torch.full_like(m, -1.0))
        p *= torch.where(active, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
        out["dx"] = (p @ w).to(s["x"].dtype)
        out["dw"] = (p.t() @ x).to(s["w"].dtype)
    return out


def _plain_clip(s):
    total = sum(t.float().square().sum(dtype=torch.float64) for t in s["grads"])
    norm = total.sqrt().float()
    c = torch.clamp(s["max_norm"] / (norm + EPS_CLIP), max=1.0)
    return dict(norm=norm, out=[(t.float() * c).to(t.dtype) for t in s["grads"]])


def _own_run(s):
    import activation_sparse_transformer_up_amd as tw
    if s["op"] == "norm":
        y, r, mean, rstd = tw.layer_norm_fwd(s["x"], s["w"], s["b"], residual=s["r"], eps=EPS_LN)
        out = dict(y=y, mean=mean, rstd=rstd)
        if s["r"] is not None:
            out["s"] = r
        return out
    if s["op"] == "norm_back":
        dx, dw, db = tw.layer_norm_bwd(s["dy"], s["s"], s["w"], s["mean"], s["rstd"], dres=s["dres"])
        return dict(dx=dx, dw=dw, db=db)
    if s["op"] == "xent":
        loss, lse = tw.linear_xent_fwd(s["x"], s["w"], s["y"])
        return dict(loss=loss, lse=lse)
    if s["op"] == "xent_back":
        loss, lse, dx, dw = tw.linear_xent_fwd_bwd(s["x"], s["w"], s["y"], s["dloss"])
        return dict(loss=loss, lse=lse, dx=dx, dw=dw)
    norm, out = tw.grad_clip(s["grads"], s["max_norm"], out=s["out"])
    return dict(norm=norm, out=out)


def run(state):
    if own:
        return _own_run(state)
    return {"norm": _plain_norm, "norm_back": _plain_norm_back, "xent": _plain_xent, "xent_back": _plain_xent,
            "clip": _plain_clip}[state["op"]](state)


# ------------------------------------------------------------------------- needs and truth


def work(case):
    if case["op"] in ("norm", "norm_back"):
        T, d, e = case["T"], case["d"], SIZE[case["type"]]
        n = T * d
        if case["op"] == "norm":
            return {"bytes": n * e * (4 if case["residual"] else 2) + 8 * d + 8 * T, "flops": 8 * n}
        return {"bytes": n * (2 * e + SIZE[case["dy"]] + (e if case["residual"] else 0)) + 12 * d + 8 * T,
                "flops": 14 * n}
    if case["op"] in ("xent", "xent_back"):
        n, d, V, e = case["T"] - case["ignored"], case["d"], case["V"], SIZE[case["type"]]
        back = case["op"] == "xent_back"
        return {"bytes": (n * d + V * d) * e + (case["T"] * d + V * d) * e * back + 16 * case["T"],
                "flops": 2 * n * d * V * (3 if back else 1) + 4 * n * V}
    small = case["layers"] * (2 * case["f"] * case["d"] + case["f"] + 2 * case["d"])
    n = small + case["V"] * case["d"]
    return {"bytes": 2 * (4 * small + 2 * case["V"] * case["d"]), "flops": 3 * n}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if s["op"] == "norm":
        x = s["x"].to(f64)
        if s["r"] is not None:
            x = (x + s["r"].to(f64)).to(s["x"].dtype).to(f64)
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = torch.rsqrt(var + EPS_LN)
        out = dict(y=torch.addcmul(s["b"].to(f64), (x - mean[:, None]) * rstd[:, None], s["w"].to(f64)),
                   mean=mean, rstd=rstd)
        if s["r"] is not None:
            out["s"] = x
        return out
    if s["op"] == "norm_back":
        # from d y / d s written out per row: J^T (w dy), the statistics taken as given
        x, dy, rstd = s["s"].to(f64), s["dy"].to(f64), s["rstd"].to(f64)
        d = x.shape[1]
        unit = (x - s["mean"].to(f64)[:, None]) * rstd[:, None]
        wdy = dy * s["w"].to(f64)[None, :]
        along = torch.matmul(wdy.unsqueeze(1), unit.unsqueeze(2))[:, 0, 0] / d
        dx = (wdy - wdy.sum(1)[:, None] / d - unit * along[:, None]) * rstd[:, None]
        if s["dres"] is not None:
            dx += s["dres"].to(f64)
        ones = torch.ones(1, x.shape[0], dtype=f64, device=x.device)
        return dict(dx=dx, dw=(ones @ (dy * unit))[0], db=(ones @ dy)[0])
    if s["op"] in ("xent", "xent_back"):
        T, V = case["T"], case["V"]
        rows = torch.nonzero(s["y"] >= 0)[:, 0]
        x, w, y = s["x"][rows].to(f64), s["w"].to(f64), s["y"][rows]
        loss, lse = (torch.zeros(T, dtype=f64, device=x.device) for _ in range(2))
        back = s["op"] == "xent_back"
        dx = torch.zeros(T, case["d"], dtype=f64, device=x.device) if back else None
        dw = torch.zeros_like(w) if back else None
        for at in range(0, len(rows), 2048):
            xs, ys, rs = x[at:at + 2048], y[at:at + 2048], rows[at:at + 2048]
            logp = torch.mm(xs, w.t())
            total = torch.logsumexp(logp, 1)
            lse[rs] = total
            logp -= total[:, None]
            here = torch.arange(len(rs), device=x.device)
            lt = logp[here, ys]
            loss[rs] = -lt
            if back:
                p = logp.exp_()
                p[here, ys] = torch.expm1(lt)            # p - 1 without cancellation
                p *= s["dloss"][rs].to(f64)[:, None]
                dx[rs] = torch.mm(p, w)
                dw.addmm_(p.t(), xs)
        return dict(loss=loss, lse=lse, dx=dx, dw=dw) if back else dict(loss=loss, lse=lse)
    norm = torch.stack([torch.linalg.vector_norm(t.to(f64)) for t in s["grads"]]).square().sum().sqrt()
    c = min(1.0, s["max_norm"] / (float(norm) + EPS_CLIP))
    return dict(norm=norm, out=[t.to(f64) * c for t in s["grads"]])
