"""Gradients of the dense layers against central differences of their forwards in fp32, argument by argument, along the
gradient itself, where the slope is its length. The allowance is the sum of what is known: the forwards' rounding
(their bound element by element, times |dy|, over the step), the difference quotient's own error, taken from the formulas
in 64 bits, and 2^-12 of the slope for the gradient's rounding (sums of up to 48 terms in three stages, 200 2^-24 at
most of absolute values that add up to less than 16 times the slope). It is held below a tenth of the slope, so that no
wrong gradient fits. Also here: infinities through relu, and that the example's losses are numbers."""
import importlib.util
import math
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
STEP = 2.0 ** -5


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    return z


def size(a, b):
    """The bound of an fp32 product's rounding."""
    return (a.shape[1] + 4) * E * (a.abs() @ b.abs())


def linear64(p, act):
    """(y, its rounding's bound, the activation's arguments)"""
    z = p["x"] @ p["w"].t() + p["b"]
    tz = size(p["x"], p["w"].t()) + 2 * E * z.abs()
    y = act64(z, act)
    return y, 1.2 * tz + 16 * E * (1 + z.abs()) + 2 * E * y.abs(), z


def gated64(p, act):
    g, u = p["x"] @ p["wg"].t() + p["bg"], p["x"] @ p["wu"].t() + p["bu"]
    tg, tu = size(p["x"], p["wg"].t()) + 2 * E * g.abs(), size(p["x"], p["wu"].t()) + 2 * E * u.abs()
    a = act64(g, act)
    h = a * u
    th = (1.2 * tg + 16 * E * (1 + g.abs())) * (u.abs() + tu) + a.abs() * tu + 2 * E * h.abs()
    return h @ p["w2"], size(h, p["w2"]) + th @ p["w2"].abs() + 2 * E * (h @ p["w2"]).abs(), g


OPS = {
    "linear": (linear64, lambda p, act: tw.linear_fwd(p["x"], p["w"], bias=p["b"], act=act)[0],
               lambda T, d, f: dict(x=(T, d), w=(f, d), b=(f,)), lambda T, d, f: (T, f)),
    "gated": (gated64, lambda p, act: tw.ffn_gated_dense_fwd(p["x"], p["wg"], p["wu"], p["w2"], bg=p["bg"], bu=p["bu"], act=act)[0],
              lambda T, d, f: dict(x=(T, d), wg=(f, d), wu=(f, d), w2=(f, d), bg=(f,), bu=(f,)), lambda T, d, f: (T, d)),
}


def gradients(op, p, dy, act):
    if op == "linear":
        _, pre = tw.linear_fwd(p["x"], p["w"], bias=p["b"], act=act, want_pre=True)
        return dict(zip(("x", "w", "b"), tw.linear_bwd(dy, p["x"], p["w"], pre=pre, act=act, want_bias=True)))
    _, g, u = tw.ffn_gated_dense_fwd(p["x"], p["wg"], p["wu"], p["w2"], bg=p["bg"], bu=p["bu"], act=act, want_saved=True)
    return dict(zip(("x", "wg", "wu", "w2", "bg", "bu"),
                    tw.ffn_gated_dense_bwd(dy, p["x"], p["wg"], p["wu"], p["w2"], g, u, act=act, want_bias=True)))


def inputs(op, act, seed, T=6, d=16, f=48):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shapes, out = OPS[op][2](T, d, f), OPS[op][3](T, d, f)
    p = {k: randn(g, *s) * (1 if k == "x" else 0.3 if len(s) == 1 else s[1 if k != "w2" else 0] ** -0.5) for k, s in shapes.items()}
    return p, randn(g, *out)


@pytest.mark.parametrize("act", list(tw.ACTS))
@pytest.mark.parametrize("op,name", [(op, k) for op in OPS for k in OPS[op][2](1, 8, 8)])
def test_slopes(op, name, act):
    f64, forward = OPS[op][:2]
    for seed in range(400):                          # relu: inputs none of whose arguments changes its sign on the way
        p, dy = inputs(op, act, seed)
        grad = gradients(op, p, dy, act)[name]
        along = grad.double() / grad.double().norm()
        ends = [dict(p, **{name: (p[name].double() + k * STEP * along).float()}) for k in (1, -1)]
        wide = [{k: v.double() for k, v in e.items()} for e in ends]
        (up, tu, zu), (down, td, zd) = (f64(e, act) for e in wide)
        if act != "relu" or not bool((zu * zd <= 0).any()):
            break
    else:
        raise AssertionError("no such inputs")
    move = wide[0][name] - wide[1][name]             # as rounded
    at = {k: v.double().requires_grad_(k == name) for k, v in p.items()}
    (f64(at, act)[0] * dy.double()).sum().backward()
    want = float((at[name].grad * move).sum())       # twice the step times the slope, all of them
    quotient = float(((up - down) * dy.double()).sum())
    rounding = float(((tu + td) * dy.double().abs()).sum())
    got = float(((forward(ends[0], act).double() - forward(ends[1], act).double()) * dy.double()).sum())
    slope = float((grad.double() * move).sum())
    tol = rounding + abs(quotient - want) + 2.0 ** -12 * abs(want)
    say(op, name, act, "slope", slope, "difference", got, "tol", tol)
    assert abs(want) > 0 and tol < 0.1 * abs(want), (tol, want, rounding, quotient)
    assert abs(got - slope) <= tol, (got, slope, tol)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinities_through_relu(dtype):
    """An infinite input: units whose weight of it is above zero are infinite, those below are zero."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x, w = randn(g, 70, 136).to(dtype), randn(g, 200, 136).to(dtype)
    w[:, 5] = torch.where(w[:, 5] == 0, torch.ones_like(w[:, 5]), w[:, 5])
    x[13, 5] = math.inf
    y = tw.linear_fwd(x, w, act="relu")[0]
    up = w[:, 5] > 0
    assert bool(up.any()) and bool((~up).any())
    assert bool((y[13][up] == math.inf).all()) and bool((y[13][~up] == 0).all())
    assert bool(torch.isfinite(y[torch.arange(70, device="cuda") != 13]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("states", ["32", "8"])
def test_example_losses_are_numbers(dtype, states):
    spec = importlib.util.spec_from_file_location("dense_step_example", os.path.join(ROOT, "examples", "dense_step.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses = ex.main(["--steps", "6", "--dtype", dtype, "--states", states, "--vocab", "499", "--tokens", "300"])
    assert len(losses) == 6 and all(math.isfinite(float(v)) for v in losses)
