"""GPU parity of the layer norm (forward with the residual add, backward with the sums over
tokens) against the formulas in 64 bits. Tolerances are written per element from the number of
fp32 roundings on the way to it (E = 2^-24 each; a sum of n terms over a workgroup takes at most
64 on any path: 16 in a thread, 6 in a wave, 16 over waves, and the products) plus the output
type's own rounding."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402

E = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(g, T, d, dtype, stride=0):
    """[T][d] on the GPU, rows `stride` elements apart where that is larger than d."""
    x = torch.randn(T, max(stride, d), generator=g) + 3 * torch.randn(T, 1, generator=g)
    return x.to(dtype).cuda()[:, :d]


def fwd64(s, w, b, eps):
    s = s.double().cpu()
    mu = s.mean(1, keepdim=True)
    v = s - mu
    rs = 1 / ((v * v).mean(1, keepdim=True) + eps).sqrt()
    y = v * rs * w.double().cpu() + (b.double().cpu() if b is not None else 0)
    return mu, rs, v, y


def check_fwd(s, w, b, eps, y, mean, rstd):
    mu, rs, v, ref = fwd64(s, w, b, eps)
    scale = s.double().cpu().abs().mean(1, keepdim=True)
    assert ((mean.double().cpu()[:, None] - mu).abs() <= 64 * E * scale).all()
    # the centring error enters the variance with its square and, weighted by the sum of v
    # (zero up to rounding), not at all; relative to the spread it is 64 E scale rs
    off = 64 * E * scale * rs
    rtol = 64 * E + off * off + 8 * E * scale * rs
    assert ((rstd.double().cpu()[:, None] / rs - 1).abs() <= rtol).all()
    aw = w.double().cpu().abs()
    tol = aw * ((v * rs).abs() * (rtol + 4 * E) + off + 2 * E * scale * rs) + 2 * E * ref.abs()
    if b is not None:
        tol = tol + 2 * E * b.double().cpu().abs()
    tol = tol + HALF[y.dtype] * (ref.abs() + tol)
    bad = (y.double().cpu() - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((y.double().cpu() - ref).abs() - tol).max()))


SIZES = [(1, 8), (1, 4096), (2, 72), (5, 64), (3, 1000), (700, 256), (257, 2048), (9, 4096), (4, 8200), (2, 16384)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("xt,yt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("residual", [False, True])
def test_fwd(T, d, xt, yt, residual):
    say("norm fwd", T, d, xt, yt, residual)
    g = gen(T * 131 + d)
    x = rows(g, T, d, xt, d + 24 if residual else 0)
    r = rows(g, T, d, xt, d + 8) if residual else None
    w, b = torch.randn(d, generator=g).cuda(), torch.randn(d, generator=g).cuda()
    b = b if T % 2 else None
    y, s, mean, rstd = tw.layer_norm_fwd(x, w, b, residual=r, eps=1e-5, y_dtype=yt)
    want = (x.float() + r.float()).to(xt) if residual else x
    assert torch.equal(s, want)
    assert y.dtype == yt and s.dtype == xt
    check_fwd(want, w, b, 1e-5, y, mean, rstd)
    y2 = tw.layer_norm_fwd(x, w, b, residual=r, eps=1e-5, y_dtype=yt, want_stats=False)[0]
    assert torch.equal(y, y2)


def test_fwd_far_and_constant_rows():
    """A row far from zero keeps its variance; a constant row gives the bias."""
    g = gen(5)
    x = torch.randn(4, 512, generator=g)
    x[0] += 4096.0                      # spacing of fp32 there: 2^-11
    x[1] = 7.25
    x[2] = 0.0
    x = x.cuda()
    w, b = torch.randn(512, generator=g).cuda(), torch.randn(512, generator=g).cuda()
    y, _, mean, rstd = tw.layer_norm_fwd(x, w, b, eps=1e-5)
    check_fwd(x[[0, 3]], w, b, 1e-5, y[[0, 3]], mean[[0, 3]], rstd[[0, 3]])
    # sums of 512 equal values of 7.25 are exact in fp32
    assert torch.equal(y[1], b) and torch.equal(y[2], b)
    assert float(mean[1]) == 7.25 and float(mean[2]) == 0.0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_fwd_nonfinite_rows_stay_alone(dtype):
    g = gen(6)
    x = torch.randn(6, 264, generator=g).to(dtype).cuda()
    w, b = torch.ones(264).cuda(), torch.zeros(264).cuda()
    clean = tw.layer_norm_fwd(x, w, b)
    x2 = x.clone()
    x2[1, 3], x2[3, 100], x2[4, 263] = float("nan"), float("inf"), float("-inf")
    y, _, mean, rstd = tw.layer_norm_fwd(x2, w, b)
    for t in (0, 2, 5):
        assert torch.equal(y[t], clean[0][t]) and mean[t] == clean[2][t] and rstd[t] == clean[3][t]
    for t in (1, 3, 4):
        assert torch.isnan(y[t].float()).all()


def bwd64(dy, s, w, mean, rstd, dres):
    dy, s, w = dy.double().cpu(), s.double().cpu(), w.double().cpu()
    mu, rs = mean.double().cpu()[:, None], rstd.double().cpu()[:, None]
    xh = (s - mu) * rs
    g = dy * w
    mg, mx = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rs * (g - mg - xh * mx)
    txh = 4 * E * (s.abs() + mu.abs()) * rs
    tol = rs * (64 * E * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
                + txh * mx.abs() + xh.abs() * (g.abs() * txh).mean(1, keepdim=True))
    if dres is not None:
        r = dres.double().cpu()
        dx = dx + r
        tol = tol + 2 * E * (r.abs() + dx.abs())
    dw, db = (dy * xh).sum(0), dy.sum(0)
    # sums over tokens: at most T / 512 + 16 + 32 additions on a path (below 128 here)
    tdw = (dy.abs() * (128 * E * xh.abs() + txh)).sum(0)
    tdb = 128 * E * dy.abs().sum(0)
    return (dx, tol), (dw, tdw), (db, tdb)


@pytest.mark.parametrize("T,d", SIZES + [(1500, 64), (513, 520)])
@pytest.mark.parametrize("xt,dyt,dxt", [(F32, F32, F32), (BF16, F32, BF16), (BF16, BF16, F32), (F32, BF16, BF16),
                                        (BF16, BF16, BF16)])
def test_bwd(T, d, xt, dyt, dxt):
    say("norm bwd", T, d, xt, dyt, dxt)
    g = gen(T * 17 + d)
    s, dy = rows(g, T, d, xt, d + 8), rows(g, T, d, dyt, d + 16)
    dres = rows(g, T, d, dxt, d + 8) if d % 16 else None
    w = torch.randn(d, generator=g).cuda()
    _, _, mean, rstd = tw.layer_norm_fwd(s, w, eps=1e-5)
    dx, dw, db = tw.layer_norm_bwd(dy, s, w, mean, rstd, dres=dres, dx_dtype=dxt)
    for name, got, (ref, tol) in zip(("dx", "dw", "db"), (dx, dw, db), bwd64(dy, s, w, mean, rstd, dres)):
        tol = tol + HALF[got.dtype] * (ref.abs() + tol)
        bad = (got.double().cpu() - ref).abs() > tol
        assert not bad.any(), (name, int(bad.sum()), float(((got.double().cpu() - ref).abs() - tol).max()))
    again = tw.layer_norm_bwd(dy, s, w, mean, rstd, dres=dres, dx_dtype=dxt, want_bias=False)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and again[2] is None


def test_bwd_against_differences():
    """dx, dw and db against central differences of the 64-bit forward (h = 1e-5: truncation
    and cancellation below 1e-9 of the values, far inside the fp32 bounds)."""
    g = gen(11)
    T, d, h = 3, 64, 1e-5
    s, dy = rows(g, T, d, F32), rows(g, T, d, F32)
    w, b = torch.randn(d, generator=g).cuda(), torch.randn(d, generator=g).cuda()
    _, _, mean, rstd = tw.layer_norm_fwd(s, w, b, eps=1e-5)
    got = tw.layer_norm_bwd(dy, s, w, mean, rstd)
    tols = [t for _, t in bwd64(dy, s, w, mean, rstd, None)]
    c = dy.double().cpu()
    s64, w64, b64 = s.double().cpu(), w.double().cpu(), b.double().cpu()

    def loss(s_, w_, b_):
        return (fwd64(s_, w_, b_, 1e-5)[3] * c).sum()
    # the kernel takes the rounded statistics: mean and rstd off by what the forward may be
    slack = 2e-5
    for k, base in enumerate((s64, w64, b64)):
        flat = base.reshape(-1)
        for i in range(0, flat.numel(), 7):
            up, dn = flat.clone(), flat.clone()
            up[i] += h
            dn[i] -= h
            args_u, args_d = [s64, w64, b64], [s64, w64, b64]
            args_u[k], args_d[k] = up.reshape(base.shape), dn.reshape(base.shape)
            diff = float((loss(*args_u) - loss(*args_d)) / (2 * h))
            val = float(got[k].double().cpu().reshape(-1)[i])
            tol = float(tols[k].reshape(-1)[i]) + slack * float(got[k].double().abs().max())
            assert abs(val - diff) <= tol, (k, i, val, diff)


def test_empty():
    w = torch.ones(64).cuda()
    x = torch.empty(0, 64).cuda()
    y, s, mean, rstd = tw.layer_norm_fwd(x, w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = tw.layer_norm_bwd(x, x, w, mean, rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_python_refusals():
    x, w = torch.zeros(4, 64).cuda(), torch.ones(64).cuda()
    st = torch.zeros(4).cuda()
    with pytest.raises(TypeError):
        tw.layer_norm_fwd(x, w.double())
    with pytest.raises(ValueError):
        tw.layer_norm_fwd(x, w[:32])
    with pytest.raises(TypeError):
        tw.layer_norm_fwd(x, w, residual=x.bfloat16())
    with pytest.raises(TypeError):
        tw.layer_norm_fwd(x.half(), w)
    with pytest.raises(ValueError):
        tw.layer_norm_fwd(torch.zeros(64, 4).cuda().t(), w)
    with pytest.raises(tw.TwellError):
        tw.layer_norm_fwd(torch.zeros(4, 65).cuda()[:, :64], w)       # rows 4 bytes off 16
    with pytest.raises(tw.TwellError):
        tw.layer_norm_fwd(torch.zeros(4, 60).cuda(), torch.ones(60).cuda())
    with pytest.raises(TypeError):
        tw.layer_norm_bwd(x, x, w, st, st, dres=x.bfloat16())
    with pytest.raises(ValueError):
        tw.layer_norm_bwd(x[:2], x, w, st, st)
    with pytest.raises(ValueError):
        tw.layer_norm_bwd(x, x, w, st[:2], st)


def test_graph_and_side_stream():
    """Captured forward and backward, replayed with new inputs and eager work in between."""
    g = gen(21)
    T, d = 600, 512
    x, dy = rows(g, T, d, BF16).contiguous(), rows(g, T, d, F32).contiguous()
    w, b = torch.randn(d, generator=g).cuda(), torch.randn(d, generator=g).cuda()

    def step():
        y, s, mean, rstd = tw.layer_norm_fwd(x, w, b, residual=x)
        return (y, mean, rstd) + tw.layer_norm_bwd(dy, s, w, mean, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, c in zip(on_side, step()):
        assert torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(rows(g, T, d, BF16))
        dy.copy_(rows(g, T, d, F32))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(out, step()):
            assert torch.equal(a, c)
