"""GPU parity of the dense layers (linear, gated block; forward and backward) against the formulas in 64
bits. Tolerances per element, with E = 2^-24 (an fp32 rounding), H the operand type's (2^-8 in bf16, 2^-24
in fp32) and O the output's:
  sums of n products          (n + 4) E sum |a b|, and the operands' own errors through |a| or |b|
  activation a(z)             its argument's error times 1.2 (the largest slope is 1.13), and 16 E (1 + |z|)
                              for its evaluation: up to 8 roundings of terms up to |z|, the exponent's argument
                              off by E |z|, the error function off by 1.5e-7 = 2.5 E
  derivative a'(z)            32 E (the same terms, z times a density below 0.4)
  h, dg, du, dz               one rounding to the operand type (H) on top; each product or sum of two a rounding E
Values below the normal range may be flushed: FLUSH per element, through the products too."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402

E = 2.0 ** -24
FLUSH = 2.0 ** -120
F32, BF16 = torch.float32, torch.bfloat16
ACTS = list(tw.ACTS)


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def half(dtype):
    return torch.finfo(dtype).eps / 2


def act64(z, act):
    """(activation, derivative) in 64 bits."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    if act == "gelu_tanh":
        c = (2 / torch.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return z * (1 + t) / 2, (1 + t) / 2 + z * (1 - t * t) / 2 * c * (1 + 3 * 0.044715 * z * z)
    return z, torch.ones_like(z)


def near(got, want, tol, what, dtype=None):
    """|got - want| <= tol and got's own rounding."""
    assert got.shape == want.shape and (dtype is None or got.dtype == dtype), what
    err = (got.double() - want).abs()
    lim = tol + half(got.dtype) * (want.abs() + tol) + FLUSH
    ok = err <= lim
    assert ok.all(), (what, int((~ok).sum()), float(err.max()), float((err / lim).max()))


def rows(g, T, d, dtype, scale=1.0, stride=0):
    """[T][d], with a row stride where one is given; what lies between the rows is NaN."""
    t = torch.full((T, max(stride, d)), float("nan"), device="cuda", dtype=dtype)
    t[:, :d] = (torch.randn(T, d, generator=g, device="cuda") * scale).to(dtype)
    return t[:, :d]


def weight(g, a, b, fan, dtype):
    return (torch.randn(a, b, generator=g, device="cuda") * fan ** -0.5).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def product(a, b, ea=None, eb=None):
    """(a b^T in 64 bits, its error): a [n][k], b [m][k], ea and eb their elements' errors."""
    k = a.shape[1]
    tol = (k + 4) * E * (a.abs() @ b.abs().t())
    if ea is not None:
        tol = tol + ea @ b.abs().t()
    if eb is not None:
        tol = tol + a.abs() @ eb.t()
    return a @ b.t(), tol


# ------------------------------------------------------------------------------------ linear


def check_linear(x, w, layout, bias, res, act, y, pre):
    w64 = (w if layout == "nk" else w.t()).double()
    z, tz = product(x.double(), w64)
    if bias is not None:
        z = z + bias.double()
        tz = tz + E * (z.abs() + tz)
    if pre is not None:
        near(pre, z, tz, "pre", x.dtype)
    a, _ = act64(z, act)
    tol = 1.2 * tz + (16 * E * (1 + z.abs()) if act not in ("none", "relu") else 0)
    if res is not None:
        a = a + res.double()
        tol = tol + E * (a.abs() + tol)
    near(y, a, tol, "y")


def run_linear(seed, T, K, N, dtype, layout="nk", act="none", bias=True, res=True, y_dtype=None, stride=0):
    say("linear", T, K, N, dtype, layout, act, bias, res, y_dtype, stride)
    g = gen(seed)
    x = rows(g, T, K, dtype, stride=K + stride)
    w = weight(g, *((N, K) if layout == "nk" else (K, N)), K, dtype)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    r = rows(g, T, N, y_dtype or dtype, stride=N + stride) if res else None
    y, pre = tw.linear_fwd(x, w, bias=b, residual=r, act=act, w_layout=layout, y_dtype=y_dtype, want_pre=True)
    assert y.dtype == (y_dtype or dtype)
    check_linear(x, w, layout, b, r, act, y, pre)
    again, none = tw.linear_fwd(x, w, bias=b, residual=r, act=act, w_layout=layout, y_dtype=y_dtype)
    assert none is None and torch.equal(again, y)


def run_linear_back(seed, T, K, N, dtype, layout="nk", act="none", stride=0):
    say("linear back", T, K, N, dtype, layout, act, stride)
    g = gen(seed)
    x, dy = rows(g, T, K, dtype, stride=K + stride), rows(g, T, N, dtype, stride=N + stride)
    w = weight(g, *((N, K) if layout == "nk" else (K, N)), K, dtype)
    pre = rows(g, T, N, dtype, 2.0) if act != "none" else None
    dx, dw, db = tw.linear_bwd(dy, x, w, pre=pre, act=act, w_layout=layout, want_bias=True)
    x64, w64, dz = x.double(), (w if layout == "nk" else w.t()).double(), dy.double()
    tz = torch.zeros_like(dz)
    th = tz
    if act != "none":
        d = act64(pre.double(), act)[1]
        tz = 32 * E * dz.abs()
        dz = dz * d
        tz = tz + E * (dz.abs() + tz)
        th = tz + half(dtype) * (dz.abs() + tz)
    near(dx, *product(dz, w64.t(), th), "dx", dtype)
    want, tol = product(dz.t(), x64.t(), th.t())
    near(dw if layout == "nk" else dw.t(), want, tol, "dw", dtype)
    near(db, dz.sum(0), tz.sum(0) + (T + 4) * E * dz.abs().sum(0), "db", F32)
    # each alone gives the same
    for k, ref in enumerate((dx, dw, db)):
        got = tw.linear_bwd(dy, x, w, pre=pre, act=act, w_layout=layout, want_dx=k == 0, want_dw=k == 1, want_bias=k == 2)
        assert torch.equal(got[k], ref) and sum(t is None for t in got) == 2


# one token to more than a tile; columns and depths that end inside tiles, stages and 16-byte units
SHAPES = [(1, 64, 64), (1, 8, 8), (3, 72, 136), (16, 1032, 2056), (33, 264, 520), (64, 4096, 256), (129, 200, 1000),
          (257, 520, 264), (700, 1544, 776), (1025, 136, 72)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear(shape, layout, dtype):
    run_linear(sum(shape), *shape, dtype, layout, act="silu")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,res,y_dtype", [(False, False, None), (True, False, F32), (False, True, BF16), (True, True, F32)])
def test_linear_epilogues(act, bias, res, y_dtype, dtype):
    run_linear(7, 65, 136, 200, dtype, "nk", act, bias, res, y_dtype, stride=8)
    run_linear(8, 5, 136, 200, dtype, "kn", act, bias, res, y_dtype, stride=16)


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("T,K,N", [(4096, 2048, 2048), (2000, 1024, 8192), (40, 14336, 4096), (1, 4096, 40008), (20, 512, 36000)])
def test_linear_large(T, K, N, layout):
    """Whole rounds of the large tiles; depth split over the CUs; streams of weights for few tokens."""
    run_linear(T, T, K, N, BF16, layout, "gelu", bias=True, res=True)


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("T,K,N", [(65, 1032, 1032), (300, 8192, 1024), (520, 4104, 4104), (1100, 2056, 8200), (2050, 8200, 2056),
                                   (61, 8200, 2056), (64, 4096, 14344)])
def test_linear_between(T, K, N, layout):
    """Every tile, and depths split in numbers of parts that are no powers of two."""
    run_linear(T + 1, T, K, N, BF16, layout, "relu", bias=False, res=True, stride=8)


PLANES = [(2048, 2048, 2048), (1500, 1992, 3000), (2055, 4104, 1032)]


def in_planes(T, K, N, layout):
    """Whether the product splits its fp32 operands, by its workspace: 6 bytes per element of both."""
    return tw.linear_fwd_workspace_bytes(T, K, N, F32, layout) >= 6 * K * (T + N)


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("shape", PLANES)
def test_linear_in_planes(shape, layout):
    assert in_planes(*shape, layout)
    run_linear(sum(shape), *shape, F32, layout, "gelu", stride=8)
    run_linear_back(sum(shape), *shape, F32, layout, "silu", stride=8)


def test_planes_of_one_operand_twice():
    """x and dy one tensor, and one memory read with two strides: every operand keeps its own planes."""
    T, d, f = 2048, 1024, 4096
    g = gen(77)
    both = torch.randn(2 * T, d, generator=g, device="cuda")
    x, dy = both[:T], both[::2]                              # the same address, rows d and 2 d apart
    wg, wu, w2 = (weight(g, f, d, d, F32) for _ in range(3))
    G, U = rows(g, T, f, F32), rows(g, T, f, F32)
    for a, b in ((x, dy), (x, x)):
        got = tw.ffn_gated_dense_bwd(b, a, wg, wu, w2, G, U)
        want = tw.ffn_gated_dense_bwd(b.clone(), a.clone(), wg, wu, w2, G, U)
        for s, t in zip(got[:4], want[:4]):
            assert torch.equal(s, t)


def test_nonfinite_rows_in_planes():
    T, K, N = 2048, 2048, 2048
    g = gen(5)
    x, w = rows(g, T, K, F32), weight(g, N, K, K, F32)
    y = tw.linear_fwd(x, w)[0]
    keep = torch.arange(T, device="cuda") != 13
    for bad in (float("nan"), float("inf")):
        xb = x.clone()
        xb[13, 5] = bad
        yb = tw.linear_fwd(xb, w)[0]
        assert torch.equal(yb[keep], y[keep]) and not torch.isfinite(yb[13]).any()
    big = x.clone()
    big[7] = 0
    big[7, 3] = 3.4e38                                       # near the largest: no infinity from rounding
    want = big[7].double() @ w.double().t()
    fits = want.abs() < 1e38
    got = tw.linear_fwd(big, w)[0][7].double()
    assert ((got - want).abs()[fits] <= 64 * E * want.abs()[fits] + 1e-30).all() and fits.any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_back(shape, layout, dtype):
    run_linear_back(sum(shape), *shape, dtype, layout, act="gelu")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_linear_back_activations(act, layout, dtype):
    run_linear_back(9, 70, 136, 200, dtype, layout, act, stride=8)


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("T,K,N", [(4093, 2048, 2048), (20000, 72, 64), (300, 4096, 8192)])
def test_linear_back_large(T, K, N, layout):
    run_linear_back(T, T, K, N, BF16, layout, "silu")


# ------------------------------------------------------------------------------------- gated


def run_gated(seed, T, d, f, dtype, act="silu", bias=True, res=True, y_dtype=None, stride=0):
    say("gated", T, d, f, dtype, act, bias, res, y_dtype, stride)
    g = gen(seed)
    x = rows(g, T, d, dtype, stride=d + stride)
    wg, wu, w2 = weight(g, f, d, d, dtype), weight(g, f, d, d, dtype), weight(g, f, d, f, dtype)
    bg, bu = (torch.randn(f, generator=g, device="cuda") for _ in range(2)) if bias else (None, None)
    r = rows(g, T, d, y_dtype or dtype, stride=d + stride) if res else None
    kw = dict(bg=bg, bu=bu, residual=r, act=act, y_dtype=y_dtype)
    y, gs, us = tw.ffn_gated_dense_fwd(x, wg, wu, w2, want_saved=True, **kw)
    y2, n1, n2 = tw.ffn_gated_dense_fwd(x, wg, wu, w2, **kw)
    assert n1 is None and n2 is None and torch.equal(y, y2) and y.dtype == (y_dtype or dtype)
    x64 = x.double()
    (G, tg), (U, tu) = product(x64, wg.double()), product(x64, wu.double())
    if bias:
        G, U = G + bg.double(), U + bu.double()
        tg, tu = tg + E * (G.abs() + tg), tu + E * (U.abs() + tu)
    near(gs, G, tg, "g", dtype)
    near(us, U, tu, "u", dtype)
    a, _ = act64(G, act)
    ta = 1.2 * tg + 16 * E * (1 + G.abs())
    h = a * U
    th = ta * (U.abs() + tu) + a.abs() * tu
    th = th + (E + half(dtype)) * (h.abs() + th)
    want, tol = product(h, w2.double().t(), th)
    if res:
        want = want + r.double()
        tol = tol + E * (want.abs() + tol)
    near(y, want, tol, "y")
    return y


def run_gated_back(seed, T, d, f, dtype, act="silu", stride=0):
    say("gated back", T, d, f, dtype, act, stride)
    g = gen(seed)
    x, dy = rows(g, T, d, dtype, stride=d + stride), rows(g, T, d, dtype, stride=d + stride)
    wg, wu, w2 = weight(g, f, d, d, dtype), weight(g, f, d, d, dtype), weight(g, f, d, f, dtype)
    G, U = rows(g, T, f, dtype, 2.0), rows(g, T, f, dtype)
    got = tw.ffn_gated_dense_bwd(dy, x, wg, wu, w2, G, U, act=act, want_bias=True)
    dx, dwg, dwu, dw2, dbg, dbu = got
    x64, dy64, G64, U64 = x.double(), dy.double(), G.double(), U.double()
    a, da = act64(G64, act)
    ea = 16 * E * (1 + G64.abs())
    dh, tdh = product(dy64, w2.double())
    dg, du, h = dh * U64 * da, dh * a, a * U64
    tdg = U64.abs() * (1.2 * tdh + 32 * E * (dh.abs() + tdh))
    tdg = tdg + 2 * E * (dg.abs() + tdg)
    tdu = tdh * (a.abs() + ea) + dh.abs() * ea
    tdu = tdu + E * (du.abs() + tdu)
    H = half(dtype)
    rdg, rdu = tdg + H * (dg.abs() + tdg), tdu + H * (du.abs() + tdu)
    th = ea * U64.abs()
    th = th + (E + H) * (h.abs() + th)
    (p, tp), (q, tq) = product(dg, wg.double().t(), rdg), product(du, wu.double().t(), rdu)
    near(dx, p + q, tp + tq + (f + 4) * E * (dg.abs() @ wg.double().abs() + du.abs() @ wu.double().abs()), "dx", dtype)
    near(dwg, *product(dg.t(), x64.t(), rdg.t()), "dwg", dtype)
    near(dwu, *product(du.t(), x64.t(), rdu.t()), "dwu", dtype)
    near(dw2, *product(h.t(), dy64.t(), th.t()), "dw2", dtype)
    near(dbg, dg.sum(0), tdg.sum(0) + (T + 4) * E * dg.abs().sum(0), "dbg", F32)
    near(dbu, du.sum(0), tdu.sum(0) + (T + 4) * E * du.abs().sum(0), "dbu", F32)
    for t, u in zip(tw.ffn_gated_dense_bwd(dy, x, wg, wu, w2, G, U, act=act)[:4], got):
        assert torch.equal(t, u)


GATED = [(1, 8, 8), (1, 64, 4104), (2, 72, 136), (17, 1032, 520), (64, 520, 2056), (130, 264, 72), (300, 136, 1000),
         (1000, 776, 264)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", GATED)
def test_gated(shape, dtype):
    run_gated(sum(shape), *shape, dtype)


def test_gated_in_planes():
    run_gated(3, 2000, 1024, 4096, F32, stride=8)
    run_gated_back(3, 2000, 1024, 4096, F32, stride=8)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,res,y_dtype", [(False, False, None), (True, True, F32), (True, False, BF16)])
def test_gated_epilogues(act, bias, res, y_dtype, dtype):
    run_gated(5, 67, 136, 200, dtype, act, bias, res, y_dtype, stride=8)


@pytest.mark.parametrize("T,d,f", [(1, 4096, 14336), (64, 2048, 8192), (2048, 1024, 4096)])
def test_gated_large(T, d, f):
    run_gated(T, T, d, f, BF16, bias=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", GATED)
def test_gated_back(shape, dtype):
    run_gated_back(sum(shape), *shape, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ACTS)
def test_gated_back_activations(act, dtype):
    run_gated_back(6, 67, 136, 200, dtype, act, stride=8)


@pytest.mark.parametrize("T,d,f", [(64, 2048, 8192), (2050, 1024, 4096), (9000, 64, 264)])
def test_gated_back_large(T, d, f):
    run_gated_back(T, T, d, f, BF16, "gelu_tanh")


# ------------------------------------------------------------------------------ around them


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(act):
    """fp32 gradients of a small block along one direction, against central differences of the forward in
    fp32: a step of 2^-6 leaves the third derivative (below 10 |direction|^3 s^2 / 6) and, over 2 s, the two
    losses' roundings (64 E each of sums of |dy y|, counted as 2^10 E); relu is not differentiable, so
    inputs keep away from its edge by the step."""
    T, d, f, s = 6, 16, 24, 2.0 ** -6
    g = gen(31)
    x, dy = rows(g, T, d, F32), rows(g, T, d, F32)
    wg, wu, w2 = weight(g, f, d, d, F32), weight(g, f, d, d, F32), weight(g, f, d, f, F32)
    v = rows(g, T, d, F32)
    v = v / v.norm()
    if act == "relu":
        z = x.double() @ wg.double().t()
        dz = v.double() @ wg.double().t()
        if bool((z.abs() <= 1.01 * s * dz.abs()).any()):
            v = v / 64
    _, gs, us = tw.ffn_gated_dense_fwd(x, wg, wu, w2, act=act, want_saved=True)
    dx = tw.ffn_gated_dense_bwd(dy, x, wg, wu, w2, gs, us, act=act)[0]
    up, down = (tw.ffn_gated_dense_fwd(x + k * s * v, wg, wu, w2, act=act)[0].double() for k in (1, -1))
    slope = float(((up - down) * dy.double()).sum() / (2 * s))
    along = float((dx.double() * v.double()).sum())
    size = float((up.abs() * dy.double().abs()).sum())
    third = 10 * float(dy.double().abs().sum()) * float(v.norm()) ** 3 * s * s / 6
    assert abs(slope - along) <= 2 * 2 ** 10 * E * size / (2 * s) + third, (slope, along)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_values(dtype):
    """Arguments at which exponentials overflow or vanish: no NaN, and the limits."""
    z = torch.tensor([-3e38, -1e20, -1000, -90, -40, -20, 0.0, -0.0, 20, 40, 90, 1000, 1e20, 3e38], device="cuda")
    z = torch.cat([z, z.new_zeros(2)])
    x = torch.zeros(1, 8, device="cuda", dtype=dtype)
    w = torch.zeros(16, 8, device="cuda", dtype=dtype)
    for act in ACTS:
        y, _ = tw.linear_fwd(x, w, bias=z, act=act, y_dtype=F32)
        assert torch.isfinite(y).all()
        near(y, act64(z.double(), act)[0][None], 16 * E * (1 + z.double().abs().clamp(max=100)) + E * z.double().clamp(min=0), act)
        pre = z[None].to(dtype)
        dy = torch.ones(1, 16, device="cuda", dtype=dtype)
        db = tw.linear_bwd(dy, x, w, pre=pre, act=act, want_bias=True)[2]
        limit = act64(pre.double().clamp(-50, 50), act)[1][0]
        assert torch.isfinite(db).all() and ((db.double() - limit).abs() <= 64 * E).all(), act


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_rows_stay_rows(bad, dtype):
    g = gen(4)
    T, d, f = 70, 136, 200
    x, dy = rows(g, T, d, dtype), rows(g, T, d, dtype)
    wg, wu, w2 = weight(g, f, d, d, dtype), weight(g, f, d, d, dtype), weight(g, f, d, f, dtype)
    y, gs, us = tw.ffn_gated_dense_fwd(x, wg, wu, w2, want_saved=True)
    dx = tw.ffn_gated_dense_bwd(dy, x, wg, wu, w2, gs, us)[0]
    keep = torch.arange(T, device="cuda") != 13
    xb, gb = x.clone(), gs.clone()
    xb[13, 5] = bad
    gb[13, 7] = bad
    yb = tw.ffn_gated_dense_fwd(xb, wg, wu, w2)[0]
    assert torch.equal(yb[keep], y[keep]) and not torch.isfinite(yb[13]).all()
    db = tw.ffn_gated_dense_bwd(dy, x, wg, wu, w2, gb, us)[0]
    assert torch.equal(db[keep], dx[keep]) and not torch.isfinite(db[13]).all()
    yl = tw.linear_fwd(xb, wg, act="relu")[0]
    assert torch.equal(yl[keep], tw.linear_fwd(x, wg, act="relu")[0][keep])
    assert not torch.isfinite(yl[13]).all() if bad != bad else True


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_tokens(dtype):
    w, wk = torch.ones(24, 16, device="cuda", dtype=dtype), torch.ones(16, 24, device="cuda", dtype=dtype)
    x, dy = torch.ones(0, 16, device="cuda", dtype=dtype), torch.ones(0, 24, device="cuda", dtype=dtype)
    y, pre = tw.linear_fwd(x, w, act="gelu", want_pre=True)
    assert y.shape == pre.shape == (0, 24)
    for lay, t in (("nk", w), ("kn", wk)):
        dx, dw, db = tw.linear_bwd(dy, x, t, pre=dy, act="gelu", w_layout=lay, want_bias=True)
        assert dx.shape == (0, 16) and not dw.any() and not db.any()
    y, g, u = tw.ffn_gated_dense_fwd(x, w, w, w, want_saved=True)
    assert y.shape == (0, 16) and g.shape == (0, 24)
    for t in tw.ffn_gated_dense_bwd(x, x, w, w, w, g, u, want_bias=True)[1:]:
        assert not t.any()


def test_outputs_stay_in_place():
    """Guard zones around outputs and workspace, of ragged sizes, keep their bytes."""
    T, d, f, dt = 67, 136, 200, BF16
    g = gen(12)
    x, w = rows(g, T, d, dt), weight(g, f, d, d, dt)
    L, stream = tw.lib(), torch.cuda.current_stream().cuda_stream
    need = L.ffn_gated_dense_bwd_workspace_bytes(T, d, f, 1, 1)
    sizes = dict(dx=T * d * 2, dwg=f * d * 2, dwu=f * d * 2, dw2=f * d * 2, dbg=f * 4, dbu=f * 4, ws=need)
    bufs = {k: torch.full((n + 2048,), 0xA5, dtype=torch.uint8, device="cuda") for k, n in sizes.items()}
    at = {k: b.data_ptr() + 1024 for k, b in bufs.items()}
    G, U = rows(g, T, f, dt), rows(g, T, f, dt)
    assert L.ffn_gated_dense_bwd(x.data_ptr(), d, x.data_ptr(), d, w.data_ptr(), w.data_ptr(), w.data_ptr(), G.data_ptr(),
                                 U.data_ptr(), 1, T, d, f, 2, *(at[k] for k in ("dx", "dwg", "dwu", "dw2", "dbg", "dbu", "ws")),
                                 need, stream) == 0
    ref = tw.ffn_gated_dense_bwd(x, x, w, w, w, G, U, want_bias=True)
    for (k, n), r in zip(sizes.items(), ref + (None,)):
        b = bufs[k]
        assert (b[:1024] == 0xA5).all() and (b[1024 + n:] == 0xA5).all(), k
        if r is not None:
            assert torch.equal(b[1024:1024 + n], r.contiguous().view(-1).view(torch.uint8)), k


def test_two_streams_and_workspaces():
    """Calls in flight at once on two streams, each with its own workspace."""
    g = gen(2)
    T, d, f = 40, 1024, 2048
    x, w = [rows(g, T, d, BF16) for _ in range(2)], weight(g, f, d, d, BF16)
    want = [tw.ffn_gated_dense_fwd(t, w, w, w)[0] for t in x]
    need = tw.ffn_gated_dense_fwd_workspace_bytes(T, d, f)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k] = tw.ffn_gated_dense_fwd(x[k], w, w, w, workspace=ws[k])[0]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [1, 24, 600])
def test_captured(T):
    """Forward and backward in a HIP graph, replayed on new inputs with eager work between the replays."""
    g = gen(T)
    d, f = 264, 1032
    x, dy = rows(g, T, d, BF16), rows(g, T, d, BF16)
    wg, wu, w2 = weight(g, f, d, d, BF16), weight(g, f, d, d, BF16), weight(g, f, d, f, BF16)

    def step():
        y, gs, us = tw.ffn_gated_dense_fwd(x, wg, wu, w2, residual=x, want_saved=True)
        z, pre = tw.linear_fwd(y, wg, act="gelu", want_pre=True)
        return (y, z) + tw.ffn_gated_dense_bwd(dy, x, wg, wu, w2, gs, us, want_bias=True) + tw.linear_bwd(
            z, y, wg, pre=pre, act="gelu", want_bias=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(rows(g, T, d, BF16))
        dy.copy_(rows(g, T, d, BF16))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), k


def test_python_refusals_on_gpu():
    x, w = torch.zeros(4, 64, device="cuda"), torch.zeros(128, 64, device="cuda")
    b16 = torch.bfloat16
    for kw, err in ((dict(residual=torch.zeros(4, 128, device="cuda", dtype=b16)), TypeError),
                    (dict(residual=torch.zeros(3, 128, device="cuda")), ValueError), (dict(residual=torch.zeros(4, 128)), ValueError),
                    (dict(bias=torch.zeros(64, device="cuda")), ValueError), (dict(bias=torch.zeros(128)), ValueError),
                    (dict(bias=torch.zeros(128, device="cuda", dtype=b16)), TypeError),
                    (dict(workspace=torch.zeros(64, dtype=torch.uint8)), ValueError), (dict(y_dtype=torch.float16), TypeError)):
        with pytest.raises(err):
            tw.linear_fwd(x, w, **kw)
    with pytest.raises(TypeError):
        tw.linear_fwd(x, w.to(b16))
    with pytest.raises(TypeError):
        tw.linear_fwd(x.half(), w.half())
    with pytest.raises(ValueError):
        tw.linear_fwd(x, torch.zeros(64, 128, device="cuda").t())
    with pytest.raises(tw.TwellError):
        tw.linear_fwd(x[:, :60].contiguous(), w[:, :60].contiguous())
    with pytest.raises(tw.TwellError):
        tw.linear_bwd(x, x, w[:64], act="relu")          # no pre
    g = torch.zeros(4, 128, device="cuda")
    with pytest.raises(ValueError):
        tw.ffn_gated_dense_bwd(x, x, w, w, w, g[:3], g)
    with pytest.raises(ValueError):
        tw.ffn_gated_dense_fwd(x, w, w[:64], w)
    with pytest.raises(tw.TwellError):
        tw.ffn_gated_dense_fwd(x, w, w, w, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------------ beyond 2^31 elements


@pytest.fixture
def much_memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of free GPU memory")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("K,N", [(4104, 64), (64, 4104)])
def test_far_rows(K, N, layout, much_memory):
    """x or y of 530003 x 4104: the first, middle and last rows, and the weights' gradient in 64 bits over parts."""
    T, dtype = 530003, BF16
    say("linear far", T, K, N, layout)
    g = gen(K)
    x, dy = (torch.empty(T, n, dtype=dtype, device="cuda") for n in (K, N))
    pre = torch.empty(T, N, dtype=dtype, device="cuda")
    for at in range(0, T, 1 << 16):
        for t in (x, dy, pre):
            p = t[at:at + (1 << 16)]
            p.copy_(torch.randn(p.shape, generator=g, device="cuda"))
    w = weight(g, *((N, K) if layout == "nk" else (K, N)), K, dtype)
    y, z = tw.linear_fwd(x, w, residual=dy, act="silu", w_layout=layout, want_pre=True)
    dx, dw, db = tw.linear_bwd(dy, x, w, pre=pre, act="silu", w_layout=layout, want_bias=True)
    for at in (0, (1 << 31) // 4104 - 3, T // 2, T - 9):
        sel = slice(at, at + 9)
        check_linear(x[sel], w, layout, None, dy[sel], "silu", y[sel], z[sel])
        d = act64(pre[sel].double(), "silu")[1]
        dz = dy[sel].double() * d
        th = 32 * E * dy[sel].double().abs() + (2 * E + half(dtype)) * dz.abs()
        near(dx[sel], *product(dz, (w if layout == "nk" else w.t()).double().t(), th), "dx", dtype)
    ref, tol, one, sums = 0, 0, 0, 0
    for at in range(0, T, 1 << 16):
        sel = slice(at, at + (1 << 16))
        dz = dy[sel].double() * act64(pre[sel].double(), "silu")[1]
        e = 32 * E * dy[sel].double().abs() + 2 * E * dz.abs()
        x64 = x[sel].double()
        ref, tol = ref + dz.t() @ x64, tol + (e + half(dtype) * dz.abs() + (T + 4) * E * dz.abs()).t() @ x64.abs()
        one, sums = one + dz.sum(0), sums + (e + (T + 4) * E * dz.abs()).sum(0)
    near(dw if layout == "nk" else dw.t(), ref, tol, "dw", dtype)
    near(db, one, sums, "db", F32)
