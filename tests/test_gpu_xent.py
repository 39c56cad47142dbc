"""GPU parity of the large-vocabulary cross entropy (loss, lse, dx, dw) against the formulas in 64
bits. Tolerances per element, with E = 2^-24 (an fp32 rounding) and H = 2^-8 (a bf16 one):
  z     d + 4 roundings of a sum of d products: tz = (d + 4) E sum |x w|
  p     its exponent is off by tz, the row's maximum and lse likewise; 256 E for the exponentials,
        the sum over the vocabulary and the logarithm: rp = 3 tz + 256 E + 4 E (|z| + |lse|)
  G     bf16: two roundings off the target, one on it, so 2 H; fp32: none
        and up to 2 FLUSH of underflow: these roundings are relative in fp32's normal range only,
        an exponential or a G below 2^-126 may be flushed to zero
  dx    sum_j |w_j| |dG_j| + V E sum_j |G_j w_j| + the output's rounding; dw likewise over T."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402

E, H = 2.0 ** -24, 2.0 ** -8
FLUSH = 2.0 ** -126
F32, BF16 = torch.float32, torch.bfloat16


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def problem(seed, T, d, V, dtype, ignored=0, stride=0, lean=12.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(generator=g, device="cuda")
    w = (torch.randn(V, d, **kw) * d ** -0.5).to(dtype)
    y = torch.randint(0, V, (T,), **kw)
    x = torch.randn(T, max(stride, d), **kw)
    x[:, :d] += lean * torch.rand(T, 1, **kw) * w[y].float()
    x = x.to(dtype)[:, :d]
    y[torch.randperm(T, **kw)[:ignored]] = -100
    dloss = torch.rand(T, **kw) + 0.5
    return x, w, y, dloss


def check(x, w, y, dloss, got, rows=None):
    """Compares (loss, lse[, dx, dw]) with 64 bits; tokens with a negative target are zero."""
    T, d = x.shape
    V = w.shape[0]
    act = y >= 0
    loss, lse = got[0].double(), got[1].double()
    assert not loss[~act].any() and not lse[~act].any()
    xs, ws, ys = x[act].double(), w.double(), y[act]
    z = xs @ ws.t()
    tz = (d + 4) * E * (xs.abs() @ ws.abs().t()).amax(1, keepdim=True)
    ref = torch.logsumexp(z, 1, keepdim=True)
    zt = z.gather(1, ys[:, None])
    rp = 3 * tz + 256 * E + 4 * E * (z.abs().amax(1, keepdim=True) + ref.abs())
    assert ((lse[act][:, None] - ref).abs() <= rp).all()
    assert ((loss[act][:, None] - (ref - zt)).abs() <= rp + tz).all()
    if len(got) == 2:
        return
    dx, dw = got[2], got[3]
    bf = x.dtype == BF16
    out = H if bf else E
    dl = dloss[act].double()[:, None]
    p = torch.exp(z - ref)
    G = p * dl
    G.scatter_(1, ys[:, None], torch.expm1(zt - ref) * dl)
    tg = G.abs() * (2 * H if bf else 8 * E) + p * dl.abs() * rp + FLUSH * (1 + dl.abs())
    for name, a, ref, tol in (("dx", dx[act], G @ ws, tg @ ws.abs() + V * E * (G.abs() @ ws.abs())),
                              ("dw", dw, G.t() @ xs, tg.t() @ xs.abs() + (T + 8) * E * (G.abs().t() @ xs.abs()))):
        tol = tol + out * (ref.abs() + tol) + FLUSH
        bad = (a.double() - ref).abs() > tol
        assert not bad.any(), (name, int(bad.sum()), float(((a.double() - ref).abs() - tol).max()))
    assert not dx[~act].any()


SHAPES = [(1, 8, 1), (1, 64, 1000), (1, 4096, 777), (3, 72, 50), (64, 128, 2048), (65, 128, 2049), (130, 200, 257),
          (256, 64, 512), (300, 520, 1999), (777, 264, 3001)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d,V", SHAPES)
def test_forward(T, d, V, dtype):
    say("xent fwd", T, d, V, dtype)
    x, w, y, dl = problem(T + d + V, T, d, V, dtype, ignored=T // 5, stride=d + 8)
    check(x, w, y, dl, tw.linear_xent_fwd(x, w, y))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d,V", SHAPES)
def test_gradients(T, d, V, dtype):
    say("xent grad", T, d, V, dtype)
    x, w, y, dl = problem(T + d + V, T, d, V, dtype, ignored=T // 3, stride=d + 16)
    got = tw.linear_xent_fwd_bwd(x, w, y, dl)
    check(x, w, y, dl, got)
    fwd = tw.linear_xent_fwd(x, w, y)
    assert torch.equal(fwd[0], got[0]) and torch.equal(fwd[1], got[1])
    for a, b in zip(got, tw.linear_xent_fwd_bwd(x, w, y, dl)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_integer_grid_is_exact(dtype):
    """Small integers: the logits are exact, so equal rows of w give equal probabilities: with
    all of w alike, loss = log V and G = (1 / V - onehot) dloss."""
    T, d, V = 70, 64, 512
    x = torch.randint(-3, 4, (T, d), device="cuda").to(dtype)
    w = torch.randint(-3, 4, (1, d), device="cuda").to(dtype).repeat(V, 1)
    y = torch.arange(T, device="cuda") * 7 % V
    dl = torch.ones(T, device="cuda")
    loss, lse, dx, dw = tw.linear_xent_fwd_bwd(x, w, y, dl)
    z = x.double() @ w[0].double()
    ref = torch.tensor(float(V)).double().log()
    assert ((loss.double() - ref).abs() <= 4 * E * (ref + z.abs() + 1)).all()
    check(x, w, y, dl, (loss, lse, dx, dw))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [40, 300])
def test_left_out_tokens_reach_nothing(T, dtype):
    x, w, y, dl = problem(9, T, 128, 700, dtype)
    y[::3] = -1
    y[1] = -(1 << 40)
    clean = tw.linear_xent_fwd_bwd(x, w, y, dl)
    x2, dl2 = x.clone(), dl.clone()
    x2[::3] = float("nan")
    x2[1] = float("inf")
    dl2[::3] = float("nan")
    dirty = tw.linear_xent_fwd_bwd(x2, w, y, dl2)
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b)
    check(x, w, y, dl, clean)
    for a, b in zip(tw.linear_xent_fwd(x2, w, y), clean):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 64, 333])
def test_all_tokens_left_out(T, dtype):
    x, w, y, dl = problem(2, T, 64, 300, dtype)
    y.fill_(-100)
    x.fill_(float("nan"))
    for t in tw.linear_xent_fwd_bwd(x, w, y, dl) + tw.linear_xent_fwd(x, w, y):
        assert not t.any()                              # NaN counts as nonzero


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_target_beyond_vocabulary(dtype):
    x, w, y, dl = problem(3, 50, 64, 300, dtype)
    y[7], y[8] = 300, 1 << 40
    loss, lse, dx, dw = tw.linear_xent_fwd_bwd(x, w, y, dl)
    rest = torch.ones(50, dtype=torch.bool, device="cuda")
    rest[7:9] = False
    assert torch.isnan(loss[7:9]).all() and torch.isfinite(loss[rest]).all() and torch.isfinite(lse).all()
    assert torch.isnan(dx[7:9].float()).all() and torch.isfinite(dx[rest].float()).all()
    assert torch.isnan(dw.float()).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [5, 100])
def test_nonfinite_token_stays_in_its_row(T, dtype):
    """A NaN or an infinity in a token that counts: its loss is NaN, other losses and rows of dx are
    untouched, dw shows it."""
    x, w, y, dl = problem(4, T, 64, 300, dtype)
    clean = tw.linear_xent_fwd_bwd(x, w, y, dl)
    x = x.clone()
    x[2, 5], x[4, 0] = float("nan"), float("inf")
    got = tw.linear_xent_fwd_bwd(x, w, y, dl)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[2] = rest[4] = False
    assert torch.isnan(got[0][2]) and torch.isnan(got[0][4])
    for k in range(3):
        assert torch.equal(got[k][rest], clean[k][rest])
    assert torch.isnan(got[3].float()).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_logits_and_sure_tokens(dtype):
    """Logits of thousands (exponentials far outside fp32's range) and tokens whose probability
    is one up to rounding: no overflow, and p - 1 keeps its digits."""
    x, w, y, dl = problem(5, 90, 64, 400, dtype, lean=0.0)
    x = (x.float() * 512).to(dtype)
    check(x, w, y, dl, tw.linear_xent_fwd_bwd(x, w, y, dl))
    x, w, y, dl = problem(6, 90, 64, 400, dtype, lean=40.0)
    check(x, w, y, dl, tw.linear_xent_fwd_bwd(x, w, y, dl))


@pytest.mark.parametrize("T,d,V,dtype,ignored", [(1000, 64, 128000, F32, 300), (4200, 64, 128000, BF16, 100),
                                                 (4200, 64, 128000, BF16, 1500)])
def test_pieces(T, d, V, dtype, ignored):
    """More tokens than one piece holds (768 fp32 or 3840 bf16 rows at this vocabulary); the last
    case leaves the second piece empty."""
    say("xent pieces", T, d, V, dtype, ignored)
    x, w, y, dl = problem(7, T, d, V, dtype, ignored=ignored)
    check(x, w, y, dl, tw.linear_xent_fwd_bwd(x, w, y, dl))


def test_against_differences():
    """dx and dw against central differences of the 64-bit loss (h = 1e-5: truncation and
    cancellation below 1e-8 of the values)."""
    T, d, V, h = 3, 16, 37, 1e-5
    x, w, y, dl = problem(8, T, d, V, F32)
    _, _, dx, dw = tw.linear_xent_fwd_bwd(x, w, y, dl)

    def f(x_, w_):
        z = x_ @ w_.t()
        return float(((torch.logsumexp(z, 1) - z.gather(1, y[:, None])[:, 0]) * dl.double()).sum())
    x64, w64 = x.double(), w.double()
    for k, (base, got) in enumerate(((x64, dx), (w64, dw))):
        # fp32: the sums' (V + d) E and the exponentials' 256 E of the largest term
        tol = 1024 * E * float(dl.max()) * (1 + float(x64.abs().max() + w64.abs().max()))
        for i in range(0, base.numel(), 5):
            up, dn = base.clone().reshape(-1), base.clone().reshape(-1)
            up[i] += h
            dn[i] -= h
            up, dn = up.reshape(base.shape), dn.reshape(base.shape)
            diff = (f(up, w64) - f(dn, w64) if k == 0 else f(x64, up) - f(x64, dn)) / (2 * h)
            assert abs(float(got.reshape(-1)[i]) - diff) <= tol + 1e-8, (k, i)


def test_empty():
    w = torch.ones(10, 64).cuda()
    x, y, dl = torch.empty(0, 64).cuda(), torch.empty(0, dtype=torch.int64).cuda(), torch.empty(0).cuda()
    assert tw.linear_xent_fwd(x, w, y)[0].shape == (0,)
    loss, lse, dx, dw = tw.linear_xent_fwd_bwd(x, w, y, dl)
    assert dx.shape == (0, 64) and not dw.any()


def test_python_refusals():
    x, w, y, dl = problem(1, 4, 64, 100, BF16)
    with pytest.raises(TypeError):
        tw.linear_xent_fwd(x, w.float(), y)
    with pytest.raises(TypeError):
        tw.linear_xent_fwd(x, w, y.int())
    with pytest.raises(TypeError):
        tw.linear_xent_fwd_bwd(x, w, y, dl.double())
    with pytest.raises(ValueError):
        tw.linear_xent_fwd(x, w[:, :32].contiguous(), y)
    with pytest.raises(ValueError):
        tw.linear_xent_fwd(x, w, y[:3])
    with pytest.raises(ValueError):
        tw.linear_xent_fwd(x, w.t().contiguous().t(), y)
    with pytest.raises(tw.TwellError):
        tw.linear_xent_fwd(x, w, y, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(tw.TwellError):
        tw.linear_xent_fwd(x[:, :60], w[:, :60].contiguous(), y)


@pytest.mark.parametrize("T", [16, 300])
def test_graph_and_side_stream(T):
    x, w, y, dl = problem(10, T, 128, 1000, BF16, ignored=5)
    x = x.contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = tw.linear_xent_fwd_bwd(x, w, y, dl)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(on_side, tw.linear_xent_fwd_bwd(x, w, y, dl)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tw.linear_xent_fwd_bwd(x, w, y, dl)
    for k in range(4):
        x2, _, y2, dl2 = problem(20 + k, T, 128, 1000, BF16, ignored=3 * k)
        x.copy_(x2)
        y.copy_(y2)
        dl.copy_(dl2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, tw.linear_xent_fwd_bwd(x, w, y, dl)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d,V", [(2049, 328, 2500), (600, 264, 9001), (1030, 520, 20011), (90, 1032, 6007),
                                   (70, 72, 30001)])
def test_tile_sizes(T, d, V, dtype):
    """Calls that take each of the tiles of the three products, ragged in every direction, with the
    tokens' list counted by its own launch (T > 2048) or not, and dx whole or split."""
    say("xent tiles", T, d, V, dtype)
    x, w, y, dl = problem(T + d, T, d, V, dtype, ignored=T // 7)
    got = tw.linear_xent_fwd_bwd(x, w, y, dl)
    check(x, w, y, dl, got)
    fwd = tw.linear_xent_fwd(x, w, y)
    check(x, w, y, dl, fwd)
    for a, b in zip(got, tw.linear_xent_fwd_bwd(x, w, y, dl)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 2, 40, 64, 65, 300, 512, 513])
@pytest.mark.parametrize("stride", [0, 264, 1 << 20, (1 << 20) + 8])
def test_few_tokens_in_place(T, stride):
    """The forward of few bf16 tokens reads x's rows where they lie, however far apart, and skips those
    without a target (NaN in them reaches nothing)."""
    d, V = 256, 3001
    x, w, y, dl = problem(T + 5, T, d, V, BF16, ignored=T // 2)
    big = torch.empty((T - 1) * max(stride, d) + d, dtype=BF16, device="cuda")
    far = big.as_strided((T, d), (max(stride, d), 1))
    far.copy_(x)
    far[y < 0] = float("nan")
    got = tw.linear_xent_fwd(far, w, y)
    check(x, w, y, dl, got)
    if T > 1:
        y[1] = V + 3
        loss, lse = tw.linear_xent_fwd(far, w, y)
        assert torch.isnan(loss[1])
        keep = torch.arange(T, device="cuda") != 1
        assert torch.equal(loss[keep], got[0][keep]) and torch.equal(lse[keep], got[1][keep])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d,V", [(60, 64, 20011), (300, 72, 2500), (2100, 64, 9000)])
def test_logits_far_from_zero(T, d, V, dtype):
    """Tokens whose logits lie around -100 .. 100: exponentials without a reference, with one in some or
    all blocks of a row, and rows beyond the range in which a factor per token can stand for one."""
    say("xent shifted", T, d, V, dtype)
    x, w, y, dl = problem(T + V, T, d, V, dtype, ignored=T // 9)
    w[:, 0] = 1
    shift = torch.tensor([0.0, -8, -15, -30, -100, 8, 20, 55, 70, 100, -60, 12], device="cuda")
    x[:, 0] = shift[torch.arange(T, device="cuda") % 12].to(dtype)
    got = tw.linear_xent_fwd_bwd(x, w, y, dl)
    check(x, w, y, dl, got)
    for a, b in zip(got, tw.linear_xent_fwd_bwd(x, w, y, dl)):
        assert torch.equal(a, b)
    fwd = tw.linear_xent_fwd(x, w, y)
    check(x, w, y, dl, fwd)


@pytest.mark.parametrize("T,dtype", [(1500, F32), (2600, F32)])
def test_more_pieces(T, dtype):
    """Two and more pieces of fp32 rows."""
    x, w, y, dl = problem(17, T, 64, 128000, dtype, ignored=T // 3)
    check(x, w, y, dl, tw.linear_xent_fwd_bwd(x, w, y, dl))


@pytest.mark.parametrize("T,d,V,dtype", [(6000, 64, 500, BF16), (6000, 64, 500, F32), (3100, 200, 1009, BF16),
                                         (3100, 200, 1009, F32), (1300, 1032, 2503, F32), (2100, 1544, 4099, F32)])
def test_many_tokens_of_a_small_head(T, d, V, dtype):
    """dw in splits of the tokens; fp32 as it is and in planes."""
    say("xent small head", T, d, V, dtype)
    x, w, y, dl = problem(T + V, T, d, V, dtype, ignored=T // 4)
    got = tw.linear_xent_fwd_bwd(x, w, y, dl)
    check(x, w, y, dl, got)
    for a, b in zip(got, tw.linear_xent_fwd_bwd(x, w, y, dl)):
        assert torch.equal(a, b)
    fwd = tw.linear_xent_fwd(x, w, y)
    check(x, w, y, dl, fwd)


@pytest.mark.parametrize("T,d,V", [(1, 72, 40001), (20, 64, 33000), (32, 136, 36003), (33, 64, 36003)])
def test_few_tokens_of_a_large_vocabulary(T, d, V):
    say("xent few", T, d, V)
    x, w, y, dl = problem(T + V, T, d, V, BF16, ignored=T // 5)
    check(x, w, y, dl, tw.linear_xent_fwd(x, w, y))
    got = tw.linear_xent_fwd_bwd(x, w, y, dl)
    check(x, w, y, dl, got)
    for a, b in zip(got, tw.linear_xent_fwd_bwd(x, w, y, dl)):
        assert torch.equal(a, b)


def test_pieces_in_planes():
    """Two pieces of rows (768 fp32 rows at this vocabulary) of products that run in bf16 planes."""
    T, d, V = 1500, 520, 100003
    say("xent planes, pieces", T, d, V)
    x, w, y, dl = problem(23, T, d, V, F32, ignored=200)
    check(x, w, y, dl, tw.linear_xent_fwd_bwd(x, w, y, dl))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pieces_of_split_tokens(dtype):
    """More than a million tokens of a small head: dw in splits of the tokens and sums over pieces."""
    T, d, V = 1150000, 16, 500
    say("xent many tokens", T, d, V, dtype)
    x, w, y, dl = problem(29, T, d, V, dtype, ignored=1000, lean=4.0)
    dl = dl / T
    got = tw.linear_xent_fwd_bwd(x, w, y, dl)
    rest = torch.randperm(T, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))[:4000]
    act = rest[y[rest] >= 0]
    xs, ws = x[act].double(), w.double()
    z = xs @ ws.t()
    lse = torch.logsumexp(z, 1)
    assert ((got[1][act].double() - lse).abs() <= 1024 * E * (1 + z.abs().amax(1))).all()
    # dw in 64 bits, in parts; its error: 2 H (bf16) or 1024 E of every term, and the output's rounding
    ref = torch.zeros(V, d, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(ref)
    for at in range(0, T, 100000):
        yy = y[at:at + 100000]
        a = yy >= 0
        xx = x[at:at + 100000][a].double()
        p = torch.softmax(xx @ ws.t(), 1)
        p[torch.arange(len(p), device="cuda"), yy[a]] -= 1
        G = p * dl[at:at + 100000][a].double()[:, None]
        ref += G.t() @ xx
        tol += G.abs().t() @ xx.abs()
    tol = tol * ((2 * H if dtype == BF16 else 0) + 1024 * E) + (H if dtype == BF16 else E) * ref.abs()
    assert ((got[3].double() - ref).abs() <= tol).all()
