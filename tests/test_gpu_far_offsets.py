"""Operands of more than 2^31 elements: the cross entropy's head and hidden states, one gradient of the
clipping. The oracles run in 64 bits over parts; tolerances as for small operands."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402
from test_gpu_grad import check_out  # noqa: E402
from test_gpu_xent import BF16, E, F32, FLUSH, H  # noqa: E402


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.fixture(autouse=True)
def much_memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GiB of free GPU memory")
    yield
    torch.cuda.empty_cache()


def fill(shape, dtype, g, scale):
    """Normal values, made in parts."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    n = max(1, (1 << 28) // shape[1])
    for at in range(0, shape[0], n):
        p = t[at:at + n]
        p.copy_(torch.randn(p.shape, generator=g, device="cuda") * scale)
    return t


def tolerances(d, dtype):
    return (2 * H if dtype == BF16 else 8 * E), (H if dtype == BF16 else E)


@pytest.mark.parametrize("T,dtype", [(40, BF16), (700, BF16), (40, F32), (700, F32)])
def test_head(T, dtype):
    """w and dw of 600003 x 4104; fp32 as it is and in planes."""
    d, V, n = 4104, 600003, 1 << 16
    say("xent far head", T, d, V, dtype)
    g = torch.Generator(device="cuda").manual_seed(T)
    w = fill((V, d), dtype, g, d ** -0.5)
    x = torch.randn(T, d, generator=g, device="cuda")
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[::3] = torch.randint(V - 1000, V, (len(y[::3]),), generator=g, device="cuda")     # beyond 2^31 elements
    x = (x + 8 * w[y].float()).to(dtype)
    dl = torch.rand(T, generator=g, device="cuda") + 0.5
    loss, lse, dx, dw = tw.linear_xent_fwd_bwd(x, w, y, dl)
    fwd = tw.linear_xent_fwd(x, w, y)
    assert torch.equal(fwd[0], loss) and torch.equal(fwd[1], lse)
    x64, dl64 = x.double(), dl.double()[:, None]
    z = torch.cat([x64 @ w[at:at + n].double().t() for at in range(0, V, n)], 1)
    tz = (d + 4) * E * torch.stack([(x64.abs() @ w[at:at + n].double().abs().t()).amax(1) for at in range(0, V, n)]).amax(0)
    ref, zt = torch.logsumexp(z, 1, keepdim=True), z.gather(1, y[:, None])
    rp = 3 * tz[:, None] + 256 * E + 4 * E * (z.abs().amax(1, keepdim=True) + ref.abs())
    assert ((lse.double()[:, None] - ref).abs() <= rp).all()
    assert ((loss.double()[:, None] - (ref - zt)).abs() <= rp + tz[:, None]).all()
    each, out = tolerances(d, dtype)
    dx_ref, dx_tol, dx_abs = 0, 0, 0
    for at in range(0, V, n):
        w64 = w[at:at + n].double()
        p = torch.exp(z[:, at:at + n] - ref) * dl64
        G = p.clone()
        here = (y >= at) & (y < at + n)
        G[here, y[here] - at] = (torch.expm1(zt - ref) * dl64)[here, 0]
        tg = G.abs() * each + p * rp + FLUSH * (1 + dl64)
        want, tol = G.t() @ x64, tg.t() @ x64.abs() + (T + 8) * E * (G.abs().t() @ x64.abs())
        assert ((dw[at:at + n].double() - want).abs() <= tol + out * (want.abs() + tol) + FLUSH).all(), at
        dx_ref, dx_tol, dx_abs = dx_ref + G @ w64, dx_tol + tg @ w64.abs(), dx_abs + G.abs() @ w64.abs()
    tol = dx_tol + V * E * dx_abs
    assert ((dx.double() - dx_ref).abs() <= tol + out * (dx_ref.abs() + tol) + FLUSH).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_hidden_states(dtype):
    """x and dx of 1200007 x 2048, a ninth of the tokens without a target."""
    T, d, V, n = 1200007, 2048, 61, 1 << 16
    say("xent far tokens", T, d, V, dtype)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = fill((T, d), dtype, g, 1.0)
    w = fill((V, d), dtype, g, d ** -0.5)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[::9] = -1
    dl = torch.rand(T, generator=g, device="cuda") + 0.5
    loss, lse, dx, dw = tw.linear_xent_fwd_bwd(x, w, y, dl)
    fwd = tw.linear_xent_fwd(x, w, y)       # fp32 as it is, where the gradients' products run in planes
    w64 = w.double()
    each, out = tolerances(d, dtype)
    dw_ref, dw_tol = 0, 0
    for at in range(0, T, n):
        s = slice(at, at + n)
        a, x64, dl64 = y[s] >= 0, x[s].double(), dl[s].double()[:, None]
        yy = y[s].clamp(min=0)[:, None]
        z = x64 @ w64.t()
        tz = (d + 4) * E * (x64.abs() @ w64.abs().t()).amax(1, keepdim=True)
        ref, zt = torch.logsumexp(z, 1, keepdim=True), z.gather(1, yy)
        rp = 3 * tz + 256 * E + 4 * E * (z.abs().amax(1, keepdim=True) + ref.abs())
        for l, e in ((loss[s], lse[s]), (fwd[0][s], fwd[1][s])):
            assert ((e.double()[:, None] - ref).abs() <= rp)[a].all() and not e[~a].any(), at
            assert ((l.double()[:, None] - (ref - zt)).abs() <= rp + tz)[a].all() and not l[~a].any(), at
        p = torch.exp(z - ref) * dl64 * a[:, None]
        G = p.scatter(1, yy, torch.expm1(zt - ref) * dl64) * a[:, None]
        tg = (G.abs() * each + p * rp + FLUSH * (1 + dl64)) * a[:, None]
        want, tol = G @ w64, tg @ w64.abs() + V * E * (G.abs() @ w64.abs())
        assert ((dx[s].double() - want).abs() <= tol + out * (want.abs() + tol) + FLUSH).all(), at
        # a split of the tokens adds at most 2^15 of them in fp32
        dw_ref, dw_tol = dw_ref + G.t() @ x64, dw_tol + tg.t() @ x64.abs() + 2 ** 15 * E * (G.abs().t() @ x64.abs())
    assert ((dw.double() - dw_ref).abs() <= dw_tol + out * (dw_ref.abs() + dw_tol)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradient(dtype):
    """One gradient of 2^31 + 12345 elements between small ones."""
    say("grad far", dtype)
    n = (1 << 31) + 12345
    g = torch.Generator(device="cuda").manual_seed(4)
    big = fill((n, 1), dtype, g, 0.01).view(n)
    grads = [torch.ones(5, device="cuda"), big, torch.ones(77, device="cuda")]
    sq = 82.0 + sum(float(big[at:at + (1 << 28)].double().square().sum()) for at in range(0, n, 1 << 28))
    norm, out = tw.grad_clip(grads, 1.0, out=[torch.empty_like(t) for t in grads])
    assert abs(float(norm) - sq ** 0.5) <= 1.01 * E * sq ** 0.5
    c = 1.0 / (sq ** 0.5 + 1e-6)
    check_out([out[0], out[2]], [grads[0], grads[2]], c)
    for at in range(0, n, 1 << 28):
        check_out([out[1][at:at + (1 << 28)]], [big[at:at + (1 << 28)]], c)
    tw.grad_clip(grads, 1.0)
    assert all(torch.equal(a, b) for a, b in zip(grads, out))
