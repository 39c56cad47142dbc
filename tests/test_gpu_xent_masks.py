"""GPU parity of the cross entropy over a vocabulary part of which is masked by a bias column (x's first
element 1, w's the bias): masked entries have probability 0 whatever value masks them. The oracle is
the same problem without them, with the tolerances of the unmasked one."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402
from test_gpu_xent import BF16, E, F32, FLUSH, H, check, problem  # noqa: E402


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def masked(T, d, V, dtype, value):
    """A problem of T tokens whose vocabulary is masked at its end (as padding is), in a run in the
    middle, and here and there; targets are unmasked."""
    x, w, y, dl = problem(T + d + V, T, d, V, dtype, ignored=T // 4)
    keep = torch.ones(V, dtype=torch.bool, device="cuda")
    keep[V - V // 4:] = False
    keep[V // 8:V // 8 + V // 5] = False
    keep[::37] = False
    place = torch.cumsum(keep, 0) - 1
    at = torch.nonzero(keep)[:, 0]
    act = y >= 0
    y[act] = at[y[act] % len(at)]
    x, w = x.clone(), w.clone()
    x[:, 0] = 1
    w[:, 0] = torch.where(keep, 0.0, value).to(dtype)
    return x, w, y, dl, keep, torch.where(act, place[y.clamp(min=0)], y)


# few tokens in place, each of the tiles of the logits, dx whole and split
BF16_SHAPES = [(1, 64, 1000), (20, 64, 33000), (40, 128, 700), (300, 200, 2049), (600, 1024, 5000), (2049, 328, 2500)]
LOWEST = torch.finfo(BF16).min


@pytest.mark.parametrize("value", [LOWEST, -2.5e38, -2.0e38, -1e30, -3e9, -1e4, -900.0])
@pytest.mark.parametrize("T,d,V", BF16_SHAPES)
def test_masked_vocabulary_bf16(T, d, V, value):
    say("xent mask bf16", T, d, V, value)
    x, w, y, dl, keep, yk = masked(T, d, V, BF16, value)
    wk = w[keep]
    check(x, wk, yk, dl, tw.linear_xent_fwd(x, w, y))
    loss, lse, dx, dw = tw.linear_xent_fwd_bwd(x, w, y, dl)
    check(x, wk, yk, dl, (loss, lse, dx, dw[keep]))
    assert not dw[~keep].any()


# fp32 as it is and in planes, with gradients and without
F32_SHAPES = [(1, 64, 1000), (40, 128, 700), (1300, 1032, 2503), (2049, 328, 2500), (2100, 1544, 4099)]


@pytest.mark.parametrize("value", [torch.finfo(F32).min, LOWEST, -2.0e38, -1e30, -1e4])
@pytest.mark.parametrize("T,d,V", F32_SHAPES)
def test_masked_vocabulary_f32(T, d, V, value):
    say("xent mask f32", T, d, V, value)
    x, w, y, dl, keep, yk = masked(T, d, V, F32, value)
    wk = w[keep]
    check(x, wk, yk, dl, tw.linear_xent_fwd(x, w, y))
    loss, lse, dx, dw = tw.linear_xent_fwd_bwd(x, w, y, dl)
    check(x, wk, yk, dl, (loss, lse, dx, dw[keep]))
    assert not dw[~keep].any()


@pytest.mark.parametrize("offset", [2.0 ** 20, -2.0 ** 20, "lowest"])
@pytest.mark.parametrize("T,d,V,dtype", [(40, 128, 700, BF16), (600, 1024, 5000, BF16), (2049, 328, 2500, BF16),
                                         (40, 128, 700, F32), (1300, 1032, 2503, F32)])
def test_rows_far_from_zero_keep_their_softmax(T, d, V, dtype, offset):
    """All logits of a token carry one offset. Small integers make them exact in fp32 (below 2^24) at an
    offset of 2^20, where lse has four bits behind the point left: softmax and loss have all theirs. An
    offset of the type's lowest value swallows the rest: p = 1 / V. Tolerances: 256 E for exponentials,
    the sum and the logarithm, 2 H per element of G in bf16 and 8 E in fp32, as without an offset."""
    say("xent offset", T, d, V, dtype, offset)
    g = torch.Generator(device="cuda").manual_seed(T + V)
    kw = dict(generator=g, device="cuda")
    offset = torch.finfo(dtype).min if offset == "lowest" else offset
    x = torch.randint(-1, 2, (T, d), **kw).to(dtype)
    w = (torch.randint(-1, 2, (V, d), **kw) * (torch.rand(V, d, **kw) < 32 / d)).to(dtype)
    y = torch.randint(0, V, (T,), **kw)
    dl = torch.rand(T, **kw) + 0.5
    x[:, 0], w[:, 0] = 1, offset
    z = x[:, 1:].double() @ w[:, 1:].double().t()
    if abs(offset) > 2.0 ** 24:
        z = torch.zeros_like(z)
    logp = torch.log_softmax(z, 1)
    zt = logp.gather(1, y[:, None])
    loss, lse, dx, dw = tw.linear_xent_fwd_bwd(x, w, y, dl)
    assert ((loss.double() + zt[:, 0]).abs() <= 256 * E * (1 + zt[:, 0].abs())).all()
    assert ((lse.double() - (offset + torch.logsumexp(z, 1))).abs() <= 2 * E * lse.double().abs()).all()
    fwd = tw.linear_xent_fwd(x, w, y)
    assert ((fwd[0].double() + zt[:, 0]).abs() <= 256 * E * (1 + zt[:, 0].abs())).all()
    p, d64 = torch.exp(logp), dl.double()[:, None]
    G = (p * d64).scatter_(1, y[:, None], torch.expm1(zt) * d64)
    tg = G.abs() * (2 * H if dtype == BF16 else 8 * E) + p * d64 * 256 * E + FLUSH * (1 + d64)
    out = H if dtype == BF16 else E
    x64, w64 = x.double(), w.double()
    ref = G.t() @ x64
    tol = tg.t() @ x64.abs() + (T + 8) * E * (G.abs().t() @ x64.abs())
    assert ((dw.double() - ref).abs() <= tol + out * (ref.abs() + tol) + FLUSH).all()
    ref = G @ w64[:, 1:]                    # the offset's own column sums G to 0 times the offset
    tol = tg @ w64[:, 1:].abs() + V * E * (G.abs() @ w64[:, 1:].abs())
    assert ((dx[:, 1:].double() - ref).abs() <= tol + out * (ref.abs() + tol) + FLUSH).all()


@pytest.mark.parametrize("T,d,V,dtype", [(1, 64, 1000, BF16), (300, 200, 2049, BF16), (600, 1024, 5000, BF16),
                                         (2049, 328, 2500, BF16), (20, 64, 33000, F32), (40, 128, 700, F32),
                                         (1300, 1032, 2503, F32)])
def test_infinite_mask(T, d, V, dtype):
    """A bias of minus infinity masks as well, in scoring by bf16 products and by fp32 ones as they are. A
    masked target's loss is infinite. The gradients of the other columns are those without the masked
    entries; the bias column of dx is 0 times infinity."""
    say("xent infinite mask", T, d, V, dtype)
    x, w, y, dl, keep, yk = masked(T, d, V, dtype, -float("inf"))
    check(x, w[keep], yk, dl, tw.linear_xent_fwd(x, w, y))
    if dtype == BF16:
        loss, lse, dx, dw = tw.linear_xent_fwd_bwd(x, w, y, dl)
        act = y >= 0
        assert torch.isnan(dx[act][:, 0].float()).all()
        dx = dx.clone()
        want = tw.linear_xent_fwd_bwd(x, w[keep].contiguous(), yk, dl)[2]
        dx[:, 0] = want[:, 0]
        check(x, w[keep], yk, dl, (loss, lse, dx, dw[keep]))
        assert not dw[~keep].any()
    y[T - 1] = int(torch.nonzero(~keep)[3])
    loss, lse = tw.linear_xent_fwd(x, w, y)
    assert loss[T - 1] == float("inf") and torch.isfinite(lse).all() and torch.isfinite(loss[:-1]).all()
