"""The cross entropy at the largest number of tokens that its header allows, where one workgroup per token
is one thread more than a launch counts."""
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


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1 << 24, (1 << 24) - 77, (1 << 23) + 1])
def test_most_tokens(T, dtype):
    """Positive x and targets that are mostly 0: no term of dw cancels, so that a piece, a split or a
    launch left out shows. Logits of 8 products: 12 E of sum |x w| <= 8, and 256 E for the rest; a
    split of at most 2^15 tokens adds dw with 2^15 E."""
    say("xent most tokens", T, dtype)
    d, V = 8, 7
    g = torch.Generator(device="cuda").manual_seed(T)
    kw = dict(generator=g, device="cuda")
    x = (0.5 + torch.rand(T, d, **kw)).to(dtype)
    w = (torch.rand(V, d, **kw) - 0.5).to(dtype)
    y = torch.where(torch.rand(T, **kw) < 0.9, 0, torch.randint(0, V, (T,), **kw))
    y[::5] = -1
    y[T - 1], y[0] = 3, 2
    dl = torch.rand(T, **kw) + 0.5
    act = y >= 0
    w64 = w.double()
    dw_ref, dw_abs = torch.zeros(V, d, dtype=torch.float64, device="cuda"), 0
    got = tw.linear_xent_fwd_bwd(x, w, y, dl)
    fwd = tw.linear_xent_fwd(x, w, y)
    assert torch.equal(fwd[0], got[0]) and torch.equal(fwd[1], got[1])
    out = H if dtype == BF16 else E
    for at in range(0, T, 1 << 22):
        p = slice(at, min(T, at + (1 << 22)))
        a, x64 = act[p], x[p].double()
        logp = torch.log_softmax(x64 @ w64.t(), 1)
        lt = logp.gather(1, y[p].clamp(min=0)[:, None])
        loss = torch.where(a, -lt[:, 0], 0.0)
        assert ((got[0][p].double() - loss).abs() <= 512 * E * (1 + loss)).all()
        G = logp.exp() * dl[p].double()[:, None]
        G.scatter_(1, y[p].clamp(min=0)[:, None], torch.expm1(lt) * dl[p].double()[:, None])
        G *= a[:, None]
        tg = G.abs() * (2 * H if dtype == BF16 else 8 * E) + 512 * E * dl[p].double()[:, None] + FLUSH
        dx = G @ w64
        tol = tg @ w64.abs()
        assert ((got[2][p].double() - dx).abs() <= tol + out * (dx.abs() + tol)).all()
        assert not got[2][p][~a].any()
        dw_ref += G.t() @ x64
        dw_abs = dw_abs + tg.t() @ x64 + 2 ** 15 * E * (G.abs().t() @ x64)
    assert ((got[3].double() - dw_ref).abs() <= dw_abs + out * (dw_ref.abs() + dw_abs)).all()
    assert (dw_abs[0] < 0.02 * dw_ref[0].abs()).all()


def test_dw_of_no_tokens_of_a_head_beyond_64_gib():
    """T = 0 clears all of dw."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 200 << 30:
        pytest.skip("needs 200 GiB of free GPU memory")
    V, d = (1 << 20) + 3, 1 << 15
    say("xent no tokens", V, d)
    w = torch.empty(V, d, dtype=BF16, device="cuda")
    old = torch.full((V, d), 1.0, dtype=BF16, device="cuda")
    del old                                 # dw takes its place
    x, y, dl = torch.empty(0, d, dtype=BF16).cuda(), torch.empty(0, dtype=torch.int64).cuda(), torch.empty(0).cuda()
    dw = tw.linear_xent_fwd_bwd(x, w, y, dl)[3]
    assert dw.shape == (V, d)
    for at in range(0, V, 1 << 15):
        assert not dw[at:at + (1 << 15)].any(), at
    del w, dw
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,d,V,ignored", [(1500, 768, 100003, 200), (1500, 1024, 100003, 600), (3000, 512, 100003, 7),
                                           (2600, 1024, 60001, 0)])
def test_pieces_in_planes(T, d, V, ignored):
    """Several pieces of rows of fp32 products that run in bf16 planes (pieces of 1024, 1024, 1024 and 1536
    rows); the last piece of the second case is empty. The workspace tells the path: as it is, fp32 takes
    no more than a piece of 1 GiB, x's copy, the lists and 200 MB of partial sums."""
    say("xent planes, pieces", T, d, V, ignored)
    need = tw.linear_xent_workspace_bytes(T, d, V, F32)
    assert need > (1 << 30) + T * d * 4 + 12 * T + 200_000_000, "not in planes"
    assert T * V * 10 > 1 << 30, "one piece"
    x, w, y, dl = problem(T + d, T, d, V, F32, ignored=ignored)
    got = tw.linear_xent_fwd_bwd(x, w, y, dl)
    check(x, w, y, dl, got)
    for a, b in zip(got, tw.linear_xent_fwd_bwd(x, w, y, dl)):
        assert torch.equal(a, b)
