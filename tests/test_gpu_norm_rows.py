"""The layer norm over more rows than its launches have workgroups, up to the last row that 32 bits
count."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402
from test_gpu_norm import HALF, bwd64, check_fwd, gen, rows  # noqa: E402

E = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.fixture
def much_memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 200 << 30:
        pytest.skip("needs 200 GiB of free GPU memory")
    yield
    torch.cuda.empty_cache()


T_MAX = (1 << 31) - 1                       # a workgroup's row passes 2^31 in its last step
# the first and last rows of the tensor, of a launch's first round and of its last
SOME = [0, 1, 4095, 4096, 8191, 8192, 1 << 20, (1 << 31) - 8194, (1 << 31) - 8192, (1 << 31) - 4097, (1 << 31) - 4096,
        T_MAX - 2, T_MAX - 1]


def parts(n=1 << 27):
    for at in range(0, T_MAX, n):
        yield slice(at, min(T_MAX, at + n))


def test_fwd_of_all_rows_that_32_bits_count(much_memory):
    """Rows of zeros give the bias; some others give what they give alone."""
    say("norm fwd", T_MAX, 8)
    g = torch.Generator().manual_seed(1)
    at = torch.tensor(SOME).cuda()
    few = torch.randn(len(SOME), 8, generator=g).to(BF16).cuda()
    w, b = torch.randn(8, generator=g).cuda(), torch.randn(8, generator=g).cuda()
    x = torch.zeros(T_MAX, 8, dtype=BF16, device="cuda")
    x[at] = few
    y, _, mean, rstd = tw.layer_norm_fwd(x, w, b)
    alone = tw.layer_norm_fwd(few, w, b)
    assert torch.equal(y[at], alone[0]) and torch.equal(mean[at], alone[2]) and torch.equal(rstd[at], alone[3])
    y[at] = b.to(BF16)
    for p in parts():
        assert (y[p] == b.to(BF16)).all(), p


def test_bwd_of_all_rows_that_32_bits_count(much_memory):
    """Rows whose dy is zero add nothing; dw and db are the sums over the others (a path of at most
    T / 4096 additions of zero, and one of each row: 128 E, as for few rows)."""
    say("norm bwd", T_MAX, 8)
    g = torch.Generator().manual_seed(2)
    at = torch.tensor(SOME).cuda()
    few, dfew = (torch.randn(len(SOME), 8, generator=g).to(BF16).cuda() for _ in range(2))
    w = torch.randn(8, generator=g).cuda()
    s = torch.zeros(T_MAX, 8, dtype=BF16, device="cuda")
    dy = torch.zeros(T_MAX, 8, dtype=BF16, device="cuda")
    mean, rstd = torch.zeros(T_MAX, device="cuda"), torch.ones(T_MAX, device="cuda")
    s[at], dy[at] = few, dfew
    dx, dw, db = tw.layer_norm_bwd(dy, s, w, mean, rstd)
    alone = tw.layer_norm_bwd(dfew, few, w, mean[at], rstd[at])
    assert torch.equal(dx[at], alone[0])
    xh, d64 = few.double(), dfew.double()   # mean 0, rstd 1
    assert ((dw.double() - (d64 * xh).sum(0)).abs() <= 128 * E * (d64 * xh).abs().sum(0)).all()
    assert ((db.double() - d64.sum(0)).abs() <= 128 * E * d64.abs().sum(0)).all()
    dx[at] = 0
    for p in parts():
        assert not dx[p].any(), p


@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("T,d,residual", [(8193, 64, True), (8200, 72, False), (20000, 64, True), (9000, 8200, True)])
def test_fwd_rows_in_rounds(T, d, xt, yt, residual):
    """More rows than workgroups (8192), with one and with two units per thread: every workgroup takes
    rows in turn, and a row of NaN leaves those that follow it alone."""
    say("norm fwd rounds", T, d, xt, yt, residual)
    g = gen(T + d)
    x = rows(g, min(T, 1000), d, xt).repeat(T // 1000 + 1, 1)[:T].contiguous()
    x[:: 3] *= 2
    r = rows(g, 1, d, xt).repeat(T, 1) if residual else None
    w, b = torch.randn(d, generator=g).cuda(), torch.randn(d, generator=g).cuda()
    clean = tw.layer_norm_fwd(x, w, b, residual=r, y_dtype=yt)
    some = torch.cat([torch.arange(0, 40), torch.arange(T // 2, T // 2 + 40), torch.arange(T - 40, T)])
    at = some.cuda()
    check_fwd(clean[1][at], w, b, 1e-5, clean[0][at], clean[2][at], clean[3][at])
    for p in range(0, T, 4096):             # each row as in a call of fewer rows
        q = slice(p, min(T, p + 4096))
        few = tw.layer_norm_fwd(x[q], w, b, residual=r[q] if residual else None, y_dtype=yt)
        assert all(torch.equal(a[q], c) for a, c in zip(clean, few))
    x[7], x[8192 - 1] = float("nan"), float("inf")
    got = tw.layer_norm_fwd(x, w, b, residual=r, y_dtype=yt)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[7] = rest[8191] = False
    assert torch.equal(got[0][rest], clean[0][rest]) and torch.equal(got[2][rest], clean[2][rest])
    assert torch.isnan(got[0][~rest].float()).all()


@pytest.mark.parametrize("xt,dyt,dxt", [(BF16, F32, BF16), (F32, F32, F32), (F32, BF16, BF16), (BF16, BF16, F32)])
@pytest.mark.parametrize("T,d", [(16384, 64), (5000, 72), (4097, 1032), (40, 8200), (700, 8200), (600, 16384)])
def test_bwd_strips(T, d, xt, dyt, dxt):
    """More than 512 strips (T > 4096), and several strips with two units per thread (d > 8192). A path of
    a sum over tokens: T / strips <= 8 rows, 16 strips of a group and 24 groups, below 128."""
    say("norm bwd strips", T, d, xt, dyt, dxt)
    g = gen(T * 3 + d)
    s, dy = rows(g, T, d, xt, d + 8), rows(g, T, d, dyt, d + 16)
    dres = rows(g, T, d, dxt, d + 24) if T % 8 else None
    w = torch.randn(d, generator=g).cuda()
    _, _, mean, rstd = tw.layer_norm_fwd(s, w, eps=1e-5)
    dx, dw, db = tw.layer_norm_bwd(dy, s, w, mean, rstd, dres=dres, dx_dtype=dxt)
    for name, got, (ref, tol) in zip(("dx", "dw", "db"), (dx, dw, db), bwd64(dy, s, w, mean, rstd, dres)):
        tol = tol + HALF[got.dtype] * (ref.abs() + tol)
        bad = (got.double().cpu() - ref).abs() > tol
        assert not bad.any(), (name, int(bad.sum()), float(((got.double().cpu() - ref).abs() - tol).max()))
    again = tw.layer_norm_bwd(dy, s, w, mean, rstd, dres=dres, dx_dtype=dxt, want_bias=False)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and again[2] is None


def test_bwd_nan_stays_in_its_place():
    """A NaN in s: its row of dx and all of dw, not db. One in dy: its row of dx, its column of dw and db."""
    g = gen(31)
    T, d = 5000, 72
    s, dy, w = rows(g, T, d, BF16), rows(g, T, d, F32), torch.randn(d, generator=g).cuda()
    _, _, mean, rstd = tw.layer_norm_fwd(s, w)
    dx0, dw0, db0 = tw.layer_norm_bwd(dy, s, w, mean, rstd)
    s2 = s.clone()
    s2[4100, 3] = float("nan")
    _, _, mean2, rstd2 = tw.layer_norm_fwd(s2, w)
    dx, dw, db = tw.layer_norm_bwd(dy, s2, w, mean2, rstd2)
    rest = torch.arange(T, device="cuda") != 4100
    assert torch.equal(dx[rest], dx0[rest]) and torch.isnan(dx[4100].float()).all()
    assert torch.isnan(dw).all() and torch.equal(db, db0)
    dy2 = dy.clone()
    dy2[4100, 3] = float("nan")
    dx, dw, db = tw.layer_norm_bwd(dy2, s, w, mean, rstd)
    cols = torch.arange(d, device="cuda") != 3
    assert torch.equal(dx[rest], dx0[rest]) and torch.isnan(dx[4100].float()).all()
    assert torch.equal(dw[cols], dw0[cols]) and torch.equal(db[cols], db0[cols])
    assert torch.isnan(dw[3]) and torch.isnan(db[3])
