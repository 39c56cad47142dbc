"""The layer norm over more rows than its launches have workgroups, up to the last row that 32 bits
count."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402

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
