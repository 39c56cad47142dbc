"""The dense layers on whole numbers. Every product, sum and activation (relu or none) of these operands is a whole
number below 2^24, exact in fp32 in any order, so that the results are equal to the formulas', fp32 ones to the bit and
bf16 ones after their one rounding: a lost or doubled term of a long sum shows, as no bound on its rounding would let it.
fp32 operands have up to 17 digits, which takes all three planes of a product that splits them."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402
from dense_shapes import CASES  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}
LIMIT = float(1 << 24) / 1.02                       # (the planes of a number add up to 1.01 times its size)


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(g, rows, cols, size, share, dtype, stride=0):
    """Whole numbers up to +-size, a share of them not zero; NaN between the rows where they lie apart."""
    t = torch.full((rows, cols + stride), float("nan"), device="cuda", dtype=dtype)
    v = torch.randint(-int(size), int(size) + 1, (rows, cols), generator=g, device="cuda", dtype=torch.int32)
    t[:, :cols] = (v * (torch.rand(rows, cols, generator=g, device="cuda") < share)).to(dtype)
    t = t[:, :cols]
    assert dtype == F32 or size <= 256
    return t


def product(a, b):
    """a b^T in 64 bits, whose partial sums are all exact in 32."""
    assert float((a.abs() @ b.abs().t()).max()) < LIMIT
    return a @ b.t()


def same(got, want, what):
    want = want.to(F32).to(got.dtype)
    assert got.shape == want.shape
    assert torch.equal(got, want), (what, int((got != want).sum()), (got != want).nonzero()[:4].tolist())


def once(t, dtype):
    """Rounded as an operand of the next product."""
    return t.to(F32).to(dtype).double()


def share_for(size, n):
    """The share of numbers that may differ from zero in a sum of n products up to size."""
    return min(1.0, 2.0 ** 22 / (size * n))


def run_linear(T, K, N, dtype, layout, wide_x):
    wide = 127 if dtype == BF16 else 1 << 17
    g, p = gen(T + K + N), share_for(wide, K)
    x = whole(g, T, K, wide if wide_x else 1, 1 if wide_x else p, dtype, 8)
    w = whole(g, *((N, K) if layout == "nk" else (K, N)), 1 if wide_x else wide, p if wide_x else 1, dtype)
    b = torch.randint(-1000, 1001, (N,), generator=g, device="cuda").float()
    r = whole(g, T, N, 100, 1, F32, 8)
    z = product(x.double(), (w if layout == "nk" else w.t()).double()) + b.double()
    y, pre = tw.linear_fwd(x, w, bias=b, residual=r, act="relu", w_layout=layout, y_dtype=F32, want_pre=True)
    same(y, z.clamp(min=0) + r.double(), "y")
    same(pre, z, "pre")
    same(tw.linear_fwd(x, w, bias=b, w_layout=layout)[0], z, "y in the operands' type")


def run_linear_back(T, K, N, dtype, layout, wide_dy):
    cap = 127 if dtype == BF16 else 1 << 17
    g = gen(T + K + N)
    if wide_dy:
        big = min(cap, max(1, (1 << 23) // T))
        dy, p = whole(g, T, N, big, 1, dtype, 8), share_for(big, max(T, N))
        small, size = p, 1
    else:
        size, small = cap, 1
        dy = whole(g, T, N, 1, share_for(cap, max(T, N)), dtype, 8)
    x, w = whole(g, T, K, size, small, dtype, 8), whole(g, *((N, K) if layout == "nk" else (K, N)), size, small, dtype)
    pre = whole(g, T, N, 3, 1, dtype)
    for act in ("relu", "none"):
        dz = dy.double() * (pre > 0) if act == "relu" else dy.double()
        assert float(dz.abs().sum(0).max()) < LIMIT
        dx, dw, db = tw.linear_bwd(dy, x, w, pre=pre, act=act, w_layout=layout, want_bias=True)
        same(dx, product(dz, (w.t() if layout == "nk" else w).double()), "dx")
        want = product(dz.t().contiguous(), x.double().t().contiguous())
        same(dw if layout == "nk" else dw.t(), want, "dw")
        same(db, dz.sum(0), "db")


def run_gated(T, d, f, dtype, act):
    g = gen(T + d + f)
    x = whole(g, T, d, 1, 0.75, dtype, 8)
    up = min(1.0, 48 / d)                               # g up to about 20; u the same, or 2^10 times that
    wide = 1 if dtype == BF16 else 1 << 10
    wg, wu = whole(g, f, d, 1, up, dtype), whole(g, f, d, wide, up, dtype)
    w2 = whole(g, f, d, 1, share_for(200 * wide, f), dtype)
    bg, bu = (torch.randint(-3, 4, (f,), generator=g, device="cuda").float() for _ in range(2))
    r = whole(g, T, d, 100, 1, F32, 8)
    G, U = product(x.double(), wg.double()) + bg.double(), product(x.double(), wu.double()) + bu.double()
    h = (G.clamp(min=0) if act == "relu" else G) * U
    assert float(h.abs().max()) < LIMIT
    want = product(once(h, dtype), w2.double().t())
    y, gs, us = tw.ffn_gated_dense_fwd(x, wg, wu, w2, bg=bg, bu=bu, residual=r, act=act, y_dtype=F32, want_saved=True)
    same(gs, G, "g")
    same(us, U, "u")
    same(y, want + r.double(), "y")
    same(tw.ffn_gated_dense_fwd(x, wg, wu, w2, bg=bg, bu=bu, act=act)[0], want, "y in the operands' type")


def run_gated_back(T, d, f, dtype, act):
    g = gen(T + d + f)
    wide = 5 if dtype == BF16 else 64
    share = min(1.0, 32 / d)
    dy, w2 = whole(g, T, d, 5, 0.5, dtype, 8), whole(g, f, d, wide, share, dtype)
    G, U = whole(g, T, f, 3, 1, dtype), whole(g, T, f, 3, 1, dtype)
    dh = product(dy.double(), w2.double())
    a, da = (G.double().clamp(min=0), (G > 0).double()) if act == "relu" else (G.double(), 1.0)
    dg, du, h = dh * U.double() * da, dh * a, a * U.double()
    big = float(torch.maximum(dg.abs(), du.abs()).mean()) + 1
    x = whole(g, T, d, 1, share_for(big, 2 * T), dtype, 8)
    wg, wu = (whole(g, f, d, 1, share_for(big, 2 * f), dtype) for _ in range(2))
    got = tw.ffn_gated_dense_bwd(dy, x, wg, wu, w2, G, U, act=act, want_bias=True)
    rg, ru, rh = (once(t, dtype) for t in (dg, du, h))
    both = torch.cat([rg, ru], 1)
    same(got[0], product(both, torch.cat([wg, wu]).double().t()), "dx")
    x64 = x.double().t().contiguous()
    same(got[1], product(rg.t().contiguous(), x64), "dwg")
    same(got[2], product(ru.t().contiguous(), x64), "dwu")
    same(got[3], product(rh.t().contiguous(), dy.double().t().contiguous()), "dw2")
    for k, t in ((4, dg), (5, du)):
        assert float(t.abs().sum(0).max()) < LIMIT
        same(got[k], t.sum(0), ("dbg", "dbu")[k - 4])
    for t, u in zip(tw.ffn_gated_dense_bwd(dy, x, wg, wu, w2, G, U, act=act)[:4], got):
        assert torch.equal(t, u)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("other", [False, True])
def test_whole_numbers(case, other):
    op, T, K, N, t, layout = case
    say("exact", case, other)
    if op == "linear":
        run_linear(T, K, N, TYPES[t], layout, other)
    elif op == "linear_back":
        run_linear_back(T, K, N, TYPES[t], layout, other)
    elif op == "gated":
        run_gated(T, K, N, TYPES[t], "relu" if other else "none")
    else:
        run_gated_back(T, K, N, TYPES[t], "relu" if other else "none")


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("K,N", [(4104, 64), (64, 4104)])
def test_far_rows(K, N, layout):
    """x or y, dz and dx of 530003 x 4104, beyond 2^31 elements: every output, the sums over all rows among them."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of free GPU memory")
    T, step = 530003, 1 << 16
    say("exact far", T, K, N, layout)
    g = gen(K)
    x, dy, pre = (torch.empty(T, n, dtype=BF16, device="cuda") for n in (K, N, N))
    for at in range(0, T, step):
        for t in (x, dy, pre):
            p = t[at:at + step]
            p.copy_(torch.randint(-3, 4, p.shape, generator=g, device="cuda"))
    w = whole(g, *((N, K) if layout == "nk" else (K, N)), 3, 1, BF16)
    w64 = (w if layout == "nk" else w.t()).double()
    y, z = tw.linear_fwd(x, w, residual=dy, act="relu", w_layout=layout, want_pre=True)
    dx, dw, db = tw.linear_bwd(dy, x, w, pre=pre, act="relu", w_layout=layout, want_bias=True)
    assert 9.0 * T < LIMIT
    sums, one = 0, 0
    for at in range(0, T, step):
        sel = slice(at, at + step)
        x64 = x[sel].double()
        want = product(x64, w64)
        same(z[sel], want, ("pre", at))
        same(y[sel], want.clamp(min=0) + dy[sel].double(), ("y", at))
        dz = dy[sel].double() * (pre[sel] > 0)
        same(dx[sel], product(dz, w64.t()), ("dx", at))
        sums, one = sums + dz.t() @ x64, one + dz.sum(0)
    assert bool((sums != 0).any()) and bool((one != 0).any())
    same(dw if layout == "nk" else dw.t(), sums, "dw")
    same(db, one, "db")
