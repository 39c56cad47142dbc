"""What a result's type promises, whatever the operands' type: activations of fp32 results, derivatives in fp32
column sums. E = 2^-24. The products are of zeros, so the activation's argument is the bias, or ``pre``, itself."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
E = 2.0 ** -24


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.mark.parametrize("act", list(tw.ACTS))
@pytest.mark.parametrize("T,K,N,layout", [(1, 8, 8200, "nk"), (5, 2056, 4104, "kn"), (300, 64, 1000, "nk"), (1200, 72, 4096, "kn"),
                                          (40, 8192, 1024, "nk")])
def test_fp32_results_of_bf16_operands(T, K, N, layout, act):
    """y in fp32 is the activation as fp32 operands have it, to the last bit: the forms that are good to a bf16
    result's rounding only (gelu at -4: 0.1% off) stay with bf16 results."""
    say("fp32 result", T, K, N, layout, act)
    z = torch.linspace(-20, 20, N, device="cuda")

    def y(dtype):
        x = torch.zeros(T, K, device="cuda", dtype=dtype)
        w = torch.zeros((N, K) if layout == "nk" else (K, N), device="cuda", dtype=dtype)
        return tw.linear_fwd(x, w, bias=z, act=act, w_layout=layout, y_dtype=F32)[0]
    got, want = y(BF16), y(F32)
    assert got.dtype == F32 and torch.equal(got, want), float((got - want).abs().max())


def derivative(z, act):
    """(a'(z), its error) in 64 bits. s = sigmoid(x), t = sigmoid(-x) with x = z (silu) or 2 a (gelu_tanh, x off by
    6 E |x| for its six roundings). The exponential e = exp(-|x|) is off by 3 E of itself and, on the hardware's exp2,
    by the rounding of |x| / ln 2 and of that constant, 2 E |x|; 1 / (1 + e) by 3 E more and by e's error times e / (1 + e) <
    min(s, t) / max(s, t). So the larger of s and t is off by 4 E + min(s, t) 2 r and the smaller by 5 E + r with
    r = (3 + 8 |x|) E. d = s + s t z x'(z), x' off by 5 E, its products and sum 4 E. An exponential below 2^-126 (from
    |x| = 87.3) may be flushed to zero: the smaller of s and t is then off by up to 2^-126, and d by 2^-126 (1 + |z x'|),
    its own flushing 2^-126 more."""
    s, t = torch.sigmoid(z), torch.sigmoid(-z)
    x, slope = z, torch.ones_like(z)
    if act == "gelu_tanh":
        c = 2 * (2 / torch.pi) ** 0.5
        x, slope = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)
        s, t = torch.sigmoid(x), torch.sigmoid(-x)
    r = (3 + 8 * x.abs()) * E
    low, high = 5 * E + r, 4 * E + 2 * r * torch.minimum(s, t)
    rs, rt = torch.where(x < 0, low, high), torch.where(x < 0, high, low)
    far = (s * t * z * slope).abs()
    return s + s * t * z * slope, rs * s + (rs + rt + 5 * E) * far + 4 * E * (s + far) + 2.0 ** -126 * (2 + (z * slope).abs())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_derivatives(act, dtype):
    """db of one token with dy = 1 is the derivative: its factor 1 - s does not lose its digits where s is near 1 (there z
    times it would bring 16 E and more)."""
    say("derivative", act, dtype)
    n = 1 << 19
    if dtype == F32:
        z = torch.linspace(-30, 30, n, device="cuda")
    else:
        z = torch.arange(1 << 16, device="cuda").to(torch.int32).to(torch.int16).view(BF16)
        z = z[z.abs() < 1000]                            # every one below it
        z = z[:z.numel() // 8 * 8].contiguous()
        n = z.numel()
    x, w = torch.zeros(1, 8, device="cuda", dtype=dtype), torch.zeros(n, 8, device="cuda", dtype=dtype)
    db = tw.linear_bwd(torch.ones(1, n, device="cuda", dtype=dtype), x, w, pre=z[None], act=act, want_dx=False, want_dw=False,
                       want_bias=True)[2].double()
    want, tol = derivative(z.double(), act)
    err = (db - want).abs()
    assert float(tol[z >= 6].max()) < 10 * E
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max() / E), float(z[(err / tol).argmax()]))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_derivatives_at_the_ends(dtype):
    """Arguments whose exponential is 0 or whose square is infinite, infinities and NaN."""
    z = torch.tensor([-3e38, -1e20, -200, -104, -88.8, 88.8, 104, 200, 1e20, 3e38, float("nan")] + [0.0] * 5, device="cuda").to(dtype)
    x, w = torch.zeros(1, 8, device="cuda", dtype=dtype), torch.zeros(16, 8, device="cuda", dtype=dtype)
    for act in ("silu", "gelu_tanh"):
        db = tw.linear_bwd(torch.ones(1, 16, device="cuda", dtype=dtype), x, w, pre=z[None], act=act, want_bias=True)[2]
        assert (db[:5].abs() <= 2.0 ** -100).all() and torch.equal(db[5:10], torch.ones(5, device="cuda")), (act, db)
        assert torch.isnan(db[10]) and (db[11:] == 0.5).all()
