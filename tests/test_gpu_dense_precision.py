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
