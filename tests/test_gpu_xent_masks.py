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
from test_gpu_xent import BF16, F32, check, problem  # noqa: E402


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
