"""The operators together in a training step (examples/train_step.py): its gradients against 64-bit
autograd of the dense formulas, and the loss over some steps."""
import importlib.util
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("train_step_example", os.path.join(ROOT, "examples", "train_step.py"))
ex = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ex)


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def dense64(m, tokens, targets):
    """Loss and gradients of the same model in 64 bits."""
    p = {k: v.double().clone().requires_grad_() for k, v in m.p.items()}

    def norm(x, w, b):
        mu = x.mean(1, keepdim=True)
        v = x - mu
        return v / ((v * v).mean(1, keepdim=True) + 1e-5).sqrt() * w + b
    x = m.emb[tokens].double()
    for i in range(m.blocks):
        a = norm(x, p[f"{i}.norm.w"], p[f"{i}.norm.b"])
        x = x + torch.relu(a @ p[f"{i}.w1t"].t() + p[f"{i}.b1"]) @ p[f"{i}.w2"]
    z = norm(x, p["norm.w"], p["norm.b"]) @ p["head"].t()
    act = targets >= 0
    loss = (torch.logsumexp(z[act], 1) - z[act].gather(1, targets[act][:, None])[:, 0]).mean()
    loss.backward()
    return loss.detach(), {k: v.grad for k, v in p.items()}


def test_gradients_in_fp32():
    """fp32 throughout: the chain's relative error stays far below 1e-4 (sums of at most a few
    thousand fp32 roundings of 2^-24 each per stage, a dozen stages)."""
    m = ex.Model(300, 128, 512, 2, torch.float32)
    tokens, targets = ex.batch(300, 200, 3)
    loss, grads = ex.loss_and_gradients(m, tokens, targets)
    ref, want = dense64(m, tokens, targets)
    assert abs(float(loss) - float(ref)) <= 1e-5 * float(ref)
    assert set(grads) == set(want)
    for k, g in grads.items():
        say(k, float((g.double() - want[k]).norm() / want[k].norm()))
        assert (g.double() - want[k]).norm() <= 1e-4 * want[k].norm(), k


def test_gradients_in_bf16():
    """bf16 weights and residual stream: half a step of 2^-8 at each of some ten roundings on a
    gradient's way, and hidden units near zero that change sides; 0.1 in the norm is an order above
    their sum, and far below a wrong term."""
    m = ex.Model(300, 128, 512, 2, torch.bfloat16)
    for k in list(m.p):
        m.p[k] = m.p[k].to(torch.bfloat16).float()          # both sides start from the same weights
    tokens, targets = ex.batch(300, 200, 4)
    loss, grads = ex.loss_and_gradients(m, tokens, targets)
    ref, want = dense64(m, tokens, targets)
    assert abs(float(loss) - float(ref)) <= 0.02 * float(ref)
    for k, g in grads.items():
        say(k, float((g.double() - want[k]).norm() / want[k].norm()))
        assert (g.double() - want[k]).norm() <= 0.1 * want[k].norm(), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_loss_falls(dtype):
    losses = ex.main(["--steps", "20", "--dtype", dtype, "--vocab", "499"])
    assert all(l == l for l in losses) and losses[-1] < losses[0] - 0.5
