"""The dense operators together in training steps (examples/dense_step.py): the gradients against 64-bit
autograd of the formulas, and steps with states in 32 and in 8 bits."""
import importlib.util
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("dense_step_example", os.path.join(ROOT, "examples", "dense_step.py"))
ex = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ex)


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def dense64(m, tokens, targets):
    """Loss and gradients of the same model in 64 bits."""
    p = {k: v.double().clone().requires_grad_() for k, v in m.p.items()}

    def norm(x, w, b):
        v = x - x.mean(1, keepdim=True)
        return v / ((v * v).mean(1, keepdim=True) + 1e-5).sqrt() * w + b
    z = m.emb[tokens].double() @ p["in.w"].t() + p["in.b"]
    x = z * torch.special.ndtr(z)
    for i in range(m.blocks):
        a = norm(x, p[f"{i}.norm.w"], p[f"{i}.norm.b"])
        g, u = a @ p[f"{i}.wg"].t() + p[f"{i}.bg"], a @ p[f"{i}.wu"].t() + p[f"{i}.bu"]
        x = x + (g * torch.sigmoid(g) * u) @ p[f"{i}.w2"]
    z = norm(x, p["norm.w"], p["norm.b"]) @ p["head"].t()
    act = targets >= 0
    loss = (torch.logsumexp(z[act], 1) - z[act].gather(1, targets[act][:, None])[:, 0]).mean()
    loss.backward()
    return loss.detach(), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("dtype,loss_off,off", [(torch.float32, 1e-5, 1e-4), (torch.bfloat16, 0.02, 0.1)])
def test_gradients(dtype, loss_off, off):
    """fp32: sums of at most a few thousand roundings of 2^-24 per stage, a dozen stages, stay far below 1e-4. bf16:
    half a step of 2^-8 at each of some fifteen roundings on a gradient's way; 0.1 in the norm is an order
    above their sum in the square, and far below a wrong term."""
    m = ex.Model(300, 128, 512, 2, dtype)
    for k in m.p:
        m.p[k] = m.p[k] + 0.1 * torch.randn_like(m.p[k]) if m.p[k].dim() == 1 else m.p[k].to(dtype).float()
    m.refresh()
    tokens, targets = ex.batch(300, 200, 3)
    loss, grads = ex.loss_and_gradients(m, tokens, targets)
    ref, want = dense64(m, tokens, targets)
    assert abs(float(loss) - float(ref)) <= loss_off * float(ref)
    assert set(grads) == set(want)
    for k, g in grads.items():
        say(k, float((g.double() - want[k]).norm() / want[k].norm()))
        assert (g.double() - want[k]).norm() <= off * want[k].norm(), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("states", ["32", "8"])
def test_steps_run(dtype, states):
    losses = ex.main(["--steps", "6", "--dtype", dtype, "--states", states, "--vocab", "499", "--tokens", "300"])
    assert len(losses) == 6 and all(l == l for l in losses)


@pytest.mark.parametrize("states", [32, 8])
def test_copies_follow_the_weights(states):
    m = ex.Model(100, 64, 128, 1, torch.bfloat16)
    opt = ex.Adam(m, lr=1e-2, states=states)
    before = {k: v.clone() for k, v in m.p.items()}
    _, grads = ex.loss_and_gradients(m, *ex.batch(100, 70, 1))
    opt.step(m, grads)
    for k, v in m.p.items():
        assert not torch.equal(v, before[k]), k
        assert torch.equal(m.w[k], v.to(torch.bfloat16) if v.dim() == 2 else v), k
