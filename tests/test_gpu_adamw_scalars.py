"""Device scalars of adamw_step that no step can be made of: the values that the host's check refuses, read by the
kernel instead, skip the step. Nothing is written."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402

NAN, INF = float("nan"), float("inf")


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def state(states):
    g = torch.Generator(device="cuda").manual_seed(1)
    p = [torch.randn(n, generator=g, device="cuda") for n in (5000, 33)]
    t = dict(params=p, grads=[0.1 * torch.randn(x.shape, generator=g, device="cuda") for x in p])
    if states == 8:
        st = [tw.adamw8_states(x) for x in p]
        t.update(zip(("m", "m_scales", "v", "v_scales"), (list(x) for x in zip(*st))))
        for m, v in zip(t["m"], t["v"]):
            m.fill_(5)
            v.fill_(100)
        for s in t["m_scales"] + t["v_scales"]:
            s.fill_(1e-8)
    else:
        t.update(m=[0.01 * x for x in p], v=[(0.1 * x).square() for x in p])
    t["copies"] = [torch.full_like(x, 5.0, dtype=torch.bfloat16) for x in p]
    return t


BAD = [dict(step=0), dict(step=-3), dict(step=-(1 << 62)), dict(lr=NAN), dict(lr=-1e-3), dict(lr=INF), dict(lr=2e30),
       dict(norm=-1.0), dict(norm=-1e-6), dict(step=0, lr=NAN), dict(step=1, lr=-INF)]


@pytest.mark.parametrize("states", [32, 8])
@pytest.mark.parametrize("bad", BAD)
def test_skipped(states, bad):
    say("scalars", states, bad)
    t = state(states)
    old = {k: [x.clone() for x in v] for k, v in t.items()}
    kw = dict(lr=1e-2, step=7)
    for k, v in bad.items():
        kw[k] = torch.tensor(v, device="cuda", dtype=torch.int64 if k == "step" else torch.float32)
    tw.adamw_step(**t, **kw)
    for k in t:
        assert all(torch.equal(a, b) for a, b in zip(t[k], old[k])), k
    kw.update(lr=1e-2, step=7, norm=None)
    tw.adamw_step(**t, **kw)                         # and the next one runs
    for k in t:
        if k != "grads":
            assert not any(torch.equal(a, b) for a, b in zip(t[k], old[k])), k


@pytest.mark.parametrize("states", [32, 8])
def test_borders(states):
    """The smallest and largest values that the host takes are a step from the GPU too, and the same one."""
    for lr, step in ((0.0, 1), (1e30, 1), (1e-3, (1 << 63) - 1)):
        a, b = state(states), state(states)
        lr32 = torch.tensor(lr, device="cuda")
        if float(lr32) > 1e30:
            lr32 = torch.nextafter(lr32, torch.zeros((), device="cuda"))
        kw = dict(betas=(0.5, 0.75), weight_decay=0.0)       # their powers are exact
        tw.adamw_step(**a, lr=lr32, step=torch.tensor(step, device="cuda"), **kw)
        tw.adamw_step(**b, lr=float(lr32), step=step, **kw)
        for k in a:
            assert all(torch.equal(x, y) for x, y in zip(a[k], b[k])), (k, lr, step)


@pytest.mark.parametrize("states", [32, 8])
def test_replayed(states):
    """A captured step whose counter starts below one: the replays before it skip, the others step."""
    t, e = state(states), state(states)
    step = torch.tensor(-2, device="cuda")
    warm = state(states)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tw.adamw_step(**warm, lr=1e-2, step=step.clone())
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        tw.adamw_step(**t, lr=1e-2, step=step, betas=(0.5, 0.75))
    for k in range(-1, 4):
        graph.replay()
        if k >= 1:
            tw.adamw_step(**e, lr=1e-2, step=k, betas=(0.5, 0.75))
        torch.cuda.synchronize()
        for name in t:
            assert all(torch.equal(a, b) for a, b in zip(t[name], e[name])), (k, name)
