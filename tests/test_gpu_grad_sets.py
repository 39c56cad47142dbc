"""Gradient norm and clipping of sets large enough that workgroups take several chunks (more than 2048
chunks of 16384 elements in a table of 64 tensors), in place and out of place, and of more than one
such table. Bounds as for small sets."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402
from test_gpu_grad import BF16, F32, check_norm, check_out  # noqa: E402


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


SETS = {
    "few large": [20_000_003, 7_777_777, 9, 0, 15_000_001, 2048 * 16384 // 3],
    "two tables": [600_011 + 7 * i for i in range(75)],
    "small after large": [36_000_000] + [33 * i for i in range(1, 140)],
}


def make(name, types, offset):
    g = torch.Generator(device="cuda").manual_seed(len(name))
    return [(torch.randn(n + offset, generator=g, device="cuda") * 10.0 ** (-i % 3)).to(types[i % len(types)])[offset:]
            for i, n in enumerate(SETS[name])]


@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("types", [(F32,), (BF16,), (F32, BF16)])
@pytest.mark.parametrize("offset", [0, 3])
def test_several_chunks_per_workgroup(name, types, offset):
    say("grad sets", name, types, offset)
    grads = make(name, types, offset)
    ref = check_norm(tw.grad_norm(grads), grads)
    before = [g.clone() for g in grads]
    limit = 0.37 * ref
    out = [torch.full(g.shape, 7.0, dtype=types[-1], device="cuda") for g in grads]
    norm, got = tw.grad_clip(grads, limit, out=out)
    check_norm(norm, grads)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    check_out(got, grads, limit / (ref + 1e-6))
    norm2, same = tw.grad_clip(grads, 2 * ref)              # below the limit: nothing changes
    assert torch.equal(norm2, norm) and all(torch.equal(a, b) for a, b in zip(same, before))
    norm2, same = tw.grad_clip(grads, limit)                # in place
    assert torch.equal(norm2, norm)
    check_out(same, before, limit / (ref + 1e-6))
    if types[-1] == types[0]:
        assert all(torch.equal(a, b) for a, b in zip(same, out))


def test_a_tensor_listed_twice():
    """Clipped in place it is refused and stays as it is; read twice it counts twice."""
    g = torch.full((5000,), 3.0, device="cuda")
    with pytest.raises(tw.TwellError):
        tw.grad_clip([g, g], 1.0)
    with pytest.raises(tw.TwellError):
        tw.grad_clip([g, g[:100]], 1.0)
    assert (g == 3.0).all()
    check_norm(tw.grad_norm([g, g]), [g, g])
    out = [torch.empty_like(g), torch.empty_like(g)]
    tw.grad_clip([g, g], 1.0, out=out)
    check_out(out, [g, g], 1.0 / (3.0 * 10000 ** 0.5 + 1e-6))
