"""GPU parity of the global gradient norm and clipping against 64-bit sums. The norm is summed in
fp64 and rounded once (E = 2^-24; the fp64 sum's own error is below 2^-40 of it); the factor
takes three more fp32 roundings, the product one, the output type its own."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402

E = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def tensors(seed, sizes, types, scale=1.0, offset=0):
    """One gradient per size, `offset` elements into its allocation."""
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n + offset, generator=g) * scale).to(types[i % len(types)]).cuda()[offset:]
            for i, n in enumerate(sizes)]


def norm64(grads):
    return float(sum(g.double().square().sum().cpu() for g in grads)) ** 0.5


def check_norm(norm, grads):
    ref = norm64(grads)
    assert abs(float(norm) - ref) <= 1.01 * E * ref, (float(norm), ref)
    return ref


def check_out(out, grads, c):
    for o, g in zip(out, grads):
        ref = g.double() * c
        tol = 5 * E * ref.abs()
        # an fp32 product below the normal range is off by half its smallest step
        tol = tol + HALF[o.dtype] * (ref.abs() + tol) + 2.0 ** -149
        assert ((o.double() - ref).abs() <= tol).all()


SETS = {
    "one": [1], "odd": [1, 3, 7, 8, 9, 2047, 2048, 2049, 4096 * 3 + 5], "empty_between": [5, 0, 0, 17, 0],
    "many": [i * 37 % 501 for i in range(131)], "large": [3_000_001, 64, 5_000_000],
}


@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("types", [(F32,), (BF16,), (F32, BF16)])
@pytest.mark.parametrize("offset", [0, 1])
def test_norm_and_clip(name, types, offset):
    say("grad", name, types, offset)
    grads = tensors(len(name), SETS[name], types, offset=offset)
    ref = check_norm(tw.grad_norm(grads), grads)
    assert torch.equal(tw.grad_norm(grads), tw.grad_norm(grads))
    before = [g.clone() for g in grads]
    limit = 0.37 * ref
    out = [torch.empty(g.shape, dtype=types[-1], device="cuda") for g in grads]
    norm, got = tw.grad_clip(grads, limit, out=out)
    assert all(a is b for a, b in zip(got, out)) and all(torch.equal(a, b) for a, b in zip(grads, before))
    check_norm(norm, grads)
    check_out(out, grads, limit / (ref + 1e-6))
    norm2, same = tw.grad_clip(grads, limit)                 # in place
    assert float(norm2) == float(norm) and all(a is b for a, b in zip(same, grads))
    check_out(grads, before, limit / (ref + 1e-6))


def test_below_the_limit_nothing_changes():
    grads = tensors(3, [1000, 33], (F32, BF16))
    before = [g.clone() for g in grads]
    out = [torch.empty_like(g) for g in grads]
    tw.grad_clip(grads, 1e9, out=out)
    tw.grad_clip(grads, float("inf"))
    for g, b, o in zip(grads, before, out):
        assert torch.equal(g, b) and torch.equal(o, b)


@pytest.mark.parametrize("scale", [1e30, 1e-30])
def test_squares_beyond_fp32(scale):
    grads = tensors(4, [5000, 77], (F32, BF16), scale=scale)
    check_norm(tw.grad_norm(grads), grads)


def test_zero_and_empty():
    z = [torch.zeros(100).cuda(), torch.zeros(0).cuda()]
    norm, out = tw.grad_clip(z, 1.0)
    assert float(norm) == 0.0 and not out[0].any()
    assert float(tw.grad_norm([])) == 0.0
    assert float(tw.grad_clip([], 1.0)[0]) == 0.0
    assert float(tw.grad_norm([z[1]])) == 0.0
    g = tensors(5, [300], (F32,))
    tw.grad_clip(g, 0.0)
    assert not g[0].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nonfinite(dtype):
    g = tensors(6, [300, 5], (dtype,))
    g[0][7] = float("inf")
    norm, out = tw.grad_clip(g, 1.0, out=[torch.empty_like(t) for t in g])
    assert float(norm) == float("inf")
    assert torch.isnan(out[0][7].float()) and not out[1].any()
    g[1][2] = float("nan")
    norm, out = tw.grad_clip(g, 1.0, out=out)
    assert torch.isnan(norm) and all(torch.isnan(o.float()).all() for o in out)


def test_python_refusals():
    g = [torch.ones(8).cuda()]
    with pytest.raises(TypeError):
        tw.grad_norm([torch.ones(8, dtype=torch.float16).cuda()])
    with pytest.raises(ValueError):
        tw.grad_norm([torch.ones(8, 8).cuda().t()])
    with pytest.raises(ValueError):
        tw.grad_norm([torch.ones(8), g[0]], norm=torch.zeros(()).cuda())
    with pytest.raises(ValueError):
        tw.grad_clip(g, 1.0, out=[torch.ones(9).cuda()])
    with pytest.raises(tw.TwellError):
        tw.grad_clip(g, -1.0)
    with pytest.raises(tw.TwellError):
        tw.grad_clip(g, float("nan"))
    with pytest.raises(tw.TwellError):
        tw.grad_norm(g, workspace=torch.empty(16, dtype=torch.uint8).cuda())


def test_graph_and_side_stream():
    grads = tensors(8, [70000, 3, 4097], (F32, BF16))
    out = [torch.empty_like(g) for g in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        n0, o0 = tw.grad_clip(grads, 1.0, out=[torch.empty_like(g) for g in grads])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm, _ = tw.grad_clip(grads, 1.0, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, n0) and all(torch.equal(a, b) for a, b in zip(out, o0))
    for k in range(3):
        for g in grads:
            g.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        n1, o1 = tw.grad_clip(grads, 1.0, out=[torch.empty_like(g) for g in grads])
        assert torch.equal(norm, n1) and all(torch.equal(a, b) for a, b in zip(out, o1))
