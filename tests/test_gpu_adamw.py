"""GPU parity of the AdamW step against its formulas in 64 bits, states in 32 and in 8 bits. With E = 2^-24, and
the factors beta, 1 - beta, eps, max_norm / norm rounded to fp32 (E each):
  g'   2 E |g'| with a norm (c: its quotient's rounding and its own, 4 E)          -> 6 E |g'|
  m    each product 2 E, the sum 1 E:  em = 4 E (|b1 m| + |(1 - b1) g'|) + (1 - b1) 6 E |g'|
  v    ev = 6 E (b2 v + (1 - b2) g'^2) + 12 E (1 - b2) g'^2
  d    m / (sqrt(v) r + eps): em / denominator, and |d| (ev / (2 v) + 8 E)
  p    4 E (|p| + rate |d|) + rate dd
An 8-bit state is within half a step of its code, in the root: with q the code and y = sqrt(|m| / s)
(v: its fourth root), |y - q| <= 1/2 (1 + 2^-12), 2^-12 for y's own error (below 8 E y and the state's error),
but a v above zero may have q = 1 for any y below 1.5; the scale is the largest state / 127^2 (255^4) within 8 E and
that state's error, at least 2^-126."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import activation_sparse_transformer_up_amd as tw  # noqa: E402

E = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
HYPER = dict(lr=1e-2, betas=(0.9, 0.97), eps=1e-8)


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def tensors(seed, sizes, p_dtype=F32, g_dtype=F32, offset=0, scale=1.0):
    """Parameters, gradients and states; `offset` elements off a 16-byte border."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(n, dtype, f):
        t = torch.empty(n + offset, dtype=dtype, device="cuda")[offset:]
        t.copy_(f(torch.randn(n, generator=g, device="cuda")))
        return t
    sizes = [s if isinstance(s, int) else s for s in sizes]
    size = [scale * 10.0 ** -(k % 4) for k in range(len(sizes))]
    return dict(params=[make(n, p_dtype, lambda r: r) for n in sizes], grads=[make(n, g_dtype, lambda r: r * s) for n, s in zip(sizes, size)],
                m=[make(n, F32, lambda r: 0.3 * s * r) for n, s in zip(sizes, size)],
                v=[make(n, F32, lambda r: (s * r) ** 2) for n, s in zip(sizes, size)])


def to_codes(t, offset=0):
    """The tensors with their states as codes of random values."""
    out = dict(t, m=[], v=[], m_scales=[], v_scales=[])
    for k, p in enumerate(t["params"]):
        g = torch.Generator(device="cuda").manual_seed(k)
        blocks = (p.numel() + 255) // 256
        qm = torch.randint(-127, 128, (p.numel() + offset,), generator=g, device="cuda").to(torch.int8)[offset:]
        qv = torch.randint(0, 256, (p.numel() + offset,), generator=g, device="cuda").to(torch.uint8)[offset:]
        qm[::17] = 0
        qv[::17] = 0
        out["m"].append(qm)
        out["v"].append(qv)
        out["m_scales"].append(1e-5 * (0.5 + torch.rand(blocks, generator=g, device="cuda")))
        out["v_scales"].append(1e-10 * (0.5 + torch.rand(blocks, generator=g, device="cuda")))
    return out


def values64(q, s):
    each = s.double().repeat_interleave(256)[:q.numel()].view(q.shape)
    c = q.double()
    return (c * c.abs() if q.dtype == torch.int8 else c ** 4) * each


def check_state(q, s, want, err):
    """Codes and scales against the state that they round, known within err."""
    power, top = (2, 127) if q.dtype == torch.int8 else (4, 255)
    n, pad = q.numel(), -q.numel() % 256
    w, e = (torch.nn.functional.pad(t.reshape(-1), (0, pad)).view(-1, 256) for t in (want, err))
    k = torch.nn.functional.pad(q.double().reshape(-1), (0, pad)).view(-1, 256)
    big = w.abs().amax(1) / top ** power
    assert ((s.double() - big.clamp(min=2.0 ** -126)).abs() <= 8 * E * s.double() + e.amax(1) / top ** power).all()
    s = s.double()[:, None]
    hi, lo = ((w.abs() + e) / s) ** (1 / power), ((w.abs() - e).clamp(min=0) / s) ** (1 / power)
    a = k.abs()
    slack = 0.5 + 2.0 ** -12
    ok = (a <= hi + slack) & (a >= lo - slack)
    if power == 4:
        ok |= (a == 1) & (lo <= 1.5) & (w + e > 0)
        assert ((a > 0) | (w - e <= 0)).all()
    ok |= torch.arange(k.numel(), device="cuda").view_as(k) >= n
    assert ok.all(), int((~ok).sum())
    assert ((torch.sign(k) * torch.sign(w) >= 0) | (w.abs() <= e)).all()


def run(t, step=7, wd=0.1, norm=None, max_norm=1.0, copies=False, **hyper):
    """One step, checked."""
    h = dict(HYPER, **hyper)
    eight = "m_scales" in t
    wds = wd if isinstance(wd, list) else [wd] * len(t["params"])
    old = {k: [x.clone() for x in v] for k, v in t.items()}
    cps = [torch.empty_like(p, dtype=BF16) for p in t["params"]] if copies else None
    tw.adamw_step(**t, step=step, weight_decay=wd, norm=norm, max_norm=max_norm, copies=cps, **h)
    (b1, b2), lr, eps = h["betas"], h["lr"], h["eps"]
    c, ec = 1.0, 0.0
    if norm is not None:
        c, ec = min(1.0, max_norm / (float(norm) + 1e-6)), 6 * E
    rate, root = lr / (1 - b1 ** step), (1 - b2 ** step) ** -0.5
    for k in range(len(t["params"])):
        p, g = old["params"][k].double(), old["grads"][k].double() * c
        assert torch.equal(t["grads"][k], old["grads"][k])
        if eight:
            m, v = values64(old["m"][k], old["m_scales"][k]), values64(old["v"][k], old["v_scales"][k])
        else:
            m, v = old["m"][k].double(), old["v"][k].double()
        em = 4 * E * (b1 * m.abs() + (1 - b1) * g.abs()) + (1 - b1) * ec * g.abs()
        ev = 6 * E * (b2 * v + (1 - b2) * g * g) + 2 * ec * (1 - b2) * g * g
        if eight:                                    # the old values' own products: 2 and 3 roundings
            em, ev = em + 2 * E * b1 * m.abs(), ev + 4 * E * b2 * v
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        den = v.sqrt() * root + eps
        d = m / den
        ed = em / den + d.abs() * (ev / (2 * v + 1e-300) + 8 * E)
        want = p * (1 - lr * wds[k]) - rate * d
        tol = 4 * E * (p.abs() + rate * d.abs()) + rate * ed + 1e-37
        half = torch.finfo(t["params"][k].dtype).eps / 2
        got = t["params"][k].double()
        assert ((got - want).abs() <= tol + half * (want.abs() + tol)).all(), k
        if copies:
            assert torch.equal(cps[k], t["params"][k].to(BF16)), k
        if eight:
            check_state(t["m"][k], t["m_scales"][k], m, em + 1e-37)
            check_state(t["v"][k], t["v_scales"][k], v, ev + 1e-37)
        else:
            assert ((t["m"][k].double() - m).abs() <= em + 1e-37).all(), k
            assert ((t["v"][k].double() - v).abs() <= ev + 1e-37).all(), k


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 5000, 0, 16384 * 3 + 5, 300001]


@pytest.mark.parametrize("states", [32, 8])
@pytest.mark.parametrize("p_dtype,g_dtype", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("offset", [0, 1])
def test_step(states, p_dtype, g_dtype, offset):
    say("adamw", states, p_dtype, g_dtype, offset)
    t = tensors(1, SIZES, p_dtype, g_dtype, offset)
    if states == 8:
        t = to_codes(t, offset)
    run(t, copies=p_dtype == F32)
    run(t, step=8, wd=[0.01 * k for k in range(len(SIZES))])          # from the states that the first left


@pytest.mark.parametrize("states", [32, 8])
@pytest.mark.parametrize("norm,max_norm", [(10.0, 1.0), (0.5, 1.0), (3.0, 0.0), (0.0, 1.0), (1e30, 1e-3)])
def test_clipped(states, norm, max_norm):
    t = tensors(2, [1000, 3000])
    run(to_codes(t) if states == 8 else t, norm=torch.tensor(norm, device="cuda"), max_norm=max_norm)


@pytest.mark.parametrize("states", [32, 8])
@pytest.mark.parametrize("step,hyper", [(1, {}), (2, dict(betas=(0.0, 0.0))), (100000, dict(betas=(0.99, 0.9999))), (3, dict(lr=0.0)),
                                        (5, dict(eps=1e-3)), (1 << 40, {}),
                                        (4, dict(eps=1e-20)), (4, dict(eps=1.2e-38))])
def test_hyper(states, step, hyper):
    t = tensors(3, [700, 4100])
    run(to_codes(t) if states == 8 else t, step=step, wd=0.0, **hyper)


@pytest.mark.parametrize("states", [32, 8])
def test_more_tensors_than_a_launch_takes(states):
    t = tensors(4, [(37 * k) % 900 for k in range(95)])
    run(to_codes(t) if states == 8 else t, copies=True)


def test_some_copies():
    """A copy of every other param; the same step as without them."""
    t = tensors(12, [300, 4097, 8, 2048])
    e = {k: [x.clone() for x in v] for k, v in t.items()}
    copies = [torch.zeros_like(p, dtype=BF16) if k % 2 else None for k, p in enumerate(t["params"])]
    tw.adamw_step(**t, step=2, copies=copies, **HYPER)
    tw.adamw_step(**e, step=2, **HYPER)
    for a, b, c in zip(t["params"], e["params"], copies):
        assert torch.equal(a, b) and (c is None or torch.equal(c, a.to(BF16)))
    with pytest.raises(ValueError):
        tw.adamw_step(**t, step=2, copies=copies[:2], **HYPER)


@pytest.mark.parametrize("states", [32, 8])
def test_chunks_per_workgroup(states):
    """More chunks than workgroups, of the largest size."""
    t = tensors(5, [40_000_003, 999])
    run(to_codes(t) if states == 8 else t)


def test_first_steps_from_zero_states():
    """8-bit states from nothing: over ten steps the parameters stay within 3% of the 32-bit run's way in the norm
    (a state's relative error is at most 1 / (2 q) of its root, q near the top code for most of a block of
    one spread, and averages out)."""
    t = tensors(6, [4096, 1000])
    a = dict(t, m=[torch.zeros_like(p) for p in t["params"]], v=[torch.zeros_like(p) for p in t["params"]],
             params=[p.clone() for p in t["params"]])
    st = [tw.adamw8_states(p) for p in t["params"]]
    b = dict(grads=t["grads"], params=[p.clone() for p in t["params"]], m=[s[0] for s in st], m_scales=[s[1] for s in st],
             v=[s[2] for s in st], v_scales=[s[3] for s in st])
    g = torch.Generator(device="cuda").manual_seed(9)
    for step in range(1, 11):
        for x in t["grads"]:
            x.copy_(0.1 * torch.randn(x.shape, generator=g, device="cuda"))
        for s in (a, b):
            tw.adamw_step(**s, step=step, weight_decay=0.0, **HYPER)
    for p0, p1, p2 in zip(t["params"], a["params"], b["params"]):
        assert (p1 - p2).norm() <= 0.03 * (p1 - p0).norm()


def test_small_and_uneven_blocks():
    """Blocks of zeros, of values that underflow, with one value far above the rest, and of the largest values."""
    for size in (0.0, 1e-30, 1e-18, 1e15):
        t = tensors(7, [1024], scale=size)
        st = tw.adamw8_states(t["params"][0])
        t.update(m=[st[0]], m_scales=[st[1]], v=[st[2]], v_scales=[st[3]])
        t["grads"][0][300] *= 1e3
        say("blocks", size)
        run(t, step=1)
        m, v = tw.adamw8_values(t["m"] + t["v"], t["m_scales"] + t["v_scales"])
        assert torch.isfinite(m).all() and torch.isfinite(v).all() and torch.isfinite(t["params"][0]).all()
        if size >= 1e-18:
            assert (v[t["grads"][0] != 0] > 0).all()


@pytest.mark.parametrize("states", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite(states, bad):
    t = tensors(8, [1000, 600])
    t = to_codes(t) if states == 8 else t
    old = {k: [x.clone() for x in v] for k, v in t.items()}
    t["grads"][0][300] = bad
    norm = tw.grad_norm(t["grads"])
    copies = [torch.full_like(p, 5.0, dtype=BF16) for p in t["params"]]
    tw.adamw_step(**t, step=3, norm=norm, copies=copies, **HYPER)       # skipped
    for k in t:
        if k != "grads":
            assert all(torch.equal(a, b) for a, b in zip(t[k], old[k])), k
    assert all((c == 5.0).all() for c in copies)
    tw.adamw_step(**t, step=3, **HYPER)                                 # reaches its element, and its block's states
    fine = torch.isfinite(t["params"][0])
    assert not fine[300] and fine.sum() == 999 and torch.isfinite(t["params"][1]).all()
    if states == 8:
        m = tw.adamw8_values(t["m"], t["m_scales"])
        ok = torch.isfinite(m[0])
        assert ok[:256].all() and not ok[300] and ok[512:].all() and torch.isfinite(m[1]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset", [0, 3])
def test_values(dtype, offset):
    t = to_codes(tensors(9, SIZES), offset)
    codes = t["m"] + t["v"]
    got = tw.adamw8_values(codes, t["m_scales"] + t["v_scales"], dtype=dtype)
    for q, s, v in zip(codes, t["m_scales"] + t["v_scales"], got):
        want = values64(q, s)
        assert v.shape == q.shape and v.dtype == dtype
        assert ((v.double() - want).abs() <= (3 * E + torch.finfo(dtype).eps / 2 * (1 + 3 * E)) * want.abs()).all()
    assert tw.adamw8_values([], []) == []


@pytest.mark.parametrize("states", [32, 8])
def test_captured_with_scalars_on_the_gpu(states):
    """A captured step with its clipping, replayed while lr and step change; against eager steps with host
    scalars, whose factors are rounded from the same 64-bit values up to one last bit (then 2 E of the step)."""
    t = tensors(10, [5000, 33, 4096])
    t = to_codes(t) if states == 8 else t
    e = {k: [x.clone() for x in v] for k, v in t.items()}
    lr, step = torch.tensor(0.0, device="cuda"), torch.zeros((), dtype=torch.int64, device="cuda")
    norm = torch.zeros((), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kw = dict(betas=(0.9, 0.97), eps=1e-8, weight_decay=0.1, max_norm=5.0)
    empty = {k: [x.clone() for x in v] for k, v in t.items()}
    with torch.cuda.stream(s):
        tw.grad_norm(empty["grads"], norm=norm)
        tw.adamw_step(**empty, lr=lr, step=step + 1, norm=norm, **kw)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        tw.grad_norm(t["grads"], norm=norm)
        tw.adamw_step(**t, lr=lr, step=step, norm=norm, **kw)
    g = torch.Generator(device="cuda").manual_seed(3)
    for k in range(1, 6):
        for a, b in zip(t["grads"], e["grads"]):
            a.copy_(torch.randn(a.shape, generator=g, device="cuda"))
            b.copy_(a)
        lr.fill_(0.25 / k)
        eager = tw.grad_norm(e["grads"])
        tw.adamw_step(**e, lr=float(lr), step=k, norm=eager, **kw)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(step) == k and float(norm) == float(eager)
        for a, b in zip(t["params"], e["params"]):
            assert ((a - b).abs() <= 8 * E * (b.abs() + 10 * 0.25)).all(), k
        for name in ("m", "v", "m_scales", "v_scales"):
            assert all(torch.equal(a, b) for a, b in zip(t.get(name, []), e.get(name, []))), (k, name)


def test_same_bits():
    for states in (32, 8):
        a = tensors(11, [9000, 100])
        a = to_codes(a) if states == 8 else a
        b = {k: [x.clone() for x in v] for k, v in a.items()}
        for t in (a, b):
            tw.adamw_step(**t, step=4, **HYPER)
        for k in a:
            assert all(torch.equal(x, y) for x, y in zip(a[k], b[k]))


def test_guard_zones():
    """Ragged sizes in one buffer each, tensors side by side: neighbours and the buffers' ends keep their bytes."""
    for states in (32, 8):
        n = [257, 1, 2051]
        kinds = dict(params=F32, grads=F32, m=F32, v=F32) if states == 32 else dict(params=F32, grads=F32, m=torch.int8, v=torch.uint8,
                                                                                       m_scales=F32, v_scales=F32)
        bufs, t = {}, {}
        for k, dt in kinds.items():
            sizes = [(x + 255) // 256 for x in n] if k.endswith("scales") else n
            bufs[k] = torch.full((sum(sizes) + 64 * 4,), 3, dtype=dt, device="cuda")
            at = 64
            t[k] = []
            for x in sizes:
                t[k].append(bufs[k][at:at + x])
                at += x + 64
        tw.adamw_step(**t, step=1, **HYPER)
        for k, b in bufs.items():
            inside = torch.zeros(b.shape, dtype=torch.bool, device="cuda")
            at = 64
            for x in t[k]:
                inside[at:at + x.numel()] = True
                at += x.numel() + 64
            assert (b[~inside] == 3).all(), k


def test_python_refusals_on_gpu():
    p, g, m, v = ([torch.ones(300, device="cuda") * k] for k in range(4))
    ok = dict(params=p, grads=g, m=m, v=v, lr=1e-3, step=1)
    st = tw.adamw8_states(p[0])
    for kw, err in ((dict(grads=[g[0][:299]]), ValueError), (dict(grads=[]), ValueError), (dict(weight_decay=[0.1, 0.1]), ValueError),
                    (dict(v=[v[0].int()]), TypeError), (dict(m_scales=[st[1]]), ValueError), (dict(grads=[g[0].half()]), TypeError), (dict(m=[m[0].bfloat16()]), TypeError),
                    (dict(m=[m[0].cpu()]), ValueError), (dict(params=[torch.ones(20, 15, device="cuda").t()]), ValueError),
                    (dict(m=[st[0]], v=[st[2]], m_scales=[st[1]]), ValueError), (dict(m_scales=[st[1]], v_scales=[st[3]]), TypeError),
                    (dict(m=[st[0]], v=[st[2]], m_scales=[st[1]], v_scales=[st[3][:1]]), ValueError),
                    (dict(copies=[p[0].clone()]), TypeError), (dict(norm=1.0), TypeError), (dict(norm=torch.ones(2, device="cuda")), TypeError),
                    (dict(step=torch.ones((), device="cuda")), TypeError), (dict(lr=torch.ones(())), ValueError),
                    (dict(lr=-1.0), tw.TwellError), (dict(step=0), tw.TwellError), (dict(params=p + p, grads=g + g, m=m + m, v=v + v), tw.TwellError),
                    (dict(m=v), tw.TwellError), (dict(grads=p), tw.TwellError)):
        with pytest.raises(err):
            tw.adamw_step(**dict(ok, **kw))
    tw.adamw_step([], [], [], [], 1e-3, 1)


def test_many_elements():
    """A tensor of more than 2^31 elements: its first, last and some middle blocks."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB of free GPU memory")
    n = (1 << 31) + 300001
    say("adamw far", n)
    p, g = torch.zeros(n, dtype=BF16, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")
    st = tw.adamw8_states(p)
    at = [0, 255, 256, (1 << 30) + 5, (1 << 31) - 1, 1 << 31, (1 << 31) + 256, n - 1]
    for k, i in enumerate(at):
        g[i] = 1.0 + k
    tw.adamw_step([p], [g], [st[0]], [st[2]], lr=0.5, step=1, weight_decay=0.0, m_scales=[st[1]], v_scales=[st[3]])
    for i in at:                                     # the first step is lr in the gradient's direction
        assert abs(float(p[i]) + 0.5) <= 0.5 * 2.0 ** -8 + 1e-6 and int(st[0][i]) > 0 and int(st[2][i]) > 0, i
    assert int(p.count_nonzero()) == len(at) and int(st[0].count_nonzero()) == len(at)
