"""Host-side checks of the entry points around the layer (layer norm, gradient norm and
clipping): invalid arguments give the documented status before anything is enqueued. Fake device
addresses are used only in calls that fail validation (or that have nothing to enqueue)."""
import ctypes

import pytest

import activation_sparse_transformer_up_amd as tw

ARG, SHAPE, ALIGN, WS, UNSUP = -1, -2, -3, -4, -7
FAKE, MIS = 0x10000, 0x10004


def gpu_present():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


pytestmark = pytest.mark.skipif(gpu_present(), reason="fake-pointer checks run only without a GPU")


def call(name, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return getattr(tw.lib(), name)(*a.values())


NORM_F = dict(x=FAKE, ldx=64, r=None, ldr=64, w=FAKE, b=None, xt=1, T=4, d=64, eps=1e-5, y=FAKE, yt=1, s=None,
              mean=None, rstd=None, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(y=None), ARG), (dict(r=FAKE), ARG), (dict(xt=2), ARG),
    (dict(yt=-1), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(T=-1), SHAPE), (dict(d=0), SHAPE),
    (dict(d=60), ALIGN), (dict(ldx=56), SHAPE), (dict(ldx=68), ALIGN), (dict(r=FAKE, s=FAKE, ldr=0), SHAPE),
    (dict(r=FAKE, s=FAKE, ldr=65), ALIGN), (dict(x=MIS), ALIGN), (dict(b=MIS), ALIGN), (dict(r=MIS, s=FAKE), ALIGN),
    (dict(mean=MIS + 1), ALIGN), (dict(rstd=MIS + 2), ALIGN), (dict(d=16392, ldx=16392), UNSUP), (dict(T=0), 0),
    (dict(T=0, x=None, y=None), 0),
])
def test_layer_norm_fwd(kw, want):
    assert call("layer_norm_fwd", NORM_F, kw) == want


NORM_B = dict(dy=FAKE, lddy=64, dyt=0, s=FAKE, lds=64, xt=1, w=FAKE, mean=FAKE, rstd=FAKE, dres=None, lddr=64, T=40, d=64,
              dx=FAKE, dxt=1, dw=FAKE, db=None, ws=FAKE, wb=1 << 20, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), ARG), (dict(s=None), ARG), (dict(w=None), ARG), (dict(mean=None), ARG), (dict(rstd=None), ARG),
    (dict(dx=None), ARG), (dict(dw=None), ARG), (dict(dyt=2), ARG), (dict(dxt=7), ARG), (dict(T=-3), SHAPE),
    (dict(d=-8), SHAPE), (dict(d=36), ALIGN), (dict(lddy=60), SHAPE), (dict(lds=70), ALIGN),
    (dict(dres=FAKE, lddr=8), SHAPE), (dict(dres=FAKE, lddr=66), ALIGN), (dict(dx=MIS), ALIGN), (dict(dw=MIS), ALIGN),
    (dict(db=MIS), ALIGN), (dict(ws=None), WS), (dict(wb=16), WS), (dict(ws=MIS), ALIGN),
    (dict(d=16392, lddy=16392, lds=16392, wb=1 << 40), UNSUP),
])
def test_layer_norm_bwd(kw, want):
    assert call("layer_norm_bwd", NORM_B, kw) == want


def test_layer_norm_bwd_workspace():
    f = tw.lib().layer_norm_bwd_workspace_bytes
    assert f(0, 64) == 0 and f(1, 64) == 0 and f(-1, 64) == 0 and f(5, 0) == 0
    assert f(100, 64) == 100 * 2 * 64 * 4
    assert f(1 << 20, 64) == f(1 << 24, 64)          # the number of strips is bounded


def arr(t, *v):
    return (t * max(len(v), 1))(*v)


def grad(name, g=(FAKE,), sizes=(16,), types=(0,), outs=(FAKE,), otypes=(0,), n=1, max_norm=1.0, norm=FAKE, ws=FAKE,
         wb=1 << 20):
    P, L, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    args = [arr(P, *g) if g is not None else None]
    if name == "grad_clip":
        args.append(arr(P, *outs) if outs is not None else None)
    args += [arr(L, *sizes) if sizes is not None else None, arr(I, *types)]
    if name == "grad_clip":
        args.append(arr(I, *otypes))
    args.append(n)
    if name == "grad_clip":
        args.append(max_norm)
    return getattr(tw.lib(), name)(*args, norm, ws, wb, None)


@pytest.mark.parametrize("name", ["grad_norm", "grad_clip"])
@pytest.mark.parametrize("kw,want", [
    (dict(g=None), ARG), (dict(sizes=None), ARG), (dict(g=(None,)), ARG), (dict(norm=None), ARG), (dict(types=(3,)), ARG),
    (dict(n=-1), SHAPE), (dict(sizes=(-1,)), SHAPE), (dict(norm=MIS + 1), ALIGN), (dict(g=(MIS + 2,)), ALIGN),
    (dict(g=(MIS + 1,), types=(1,), otypes=(1,)), ALIGN), (dict(ws=None), WS), (dict(wb=8), WS), (dict(ws=MIS), ALIGN),
    (dict(sizes=((1 << 40) + 1,)), UNSUP),
    (dict(g=(FAKE, FAKE), outs=(FAKE, FAKE), sizes=(1 << 40, 1), types=(0, 0), otypes=(0, 0), n=2), UNSUP),
])
def test_grad_rejects(name, kw, want):
    assert grad(name, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(outs=None), ARG), (dict(outs=(None,)), ARG), (dict(max_norm=-1.0), ARG), (dict(max_norm=float("nan")), ARG),
    (dict(otypes=(4,)), ARG), (dict(otypes=(1,)), ARG), (dict(outs=(MIS + 2,)), ALIGN),
])
def test_grad_clip_rejects(kw, want):
    assert grad("grad_clip", **kw) == want


def test_grad_workspace():
    f = tw.lib().grad_norm_workspace_bytes
    assert f(0) == 0 and f(-4) == 0 and f(1) > 0 and f(64) == f(1) and f(65) == 2 * f(1)


XENT_F = dict(x=FAKE, ldx=64, w=FAKE, y=FAKE, dt=1, T=4, d=64, V=100, loss=FAKE, lse=FAKE, ws=FAKE, wb=1 << 30, stream=None)
XENT_B = dict(x=FAKE, ldx=64, w=FAKE, y=FAKE, dl=FAKE, dt=1, T=4, d=64, V=100, loss=FAKE, lse=FAKE, dx=FAKE, dw=FAKE, ws=FAKE,
              wb=1 << 30, stream=None)


@pytest.mark.parametrize("name", ["linear_xent_fwd", "linear_xent_fwd_bwd"])
@pytest.mark.parametrize("kw,want", [
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(y=None), ARG), (dict(loss=None), ARG), (dict(lse=None), ARG),
    (dict(dt=2), ARG), (dict(T=-1), SHAPE), (dict(d=0), SHAPE), (dict(V=0), SHAPE), (dict(ldx=32), SHAPE),
    (dict(d=63), ALIGN), (dict(ldx=65), ALIGN), (dict(x=MIS), ALIGN), (dict(w=MIS), ALIGN), (dict(y=MIS), ALIGN),
    (dict(loss=MIS + 1), ALIGN), (dict(ws=None), WS), (dict(wb=1000), WS), (dict(ws=MIS), ALIGN),
    (dict(V=(1 << 21) + 1), UNSUP), (dict(T=(1 << 24) + 1), UNSUP), (dict(d=(1 << 16) + 8, ldx=1 << 17), UNSUP),
])
def test_linear_xent(name, kw, want):
    assert call(name, XENT_F if name == "linear_xent_fwd" else XENT_B, kw) == want


@pytest.mark.parametrize("kw,want", [(dict(dl=None), ARG), (dict(dx=None), ARG), (dict(dw=None), ARG), (dict(dx=MIS), ALIGN),
                                     (dict(dw=MIS), ALIGN), (dict(dl=MIS + 2), ALIGN)])
def test_linear_xent_gradients(kw, want):
    assert call("linear_xent_fwd_bwd", XENT_B, kw) == want


def test_linear_xent_empty_and_workspace():
    assert call("linear_xent_fwd", XENT_F, dict(T=0, x=None, y=None, loss=None, lse=None, ws=None, wb=0)) == 0
    f = tw.lib().linear_xent_workspace_bytes
    assert f(0, 64, 100, 1, 1) == 0 and f(4, 60, 100, 1, 1) == 0 and f(4, 64, 100, 5, 1) == 0
    assert 0 < f(4, 64, 100, 1, 0) < f(4, 64, 100, 1, 1) < f(4, 64, 100, 0, 1)
    # what is kept between the launches is bounded, whatever the number of tokens: the growth past
    # the first pieces is x's copy and the row lists
    a, b = f(1 << 16, 512, 32000, 1, 1), f(1 << 20, 512, 32000, 1, 1)
    assert b - a <= ((1 << 20) - (1 << 16)) * (512 * 2 + 12) + (1 << 20)
    assert a <= (1 << 30) + 2 * 32000 * 512 * 4 + (1 << 16) * (512 * 2 + 12) + (1 << 26)
