"""Host-side checks of the dense layers and of AdamW: invalid arguments give the documented status before
anything is enqueued, workspaces stay within the header's bound. Fake device addresses are used only in
calls that fail validation (or that have nothing to enqueue)."""
import ctypes
import random

import pytest

import activation_sparse_transformer_up_amd as tw
from test_step_host import ALIGN, ARG, FAKE, MIS, SHAPE, UNSUP, WS, call, gpu_present

pytestmark = pytest.mark.skipif(gpu_present(), reason="fake-pointer checks run only without a GPU")

NAN, INF = float("nan"), float("inf")

LIN_F = dict(x=FAKE, ldx=64, w=FAKE, lay=0, b=None, r=None, ldr=128, dt=1, T=4, K=64, N=128, act=0, y=FAKE, yt=1, pre=None,
             ws=FAKE, wb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(y=None), ARG), (dict(lay=2), ARG), (dict(lay=-1), ARG),
    (dict(dt=2), ARG), (dict(yt=-1), ARG), (dict(act=5), ARG), (dict(act=-1), ARG), (dict(T=-1), SHAPE), (dict(K=0), SHAPE),
    (dict(N=-8), SHAPE), (dict(K=60), ALIGN), (dict(N=100), ALIGN), (dict(ldx=56), SHAPE), (dict(ldx=68), ALIGN),
    (dict(r=FAKE, ldr=8), SHAPE), (dict(r=FAKE, ldr=129), ALIGN), (dict(x=MIS), ALIGN), (dict(w=MIS), ALIGN),
    (dict(b=MIS), ALIGN), (dict(r=MIS), ALIGN), (dict(y=MIS), ALIGN), (dict(pre=MIS), ALIGN),
    (dict(T=(1 << 24) + 1), UNSUP), (dict(K=(1 << 20) + 8, ldx=1 << 21), UNSUP), (dict(N=(1 << 20) + 8), UNSUP),
    (dict(ldx=(1 << 21) + 8), UNSUP), (dict(r=FAKE, ldr=1 << 40), UNSUP),
    (dict(K=4096, ldx=4096, ws=None, wb=0), WS), (dict(K=4096, ldx=4096, wb=8), WS), (dict(K=4096, ldx=4096, ws=MIS), ALIGN),
    (dict(T=0), 0), (dict(T=0, x=None, y=None, ws=None, wb=0), 0),
])
def test_linear_fwd(kw, want):
    assert call("linear_fwd", LIN_F, kw) == want


LIN_B = dict(dy=FAKE, lddy=128, x=FAKE, ldx=64, w=FAKE, lay=0, pre=FAKE, dt=1, T=4, K=64, N=128, act=2, dx=FAKE, dw=FAKE, db=FAKE,
             ws=FAKE, wb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), ARG), (dict(x=None), ARG), (dict(w=None), ARG), (dict(pre=None), ARG), (dict(lay=2), ARG), (dict(dt=3), ARG),
    (dict(act=9), ARG), (dict(T=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE), (dict(K=4), ALIGN), (dict(N=12), ALIGN),
    (dict(lddy=120), SHAPE), (dict(lddy=130), ALIGN), (dict(ldx=8), SHAPE), (dict(ldx=65), ALIGN), (dict(dy=MIS), ALIGN),
    (dict(x=MIS), ALIGN), (dict(w=MIS), ALIGN), (dict(pre=MIS), ALIGN), (dict(dx=MIS), ALIGN), (dict(dw=MIS), ALIGN),
    (dict(db=MIS), ALIGN), (dict(ws=None), WS), (dict(wb=16), WS), (dict(ws=MIS), ALIGN), (dict(T=(1 << 24) + 1), UNSUP),
    (dict(K=(1 << 20) + 8, ldx=1 << 21), UNSUP), (dict(lddy=(1 << 21) + 8), UNSUP), (dict(ldx=(1 << 21) + 8), UNSUP),
    # what is not needed is not looked at
    (dict(dx=None, w=MIS, wb=0), WS), (dict(dw=None, x=MIS, wb=0), WS), (dict(act=0, pre=MIS, wb=0), WS),
    # nothing wanted: nothing is read or written
    (dict(dx=None, dw=None, db=None, ws=None, wb=0), 0), (dict(dx=None, dw=None, db=None, dy=None, x=None, w=None, pre=None), 0),
])
def test_linear_bwd(kw, want):
    assert call("linear_bwd", LIN_B, kw) == want


GATE_F = dict(x=FAKE, ldx=64, wg=FAKE, wu=FAKE, w2=FAKE, bg=None, bu=None, r=None, ldr=64, dt=1, T=4, d=64, f=128, act=2, y=FAKE,
              yt=1, g=None, u=None, ws=FAKE, wb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), ARG), (dict(wg=None), ARG), (dict(wu=None), ARG), (dict(w2=None), ARG), (dict(y=None), ARG),
    (dict(g=FAKE), ARG), (dict(u=FAKE), ARG), (dict(dt=2), ARG), (dict(yt=2), ARG), (dict(act=5), ARG), (dict(T=-1), SHAPE),
    (dict(d=0), SHAPE), (dict(f=0), SHAPE), (dict(d=60), ALIGN), (dict(f=100), ALIGN), (dict(ldx=56), SHAPE),
    (dict(ldx=66), ALIGN), (dict(r=FAKE, ldr=8), SHAPE), (dict(r=FAKE, ldr=68), ALIGN), (dict(x=MIS), ALIGN),
    (dict(wg=MIS), ALIGN), (dict(wu=MIS), ALIGN), (dict(w2=MIS), ALIGN), (dict(bg=MIS), ALIGN), (dict(bu=MIS), ALIGN),
    (dict(r=MIS), ALIGN), (dict(y=MIS), ALIGN), (dict(g=MIS, u=FAKE), ALIGN), (dict(g=FAKE, u=MIS), ALIGN), (dict(ws=None), WS),
    (dict(wb=100), WS), (dict(ws=MIS), ALIGN), (dict(T=(1 << 24) + 1), UNSUP), (dict(f=(1 << 20) + 8), UNSUP), (dict(T=0), 0),
])
def test_gated_fwd(kw, want):
    assert call("ffn_gated_dense_fwd", GATE_F, kw) == want


GATE_B = dict(dy=FAKE, lddy=64, x=FAKE, ldx=64, wg=FAKE, wu=FAKE, w2=FAKE, g=FAKE, u=FAKE, dt=1, T=4, d=64, f=128, act=2, dx=FAKE,
              dwg=FAKE, dwu=FAKE, dw2=FAKE, dbg=None, dbu=None, ws=FAKE, wb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,want", [(dict([(k, None)]), ARG) for k in ("dy", "x", "wg", "wu", "w2", "g", "u", "dx", "dwg", "dwu", "dw2")] +
                         [(dict([(k, MIS)]), ALIGN) for k in ("dy", "x", "wg", "wu", "w2", "g", "u", "dx", "dwg", "dwu", "dw2",
                                                             "dbg", "dbu", "ws")] +
                         [(dict(dt=2), ARG), (dict(act=7), ARG), (dict(T=-1), SHAPE), (dict(d=-8), SHAPE), (dict(f=20), ALIGN),
                          (dict(lddy=8), SHAPE), (dict(lddy=65), ALIGN), (dict(ldx=8), SHAPE), (dict(ldx=65), ALIGN),
                          (dict(ws=None), WS), (dict(wb=4), WS), (dict(d=(1 << 20) + 8, ldx=1 << 21, lddy=1 << 21), UNSUP)])
def test_gated_bwd(kw, want):
    assert call("ffn_gated_dense_bwd", GATE_B, kw) == want


def test_workspaces():
    """What the header says they hold: operands of the next product, at most 256 MB of partial sums, the planes
    of one product's fp32 operands, the column sums' blocks."""
    L, rng = tw.lib(), random.Random(3)
    assert L.linear_fwd_workspace_bytes(0, 64, 64, 1, 0) == 0 and L.linear_fwd_workspace_bytes(4, 60, 64, 1, 0) == 0
    assert L.linear_fwd_workspace_bytes(4, 64, 64, 1, 2) == 0 and L.linear_bwd_workspace_bytes(4, 64, 64, 1, 0, 9, 1, 1, 1) == 0
    assert L.ffn_gated_dense_fwd_workspace_bytes(4, 64, 64, 3) == 0 and L.ffn_gated_dense_bwd_workspace_bytes(-1, 64, 64, 1, 0) == 0
    for _ in range(2000):
        T, K, N = int(2 ** rng.uniform(0, 24)), 8 * int(2 ** rng.uniform(0, 17)), 8 * int(2 ** rng.uniform(0, 17))
        dt, lay, act = rng.randint(0, 1), rng.randint(0, 1), rng.randint(0, 4)
        n = T * N * (2 if dt else 4)
        cap = (256 << 20) + 8192 + (0 if dt else 6 * (T * (K + N) + 2 * K * N))
        assert L.linear_fwd_workspace_bytes(T, K, N, dt, lay) <= cap
        assert L.linear_bwd_workspace_bytes(T, K, N, dt, lay, act, 1, 1, 0) <= n * (act > 0) + cap
        sums = (T // 16 + 1024) * N * 4
        assert L.linear_bwd_workspace_bytes(T, K, N, dt, lay, act, 0, 0, 1) <= sums
        cap += 0 if dt else 6 * 3 * (T * (K + N) + K * N)
        assert n <= L.ffn_gated_dense_fwd_workspace_bytes(T, K, N, dt) <= n + cap
        assert 3 * n <= L.ffn_gated_dense_bwd_workspace_bytes(T, K, N, dt, 0) <= 3 * n + cap
        assert L.ffn_gated_dense_bwd_workspace_bytes(T, K, N, dt, 1) <= 3 * n + cap + 2 * sums


# ------------------------------------------------------------------------------------- AdamW

P, I64, I32, F64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double
A, B, C, D, E, F, G = (0x100000 * k for k in range(1, 8))


def adamw(p=(A,), g=(B,), m=(C,), v=(D,), ms=None, vs=None, copies=None, sizes=(16,), dt=(0,), gt=(0,), wd=(0.0,), n=None, bits=32,
          lr=1e-3, lr_dev=None, b1=0.9, b2=0.95, eps=1e-8, step=1, step_dev=None, norm=None, max_norm=1.0):
    def arr(t, x):
        return None if x is None else (t * max(len(x), 1))(*x)
    return tw.lib().adamw_step(arr(P, p), arr(P, g), arr(P, m), arr(P, v), arr(P, ms), arr(P, vs), arr(P, copies), arr(I64, sizes),
                               arr(I32, dt), arr(I32, gt), arr(F64, wd), len(p) if n is None else n, bits, lr, lr_dev, b1, b2, eps,
                               step, step_dev, norm, max_norm, None)


EIGHT = dict(bits=8, ms=(E,), vs=(F,))


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), SHAPE), (dict(sizes=(-1,)), SHAPE), (dict(bits=16), ARG), (dict(g=None), ARG), (dict(m=None), ARG),
    (dict(v=None), ARG), (dict(sizes=None), ARG), (dict(dt=None), ARG), (dict(gt=None), ARG), (dict(wd=None), ARG),
    (dict(p=(None,)), ARG), (dict(g=(None,)), ARG), (dict(m=(None,)), ARG), (dict(v=(None,)), ARG), (dict(bits=8), ARG),
    (dict(bits=8, ms=(E,)), ARG), (dict(bits=8, ms=(None,), vs=(F,)), ARG), (dict(dt=(2,)), ARG), (dict(gt=(-1,)), ARG),
    (dict(lr=-1.0), ARG), (dict(lr=NAN), ARG), (dict(lr=INF), ARG), (dict(b1=1.0), ARG), (dict(b1=-0.1), ARG), (dict(b2=NAN), ARG),
    (dict(eps=0.0), ARG), (dict(eps=1e-46), ARG), (dict(eps=NAN), ARG), (dict(step=0), ARG), (dict(wd=(-0.1,)), ARG),
    (dict(wd=(NAN,)), ARG), (dict(norm=G, max_norm=-1.0), ARG), (dict(norm=G, max_norm=NAN), ARG),
    (dict(copies=(E,), dt=(1,)), ARG), (dict(p=(A + 2,)), ALIGN), (dict(p=(A + 1,), dt=(1,)), ALIGN), (dict(g=(B + 1,), gt=(1,)), ALIGN),
    (dict(g=(B + 2,)), ALIGN), (dict(m=(C + 2,)), ALIGN), (dict(v=(D + 1,)), ALIGN), (dict(copies=(E + 1,)), ALIGN),
    (dict(EIGHT, ms=(E + 2,)), ALIGN), (dict(EIGHT, vs=(F + 1,)), ALIGN), (dict(norm=G + 2), ALIGN), (dict(lr_dev=G + 1), ALIGN),
    (dict(step_dev=G + 4), ALIGN), (dict(sizes=((1 << 40) + 1,)), UNSUP),
    # overlaps: outputs with each other, with a gradient, with the scalars
    (dict(g=(A,)), ARG), (dict(m=(A,)), ARG), (dict(v=(C,)), ARG), (dict(m=(A + 60,)), ARG), (dict(copies=(A,)), ARG),
    (dict(copies=(B + 62,)), ARG), (dict(norm=A + 4), ARG), (dict(lr_dev=C), ARG), (dict(step_dev=D + 56), ARG),
    (dict(EIGHT, ms=(C,)), ARG), (dict(EIGHT, vs=(E,)), ARG), (dict(EIGHT, ms=(C + 12,)), ARG),
    (dict(p=(A, A), g=(B, B), m=(C, C + 64), v=(D, D + 64), sizes=(16, 16), dt=(0, 0), gt=(0, 0), wd=(0.0, 0.0)), ARG),
    # the last tensor's shape is looked at too
    (dict(p=(A, A + 64), g=(B, B), m=(C, C + 64), v=(D, D + 64), sizes=(16, -3), dt=(0, 0), gt=(0, 0), wd=(0.0, 0.0)), SHAPE),
    # nothing to do
    (dict(n=0), 0), (dict(sizes=(0,), p=(None,), g=(None,), m=(None,), v=(None,)), 0),
])
def test_adamw_rejects(kw, want):
    assert adamw(**kw) == want


def values(q=(A,), s=(B,), second=(0,), sizes=(300,), n=None, outs=(C,), dt=0):
    return tw.lib().adamw8_values((P * 2)(*q), (P * 2)(*s), (I32 * 2)(*second), (I64 * 2)(*sizes), len(q) if n is None else n,
                                  (P * 2)(*outs), dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), SHAPE), (dict(sizes=(-1,)), SHAPE), (dict(dt=2), ARG), (dict(q=(None,)), ARG), (dict(s=(None,)), ARG),
    (dict(outs=(None,)), ARG), (dict(s=(B + 1,)), ALIGN), (dict(outs=(C + 2,)), ALIGN), (dict(outs=(C + 1,), dt=1), ALIGN),
    (dict(sizes=((1 << 40) + 1,)), UNSUP), (dict(outs=(A,)), ARG), (dict(outs=(B + 4,)), ARG), (dict(outs=(A - 1196,)), ARG),
    (dict(q=(A, A), s=(B, B), second=(0, 0), sizes=(300, 300), outs=(C, C + 1196)), ARG), (dict(n=0), 0), (dict(sizes=(0,)), 0),
])
def test_adamw8_values_rejects(kw, want):
    assert values(**kw) == want


def test_python_refusals():
    """Before the library is called, on CPU tensors: names, shapes and types; then that they are no GPU's."""
    import torch
    x, w = torch.zeros(4, 64), torch.zeros(128, 64)
    for bad in (dict(act="swish"), dict(w_layout="mn"), dict(w_layout="kn")):
        with pytest.raises(ValueError):
            tw.linear_fwd(x, w, **bad)
    with pytest.raises(ValueError, match="GPU"):
        tw.linear_fwd(x, w)
    with pytest.raises(ValueError, match="GPU"):
        tw.ffn_gated_dense_fwd(x, w, w, w)
    with pytest.raises(ValueError):
        tw.linear_bwd(torch.zeros(5, 128), x, w)
    with pytest.raises(ValueError, match="32 bits"):
        tw.linear_fwd_workspace_bytes(1 << 40, 64, 64)
    p = [torch.zeros(8)]
    for call in (lambda: tw.adamw_step(p, p, p, p, 1e-3, 1), lambda: tw.adamw8_values([torch.zeros(8, dtype=torch.int8)], p)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    m, ms, v, vs = tw.adamw8_states(torch.zeros(3, 100))
    assert m.shape == v.shape == (3, 100) and ms.shape == vs.shape == (2,) and m.dtype == torch.int8 and v.dtype == torch.uint8
