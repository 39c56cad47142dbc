"""grad_clip refuses outputs that overlap each other or another tensor's gradient (their elements would
be scaled once or twice, as the workgroups happen to run), before anything is enqueued: a call that
passes this check here ends at the workspace's."""
import ctypes

import pytest

import activation_sparse_transformer_up_amd as tw

ARG, WS = -1, -4
F32, BF16 = 0, 1


def clip(*tensors):
    """tensors: (gradient address, output address, elements, dtype, output dtype). No workspace."""
    P, L, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    n = len(tensors)
    g, o, s, t, ot = ((c * n)(*(x[k] for x in tensors)) for k, c in enumerate((P, P, L, I, I)))
    return tw.lib().grad_clip(g, o, s, t, ot, n, 1.0, 0x10000, None, 0, None)


A, B, C = 0x100000, 0x200000, 0x300000


@pytest.mark.parametrize("tensors,want", [
    # apart: in place, elsewhere, touching neighbours in any order, one gradient read for two outputs
    ([(A, A, 16, F32, F32)], WS),
    ([(A, A, 16, F32, F32), (A + 64, A + 64, 16, F32, F32)], WS),
    ([(A + 64, A + 64, 16, F32, F32), (A, A, 16, F32, F32)], WS),
    ([(A, B + 32, 16, F32, BF16), (A + 64, B, 16, F32, BF16)], WS),
    ([(A, B, 16, F32, F32), (A, C, 16, F32, F32)], WS),
    ([(A, A, 16, BF16, BF16), (A + 32, B, 16, BF16, BF16)], WS),
    # empty tensors are nowhere
    ([(A, A, 16, F32, F32), (A, A, 0, F32, F32)], WS),
    # the same tensor twice
    ([(A, A, 16, F32, F32), (A, A, 16, F32, F32)], ARG),
    ([(A, A, 16, F32, F32), (B, B, 16, F32, F32), (A, A, 16, F32, F32)], ARG),
    # outputs that share elements
    ([(A, C, 16, F32, F32), (B, C, 16, F32, F32)], ARG),
    ([(A, C, 16, F32, F32), (B, C + 60, 16, F32, F32)], ARG),
    ([(A, C + 30, 16, F32, BF16), (B, C, 16, F32, BF16)], ARG),
    # an output in another tensor's gradient, or shifted in its own
    ([(A, B, 16, F32, F32), (B, C, 16, F32, F32)], ARG),
    ([(A, B + 60, 16, F32, F32), (B, C, 16, F32, F32)], ARG),
    ([(A, A, 16, F32, F32), (A + 60, C, 16, F32, F32)], ARG),
    ([(A, A + 4, 16, F32, F32)], ARG),
    ([(A + 4, A, 16, F32, F32)], ARG),
    # in place as another type
    ([(A, A, 16, F32, BF16)], ARG),
])
def test_overlap(tensors, want):
    assert clip(*tensors) == want
    # the same among more tensors than one launch takes
    far = [(0x10000000 + 256 * k, 0x10000000 + 256 * k, 64, F32, F32) for k in range(100)]
    assert clip(*far[:50], *tensors, *far[50:]) == want
