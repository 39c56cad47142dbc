"""The workspace of the cross entropy against the bound in its header, over the shapes it takes."""
import random

import pytest

import activation_sparse_transformer_up_amd as tw

GIB = 1 << 30


def bound(T, d, V, bf16, grad):
    lde = (V + 255) // 256 * 256
    token = (lde // 16 + 16) * 8 + (lde * (2 if bf16 else 10) if grad else 0)
    piece = max(GIB, 256 * token) + (4 * V * d if bf16 and grad else 0)
    return piece + T * d * (2 if bf16 else 6) + 12 * T + (0 if bf16 else 6 * V * d) + 200_000_000


CORNERS = [(T, d, V, b, g) for T in (1, 300, 1 << 24) for d in (8, 1 << 16) for V in (1, 50021, 1 << 21) for b in (0, 1)
           for g in (0, 1)]


def shapes():
    rng = random.Random(5)
    for _ in range(3000):
        yield (int(2 ** rng.uniform(0, 24)), 8 * int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(0, 21)),
               rng.randint(0, 1), rng.randint(0, 1))


def test_bound():
    f = tw.lib().linear_xent_workspace_bytes
    for T, d, V, bf16, grad in CORNERS + list(shapes()):
        assert 0 < f(T, d, V, bf16, grad) <= bound(T, d, V, bf16, grad), (T, d, V, bf16, grad)


@pytest.mark.parametrize("V", [1 << 20, 1 << 21])
def test_fp32_pieces_of_a_huge_vocabulary_are_256_tokens(V):
    """Many more tokens take no larger piece: what grows is x's copy and the lists."""
    f, d = tw.lib().linear_xent_workspace_bytes, 4096
    a, b = f(1 << 12, d, V, 0, 1), f(1 << 16, d, V, 0, 1)
    assert a > 256 * 10 * V + 6 * V * d     # in planes
    assert b - a <= ((1 << 16) - (1 << 12)) * (6 * d + 12) + 1024
