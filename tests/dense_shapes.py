"""Shapes of the dense layers that between them run every kernel the plan can choose, each also with its depth
split where that occurs (test_dense_plan_host.py holds them to it; test_gpu_dense_exact.py runs them): (operator, T,
d_in or d, d_out or f, type, layout)."""

CASES = [
    ("linear", 64, 14336, 4096, "bf16", "kn"), ("linear", 49, 5936, 12304, "bf16", "kn"), ("linear", 6, 13768, 6720, "f32", "nk"),
    ("linear", 344, 8696, 10032, "f32", "kn"),
    ("linear_back", 11019, 136, 5928, "bf16", "kn"), ("linear_back", 131, 2504, 6384, "f32", "kn"),
    ("linear_back", 2890, 1240, 920, "f32", "kn"), ("linear_back", 2, 8344, 12896, "bf16", "kn"),
    ("linear_back", 740, 2768, 1440, "f32", "kn"), ("linear_back", 3781, 8256, 80, "f32", "kn"),
    ("linear_back", 2, 40, 3456, "bf16", "kn"), ("linear_back", 403, 56, 40, "bf16", "kn"),
    ("gated", 2, 448, 1776, "f32", "nk"), ("gated", 9, 3064, 2608, "f32", "nk"), ("gated", 744, 1872, 12960, "f32", "nk"),
    ("gated", 214, 1536, 10760, "bf16", "nk"), ("gated", 15, 3400, 560, "bf16", "nk"), ("gated", 9319, 4056, 40, "bf16", "nk"),
    ("gated", 1080, 4144, 2008, "bf16", "nk"), ("gated", 2106, 2192, 232, "f32", "nk"), ("gated", 4170, 1632, 256, "f32", "nk"),
    ("gated", 15381, 280, 40, "bf16", "nk"), ("gated", 65, 2408, 40, "bf16", "nk"), ("gated", 2, 40, 8216, "f32", "nk"),
    ("gated", 8137, 152, 992, "f32", "nk"), ("gated", 297, 40, 11808, "bf16", "nk"), ("gated", 2, 336, 40, "f32", "nk"),
    ("gated", 2, 40, 40, "bf16", "nk"), ("gated", 2, 40, 40, "f32", "nk"),
    ("gated_back", 2, 448, 1776, "f32", "nk"), ("gated_back", 9, 3064, 2608, "f32", "nk"), ("gated_back", 1282, 992, 960, "bf16", "nk"),
    ("gated_back", 7927, 952, 264, "f32", "nk"), ("gated_back", 1589, 64, 1832, "bf16", "nk"),
    ("gated_back", 4827, 1696, 440, "f32", "nk"), ("gated_back", 194, 1016, 5024, "f32", "nk"),
    ("gated_back", 724, 72, 11024, "bf16", "nk"), ("gated_back", 2, 3704, 1864, "bf16", "nk"), ("gated_back", 2, 40, 40, "bf16", "nk"),
]


def products(op, T, K, N, layout):
    """An operator's products, as the plan is asked for them: (kind, dual, M, N, K, batch); kinds: 0 both operands
    along k, 1 the first across it, 2 both across."""
    if op == "linear":
        return [(0 if layout == "nk" else 1, 0, N, T, K, 1)]
    if op == "linear_back":
        return [(1 if layout == "nk" else 0, 0, K, T, N, 1), (2, 0, *((K, N) if layout == "nk" else (N, K)), T, 1)]
    if op == "gated":
        return [(0, 1, N, T, K, 1), (1, 0, K, T, N, 1)]
    return [(0, 0, N, T, K, 1), (1, 0, K, T, 2 * N, 1), (2, 0, K, N, T, 3)]
