"""Sizes beyond 32 bits are refused by the Python entry points of the norm and the loss: the library takes
32 bits, and a size cut to them would name a smaller tensor whose call succeeds. Tensors without
storage stand for large ones."""
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_transformer_up_amd as tw  # noqa: E402

BIG = (1 << 32) + 8                         # cut to 32 bits: 8
BF16, F32 = torch.bfloat16, torch.float32


def meta(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="meta")


CALLS = {
    "norm rows": lambda: tw.layer_norm_fwd(meta(BIG, 8), meta(8, dtype=F32)),
    "norm row of 2^31": lambda: tw.layer_norm_fwd(meta(1 << 31, 8), meta(8, dtype=F32)),
    "norm d": lambda: tw.layer_norm_fwd(meta(2, BIG), meta(BIG, dtype=F32)),
    "norm back rows": lambda: tw.layer_norm_bwd(meta(BIG, 8), meta(BIG, 8), meta(8, dtype=F32), meta(BIG, dtype=F32),
                                                meta(BIG, dtype=F32)),
    "norm back workspace": lambda: tw.layer_norm_bwd_workspace_bytes(BIG, 64),
    "xent tokens": lambda: tw.linear_xent_fwd(meta(BIG, 8), meta(9, 8), meta(BIG, dtype=torch.int64)),
    "xent d": lambda: tw.linear_xent_fwd(meta(1, BIG), meta(2, BIG), meta(1, dtype=torch.int64)),
    "xent vocabulary": lambda: tw.linear_xent_fwd_bwd(meta(3, 8), meta(BIG, 8), meta(3, dtype=torch.int64),
                                                      meta(3, dtype=F32)),
    "xent workspace": lambda: tw.linear_xent_workspace_bytes(4, 64, BIG),
    "clip workspace": lambda: tw.grad_norm_workspace_bytes(BIG),
}


@pytest.mark.parametrize("name", CALLS)
def test_sizes_beyond_32_bits(name):
    with pytest.raises(ValueError, match="32 bits"):
        CALLS[name]()


def test_sizes_in_32_bits():
    assert tw.layer_norm_bwd_workspace_bytes((1 << 31) - 1, 64) > 0
    with pytest.raises(ValueError, match="on the GPU"):
        tw.layer_norm_fwd(meta((1 << 31) - 1, 8), meta(8, dtype=F32))
