"""MoELayerBF16 reads the caller's weights where they lie: what the products
could not read is refused when it is handed over, not at the next step."""
import pytest
import torch

from helpers import build_lib, gpu_ops

BF = torch.bfloat16
SHAPE = torch.Size((3, 16, 24))


def good():
    """as they lie: contiguous, rows apart, matrices apart, one row, one matrix"""
    yield torch.zeros(SHAPE, dtype=BF)
    yield torch.zeros((3, 16, 40), dtype=BF)[:, :, 8:32]
    yield torch.zeros((3, 20, 24), dtype=BF)[:, :16]
    yield torch.zeros((3, 1, 24), dtype=BF).as_strided((3, 1, 24), (24, 5, 1))
    yield torch.zeros((1, 16, 24), dtype=BF).as_strided((1, 16, 24), (3, 24, 1))


def bad():
    w = torch.zeros(SHAPE, dtype=BF)
    yield w.float()
    yield w.half()
    yield w.to("meta")
    yield w[:2]
    yield w.transpose(1, 2)
    yield torch.zeros((3, 24, 16), dtype=BF).transpose(1, 2)
    yield w[:1].expand(SHAPE)
    yield w[:, :1].expand(SHAPE)
    yield torch.zeros((3, 16, 28), dtype=BF)[:, :, :24]
    yield torch.zeros((3, 16, 32), dtype=BF)[:, :, 1:25]
    yield torch.zeros((3 * 388 + 1,), dtype=BF).as_strided(SHAPE, (388, 24, 1))
    yield None
    yield [[0.0]]


def test_what_the_products_read():
    build_lib()
    from grouped_gemm_top_gb300.layer_bf16 import _as_operand
    for w in good():
        assert _as_operand("W", w, w.shape, torch.device("cpu")) is w
    for w in bad():
        with pytest.raises(ValueError):
            _as_operand("W", w, SHAPE, torch.device("cpu"))


def test_odd_widths_are_refused():
    build_lib()
    from grouped_gemm_top_gb300.layer_bf16 import MoELayerBF16
    for d, f in ((60, 64), (64, 60)):
        with pytest.raises(ValueError):
            MoELayerBF16(16, d, 4, 2, f)


@pytest.mark.gpu
def test_set_weights():
    gpu_ops()
    from grouped_gemm_top_gb300.layer_bf16 import MoELayerBF16
    L = MoELayerBF16(16, 64, 4, 2, 40)
    W1, W2 = torch.zeros((4, 64, 80), dtype=BF, device="cuda"), torch.zeros((4, 40, 64), dtype=BF, device="cuda")
    L.set_weights(W1, W2)
    for a, b in ((W1.float(), W2), (W1, W2.cpu()), (W1, W2.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            L.set_weights(a, b)
        assert L.W1 is W1 and L.W2 is W2      # as they were
