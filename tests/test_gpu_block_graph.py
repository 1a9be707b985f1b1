"""Weights that change between the replays of a captured step: the MoE layer's
operands stay where the graph reads them, and a TrainBlock's step, its update
included, trains the same way captured and eager."""
import pytest
import torch

from helpers import gpu_ops

pytestmark = pytest.mark.gpu

T, d, E, k, f_moe, f = 256, 512, 8, 2, 256, 264
OPERANDS = [w + s for w in ("W1f", "W2f", "W1d", "W2d") for s in ("", "_s")]


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def make(bits):
    from grouped_gemm_top_gb300 import synth
    from grouped_gemm_top_gb300.block import TrainBlock
    b = TrainBlock(T, d, E, k, f_moe, f)
    b.init_weights(3)
    b.make_optimizer(lr=1e-2, state_bits=bits)
    b.s.copy_(synth.make_normal_bf16((T, d), 50, b.device))
    b.dout.copy_(synth.make_normal_bf16((T, d), 60, b.device, 0.1))
    return b


def test_operands_stay_in_place(ops):
    from grouped_gemm_top_gb300 import synth
    from grouped_gemm_top_gb300.layer import MoELayer
    L, M = MoELayer(T, d, E, k, f_moe), MoELayer(T, d, E, k, f_moe)
    w = [[synth.make_normal_bf16(s, i, "cuda", 0.05) for s in ((E, d, 2 * f_moe), (E, f_moe, d))] for i in (1, 2)]
    L.set_weights(*w[0])
    at = {n: getattr(L, n).data_ptr() for n in OPERANDS}
    L.set_weights(*w[1])
    assert at == {n: getattr(L, n).data_ptr() for n in OPERANDS}
    M.set_weights(*w[1])                       # and hold what a fresh layer's do
    assert all(torch.equal(getattr(L, n), getattr(M, n)) for n in OPERANDS)


def test_captured_layer_sees_new_weights(ops):
    from grouped_gemm_top_gb300 import synth
    from grouped_gemm_top_gb300.layer import MoELayer
    L, M = MoELayer(T, d, E, k, f_moe), MoELayer(T, d, E, k, f_moe)
    for y in (L, M):
        y.x.copy_(synth.make_normal_bf16((T, d), 7, "cuda"))
        y.dout.copy_(synth.make_normal_bf16((T, d), 8, "cuda"))
        y.logits.copy_(synth.make_normal_bf16((T, E), 9, "cuda"))
    for i in range(3):
        w = [synth.make_normal_bf16(s, 10 + i, "cuda", 0.05) for s in ((E, d, 2 * f_moe), (E, f_moe, d))]
        L.set_weights(*w)
        M.set_weights(*w)
        if i == 0:
            L.capture()
        L.replay()
        M.step_()
        assert all(torch.equal(getattr(L, n), getattr(M, n)) for n in ("out", "dx", "dW1", "dW2")), i
    L.check_err()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("update_captured", [True, False])
def test_replays_train_as_eager_steps_do(ops, bits, update_captured):
    a, b = make(bits), make(bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.forward_()
        b.backward_()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward_()
        b.backward_()
        if update_captured:
            b.update_()
    before = [t.clone() for t in a.optimizer.masters]
    for t in range(3):
        a.forward_()
        a.backward_()
        a.update_()
        graph.replay()
        if not update_captured:
            b.update_()
        same = [(getattr(a, n), getattr(b, n), n) for n in ("out", "ds", "W1", "W2", "We1", "We2", "Wr", "w_norm1", "w_norm2")]
        same += [(getattr(a.moe, n), getattr(b.moe, n), n) for n in OPERANDS + ["Wr", "WrT"]]
        same += [(x, y, "master") for x, y in zip(a.optimizer.masters, b.optimizer.masters)]
        for x, y, name in same:
            assert torch.equal(x, y), (t, name)
    assert all(not torch.equal(x, y) for x, y in zip(before, a.optimizer.masters))
    a.moe.check_err()
    b.moe.check_err()
