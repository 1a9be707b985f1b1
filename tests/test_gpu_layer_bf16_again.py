"""MoELayerBF16's backward pass does not use up what the forward pass kept: it can
be repeated, eagerly and replayed, as MoELayer's can."""
import pytest
import torch

from helpers import gpu_ops
from test_gpu_distill_step import layer

pytestmark = pytest.mark.gpu

OUT = ("dx", "dW1", "dW2", "dw", "dlogits")


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def of(L):
    return [getattr(L, n).clone() for n in OUT]


@pytest.mark.parametrize("T,d,E,k,f,router", [(256, 136, 8, 2, 72, False), (1, 64, 4, 2, 64, False), (256, 128, 8, 2, 64, True)])
def test_backward_again(ops, T, d, E, k, f, router):
    from grouped_gemm_top_gb300 import synth
    L, M = layer(T, d, E, k, f, router=router), layer(T, d, E, k, f, router=router)
    L.forward_()
    kept = L.a.clone()
    L.backward_()
    first = of(L)
    assert torch.equal(L.gate_up, kept) and not torch.equal(L.a, kept)
    L.backward_()
    assert all(torch.equal(p, q) for p, q in zip(first, of(L)))
    # of another output gradient, after the same forward pass
    dout = synth.make_normal_bf16((T, d), 77, "cuda")
    for y in (L, M):
        y.dout.copy_(dout)
    L.backward_()
    M.step_()
    assert all(torch.equal(p, q) for p, q in zip(of(M), of(L)))
    L.check_err()


def test_backward_replayed(ops):
    """a captured backward pass, twice for each eager forward pass"""
    L, M = layer(seed=3), layer(seed=3)
    L.step_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.backward_()
    for i in range(2):
        for y in (L, M):
            y.x.mul_(0.5)
            y.forward_()
        M.backward_()
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(of(M), of(L))), i
