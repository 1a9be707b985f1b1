"""TrainBlock: the norm, the MoE layer, the dense feed-forward sublayer and
AdamW together as a training step uses them.  Each stage is compared with the
fp64 definition on the values that the GPU handed it, so the tolerances are
those of the stages (a bf16 store 2^-8 of the value, rounded operands of the
backward products 2^-8 of the terms' sizes)."""
import numpy as np
import pytest
import torch

from helpers import gpu_ops
from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu

T, d, E, k, f_moe, f = 256, 512, 8, 2, 256, 264
HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def f64(t):
    return t.double().cpu().numpy()


def make(seed=0, **opt):
    from grouped_gemm_top_gb300.block import TrainBlock
    from grouped_gemm_top_gb300 import synth
    b = TrainBlock(T, d, E, k, f_moe, f)
    b.init_weights(seed)
    if opt:
        b.make_optimizer(**opt)
    b.s.copy_(synth.make_normal_bf16((T, d), 50 + seed, b.device))
    b.dout.copy_(synth.make_normal_bf16((T, d), 60 + seed, b.device, 0.1))
    return b


def near(got, want, size):
    """Half a bf16 step of the value, and 2^-12 of the terms' sizes."""
    assert np.all(np.abs(f64(got) - want) <= np.abs(want) * HALF + size * 2.0 ** -12 + 1e-30)


def test_stages(ops):
    b = make()
    m = b.moe
    b.forward_()
    a_kept = f64(b.a)
    b.backward_()
    torch.cuda.synchronize()
    m.check_err()
    # forward: what each call made of its inputs
    _, _, n1 = D.rmsnorm_residual(f64(b.s), None, f64(b.w_norm1), b.eps)
    near(m.x, n1, np.abs(n1))
    r, rstd2, n2 = D.rmsnorm_residual(f64(m.out), f64(b.s), f64(b.w_norm2), b.eps)
    near(b.r, r, np.abs(r))
    near(b.n2, n2, np.abs(n2))
    h, a = D.gated_ffn(f64(b.n2), f64(b.W1))
    size = np.abs(f64(b.n2)) @ np.abs(f64(b.W1))
    near(b.h, h, size[:, :f] * (1 + np.abs(a[:, f:])) + size[:, f:] * (1 + np.abs(a[:, :f])))
    out, _ = D.linear(f64(b.h), f64(b.W2), residual=f64(b.r))
    near(b.out, out, np.abs(f64(b.h)) @ np.abs(f64(b.W2)) + np.abs(f64(b.r)))
    # backward
    dh, dW2, _, _ = D.linear_bwd(f64(b.dout), f64(b.h), f64(b.W2))
    near(b.dh, dh, np.abs(f64(b.dout)) @ np.abs(f64(b.W2)).T)
    near(b.dW2, dW2, np.abs(f64(b.h)).T @ np.abs(f64(b.dout)))
    dn2, dW1, da = D.gated_ffn_bwd(f64(b.dh), a_kept, f64(b.n2), f64(b.W1))
    rounded = 16 * np.abs(da)                       # da's rounding: 2^-8 of the terms
    near(b.dn2, dn2, rounded @ np.abs(f64(b.W1)).T)
    near(b.dW1, dW1, np.abs(f64(b.n2)).T @ rounded)
    dr, dw = D.rmsnorm_residual_bwd(f64(b.dn2), f64(b.r), f64(b.w_norm2), f64(b.rstd2), f64(b.dout))
    near(m.dout, dr, np.abs(f64(b.dn2)).max() + np.abs(dr))
    assert np.allclose(f64(b.dw_norm2), dw, rtol=1e-4, atol=1e-4 * np.abs(dw).max())
    ds, dw = D.rmsnorm_residual_bwd(f64(m.dx), f64(b.s), f64(b.w_norm1), f64(b.rstd1), f64(m.dout))
    near(b.ds, ds, np.abs(f64(m.dx)).max() + np.abs(ds))
    assert np.allclose(f64(b.dw_norm1), dw, rtol=1e-4, atol=1e-4 * np.abs(dw).max())


@pytest.mark.parametrize("bits", [32, 8])
def test_update_and_captured_step(ops, bits):
    """The step captured as a graph (forward, backward, AdamW) and replayed
    gives the bits of the eager one, and the masters move as AdamW's formula
    says."""
    a, b = make(lr=1e-3, state_bits=bits), make(lr=1e-3, state_bits=bits)
    before = [t.clone() for t in a.optimizer.masters]

    def step(x):
        x.forward_()
        x.backward_()
        x.optimizer.step_()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.forward_()
        b.backward_()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for t in range(1, 4):
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        if t == 1:
            grads = [a.dW1, a.dW2, a.moe.dW1, a.moe.dW2, a.moe.dWr, a.dw_norm1, a.dw_norm2]
            decay = [0.1] * 4 + [0.0] * 3
            for m0, m1, g, wd in zip(before, a.optimizer.masters, grads, decay):
                g = f64(g).reshape(-1)
                zero = np.zeros_like(g)
                want, _, _ = D.adamw(f64(m0), g, zero, zero, 1, 1e-3, 0.9, 0.999, 1e-8, wd)
                assert np.all(np.abs(f64(m1) - want) <= 2.0 ** -21 * np.abs(want) + 1e-3 * 2.0 ** -16)
        a.set_weights()
        b.set_weights()          # new operands for the eager forward; the graph reads its own
        assert int(a.optimizer.groups[0][1]) == t and int(b.optimizer.groups[0][1]) == t
        if t == 1:               # (later replays multiply by the MoE operands of the capture)
            for x, y in zip(a.optimizer.masters, b.optimizer.masters):
                assert torch.equal(x, y)
            assert torch.equal(a.W1, a.optimizer.masters[0].view_as(a.W1).bfloat16())


def test_training_lowers_the_loss(ops):
    b = make(lr=2e-3, state_bits=8)
    target = torch.randn((T, d), generator=torch.Generator(device="cuda").manual_seed(9), device="cuda")
    losses = []
    for _ in range(20):
        b.forward_()
        e = b.out.float() - target
        losses.append(float(e.square().mean()))
        b.dout.copy_(e / T)
        b.backward_()
        b.update_()
    b.moe.check_err()
    assert losses[-1] < 0.8 * losses[0] and all(np.isfinite(losses))
