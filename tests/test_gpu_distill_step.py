"""The 16-bit MoE layer, a TrainBlock with it, and the distillation head as a
training step uses them together.  Each stage is compared with its definition
in 64 bits on the values that the GPU handed it (tolerances of the stages)."""
import numpy as np
import pytest
import torch

from helpers import gpu_ops
from oracle.distill_oracle import distill
from test_gpu_grouped import HALF, acc, ffn_check, product

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def layer(T=256, d=136, E=8, k=2, f=72, seed=0, router=False):
    from grouped_gemm_top_gb300 import synth
    from grouped_gemm_top_gb300.layer_bf16 import MoELayerBF16
    L = MoELayerBF16(T, d, E, k, f, "softmax", True, router=router)
    L.set_weights(synth.make_normal_bf16((E, d, 2 * f), seed, "cuda", 0.1), synth.make_normal_bf16((E, f, d), seed + 1, "cuda", 0.1))
    L.x.copy_(synth.make_normal_bf16((T, d), seed + 2, "cuda"))
    L.dout.copy_(synth.make_normal_bf16((T, d), seed + 3, "cuda"))
    if router:
        L.set_router_weights(synth.make_normal_bf16((d, E), seed + 4, "cuda", 0.1))
    else:
        L.logits.copy_(synth.make_normal_bf16((T, E), seed + 5, "cuda"))
    return L


def close(got, want, tol, what):
    off = (got.double() - want).abs() - tol
    assert bool((off <= 1e-30).all()), (what, float(off.max()))


@pytest.mark.parametrize("T,d,E,k,f", [(256, 136, 8, 2, 72), (1, 64, 4, 2, 64), (5, 264, 16, 3, 40), (700, 512, 4, 1, 256)])
def test_layer_stages(ops, T, d, E, k, f):
    L = layer(T, d, E, k, f)
    if T > 5:
        L.logits[:, 1] = -50.0      # an expert without rows
    L.forward_()
    a_kept = L.a.clone()
    L.backward_()
    L.check_err()
    if T > 5 and k < E:
        assert int(L.counts[1]) == 0 and float(L.dW1[1].abs().max()) == 0 and float(L.dW2[1].abs().max()) == 0
    starts, counts, slots = L.gofs.tolist(), L.counts.tolist(), L.slot_of.long()
    assert sum(counts) == T * k
    assert torch.equal(L.x_perm[slots.view(-1)], L.x.repeat_interleave(k, 0))
    for g in range(E):
        lo, hi = starts[g], starts[g] + counts[g]
        if lo == hi:
            continue
        ffn_check(L.h[lo:hi], a_kept[lo:hi], L.x_perm[lo:hi], L.W1[g], "silu", f"expert {g}")
        product(L.y_perm[lo:hi], L.h[lo:hi], L.W2[g], f"y {g}")
        product(L.dh[lo:hi], L.dy_perm[lo:hi], L.W2[g].T, f"dh {g}")
        product(L.dW2[g], L.h[lo:hi].T, L.dy_perm[lo:hi], f"dW2 {g}")
        product(L.dx_perm[lo:hi], L.a[lo:hi], L.W1[g].T, f"dx {g}")              # a holds da
        product(L.dW1[g], L.x_perm[lo:hi].T, L.a[lo:hi], f"dW1 {g}")
    w = L.topk_w.double()
    rows = L.y_perm[slots].double()
    want = (rows * w[:, :, None]).sum(1)
    close(L.out, want, want.abs() * HALF + (rows.abs() * w[:, :, None]).sum(1) * k * 2.0 ** -23, "combine")
    close(L.dy_perm[slots], w[:, :, None] * L.dout.double()[:, None], (w[:, :, None] * L.dout.double()[:, None]).abs() * (HALF + 2.0 ** -23), "dy")
    dw = (rows * L.dout.double()[:, None]).sum(2)
    close(L.dw, dw, (rows * L.dout.double()[:, None]).abs().sum(2) * d * 2.0 ** -24, "dw")
    got, dx = L.dx_perm[slots].double(), L.dx
    close(dx, got.sum(1), got.sum(1).abs() * HALF + got.abs().sum(1) * k * 2.0 ** -23, "dx")


def test_layer_against_the_mxfp8_layer(ops):
    """the same layer in 8 bits gives about the same: its codes have 3 bits of mantissa"""
    from grouped_gemm_top_gb300.layer import MoELayer
    T, d, E, k, f = 256, 512, 8, 2, 256
    L = layer(T, d, E, k, f)
    M = MoELayer(T, d, E, k, f, "softmax", True)
    M.set_weights(L.W1, L.W2)
    for name in ("x", "dout", "logits"):
        getattr(M, name).copy_(getattr(L, name))
    L.step_()
    M.step_()
    assert torch.equal(L.topk_idx, M.topk_idx) and torch.equal(L.slot_of, M.slot_of)
    # four roundings of at most 2^-4 each on a path, random in sign
    for name in ("out", "dx", "dW1", "dW2"):
        p, q = getattr(L, name).double(), getattr(M, name).double()
        assert float((p - q).norm() / p.norm()) < 4 * 2.0 ** -4, name


def test_layer_captured_and_other_routing(ops):
    """a captured step replayed over other inputs, weights and routing"""
    L, M = layer(seed=10), layer(seed=10)
    L.step_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.step_()
    from grouped_gemm_top_gb300 import synth
    for i in range(3):
        for y in (L, M):
            y.logits.copy_(synth.make_normal_bf16((256, 8), 30 + i, "cuda", 3.0))
            y.W1.copy_(synth.make_normal_bf16(tuple(y.W1.shape), 40 + i, "cuda", 0.1))
        graph.replay()
        M.step_()
        torch.cuda.synchronize()
        for name in ("out", "dx", "dW1", "dW2", "dlogits"):
            assert torch.equal(getattr(L, name), getattr(M, name)), (i, name)
        L.check_err()


def test_router_gradients(ops):
    L = layer(256, 128, 8, 2, 64, seed=20, router=True)
    L.step_()
    L.check_err()
    x, dl = L.x.double(), L.dlogits.bfloat16().double()
    close(L.dWr, x.T @ dl, x.abs().T @ dl.abs() * acc(256), "dWr")
    rows = L.dx_perm[L.slot_of.long()].double()
    want = rows.sum(1) + dl @ L.Wr.double().T
    close(L.dx, want, want.abs() * HALF + (rows.abs().sum(1) + dl.abs() @ L.Wr.double().abs().T) * (acc(8) + 2.0 ** -21), "dx")


def head(T=130, d=72, V=1003, k=9, tail=False, tau=2.0, seed=0):
    from grouped_gemm_top_gb300 import synth
    from grouped_gemm_top_gb300.head import DistillHead
    h = DistillHead(T, d, V, k, tau, tail)
    h.init_weights(seed, 0.2)
    g = torch.Generator(device="cuda").manual_seed(seed)
    h.s.copy_(synth.make_normal_bf16((T, d), seed + 1, "cuda"))
    h.idx.copy_(torch.stack([torch.randperm(V, generator=g, device="cuda")[:k] for _ in range(T)]))
    h.idx[T // 2:T // 2 + 3] = -1                        # masked tokens
    h.teacher.copy_(2 * torch.randn((T, k), generator=g, device="cuda"))
    h.weight.mul_(torch.rand((T,), generator=g, device="cuda"))
    if tail:
        h.teacher_lse.copy_(torch.logsumexp(h.teacher / tau, 1) + 0.2)
    return h


@pytest.mark.parametrize("tail", [False, True])
def test_head(ops, tail):
    h = head(tail=tail)
    h.forward_()
    logits, loss = h.logits.clone(), h.loss.clone()
    h.forward_backward_()
    h.check_err()
    lse = None if h.teacher_lse is None else h.teacher_lse.double().cpu().numpy()
    want, dx = distill(logits.double().cpu().numpy(), h.idx.cpu().numpy(), h.teacher.double().cpu().numpy(), lse, 2.0,
                       h.weight.double().cpu().numpy())
    assert np.allclose(h.loss.double().cpu().numpy(), want, rtol=1e-5, atol=1e-5)
    assert np.allclose(loss.double().cpu().numpy(), want, rtol=1e-5, atol=1e-5)
    dl = h.logits.double().cpu().numpy()                 # the gradient, in the logits' place
    assert np.all(np.abs(dl - dx) <= np.abs(dx) * HALF + 1e-5 * np.abs(dx).max())
    assert np.all(dl[h.T // 2:h.T // 2 + 3] == 0)
    product(h.dW, h.n.T, h.logits, "dW")
    product(h.dn, h.logits, h.W.T, "dn")
    n, r = h.n.double(), h.rstd.double()[:, None]
    xhat = h.s.double() * r
    t = h.dn.double() * h.w_norm.double()
    ds = r * (t - xhat * (t * xhat).mean(1, keepdim=True))
    close(h.ds, ds, ds.abs() * HALF + r * t.abs().amax(1, keepdim=True) * 2.0 ** -18, "ds")


def block(bits, seed=0):
    from grouped_gemm_top_gb300 import synth
    from grouped_gemm_top_gb300.block import TrainBlock
    T, d = 256, 512
    b = TrainBlock(T, d, 8, 2, 256, 264, experts="bf16")
    b.init_weights(seed)
    h = head(T, d, 1003, 9, seed=seed)
    b.make_optimizer(lr=1e-2, state_bits=bits, others=h.parameters())
    b.s.copy_(synth.make_normal_bf16((T, d), 50 + seed, "cuda"))
    return b, h


def step(b, h):
    b.forward_()
    h.s.copy_(b.out)
    h.forward_backward_()
    b.dout.copy_(h.ds)
    b.backward_()
    b.update_()


@pytest.mark.parametrize("bits", [32, 8])
def test_training_step_captured_and_eager(ops, bits):
    """norm, 16-bit MoE, dense sublayer, head, loss, backward and AdamW: the whole step
    captured in a graph trains as the eager one does, bit by bit"""
    (b, h), (c, g) = block(bits), block(bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):        # warm-up without an update
        c.forward_()
        g.s.copy_(c.out)
        g.forward_backward_()
        c.dout.copy_(g.ds)
        c.backward_()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, g)
    for i in range(4):
        step(b, h)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in ((b.out, c.out), (h.loss, g.loss), (b.ds, c.ds), (b.moe.dW1, c.moe.dW1), (h.dW, g.dW), (h.W, g.W),
                     (b.We1, c.We1), (b.Wr, c.Wr)):
            assert torch.equal(x, y), i
    b.moe.check_err()
    h.check_err()
    assert bool(torch.isfinite(h.loss).all()) and float(h.dW.abs().max()) > 0


@pytest.mark.parametrize("argv", [["--experts", "bf16"], ["--distill"], ["--experts", "bf16", "--distill"]])
def test_command(ops, argv, capsys):
    from grouped_gemm_top_gb300 import block as module
    module.main(argv + ["--steps", "3"])
    assert "step 1: loss" in capsys.readouterr().out


def test_refusals(ops):
    from grouped_gemm_top_gb300.block import TrainBlock
    from grouped_gemm_top_gb300.layer_bf16 import MoELayerBF16
    with pytest.raises(ValueError):
        TrainBlock(128, 64, 8, 2, 64, 64, experts="fp4")
    with pytest.raises(ValueError):
        MoELayerBF16(100, 64, 8, 2, 64, router=True)
    L = MoELayerBF16(16, 64, 4, 2, 64)
    with pytest.raises(RuntimeError):
        L.step_()
    with pytest.raises(ValueError):
        L.set_weights(torch.empty((4, 64, 64), dtype=BF, device="cuda"), torch.empty((4, 64, 64), dtype=BF, device="cuda"))
