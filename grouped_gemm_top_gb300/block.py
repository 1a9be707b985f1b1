"""TrainBlock: a pre-norm transformer block's feed-forward half as it is
trained next to the MoE layer -- an MoE sublayer, a dense gated feed-forward
sublayer, and AdamW over the weights of both:

    n1 = norm(s),           m = MoE(n1)
    r  = s + m,             n2 = norm(r)             one call
    h  = act(gate) * up,    [gate | up] = n2 W1      one kernel
    out = r + h W2                                   residual in the epilogue

and the backward pass and update of every step.  Buffers are sized once;
forward_, backward_ and (once the weights have been set) update_ allocate
nothing and never synchronise, so they can be captured in a CUDA graph, in
one or apart: an update writes every weight and operand in place.

``python -m grouped_gemm_top_gb300.block`` trains one on synthetic data."""
from __future__ import annotations

import torch

from . import ops, synth
from .layer import MoELayer
from .optim import AdamW


class TrainBlock:
    def __init__(self, T, d, E, k, f_moe, f, act="silu", eps=1e-6, score="softmax", normalize=True, device="cuda:0"):
        """T tokens of width d; an MoE sublayer of E experts of width f_moe,
        top-k, with its router; a dense gated sublayer of width f (f % 8 == 0)."""
        self.T, self.d, self.f, self.act, self.eps = T, d, f, act, eps
        self.device = torch.device(device)
        self.moe = MoELayer(T, d, E, k, f_moe, score, normalize, device=device, router=True)

        def z(shape, dtype=torch.bfloat16):
            return torch.zeros(shape, dtype=dtype, device=self.device)

        # parameters (bf16) and their gradients
        self.w_norm1, self.w_norm2 = z((d,)).fill_(1.0), z((d,)).fill_(1.0)
        self.W1, self.W2 = z((d, 2 * f)), z((f, d))
        self.dW1, self.dW2 = z((d, 2 * f)), z((f, d))
        self.dw_norm1, self.dw_norm2 = z((d,), torch.float32), z((d,), torch.float32)
        # the MoE sublayer's bf16 weights (it quantizes its operands from them)
        self.We1, self.We2 = z((E, d, 2 * f_moe)), z((E, f_moe, d))
        self.Wr = z((d, E))
        # the stream in and out, and what the backward pass needs
        self.s, self.out = z((T, d)), z((T, d))
        self.dout, self.ds = z((T, d)), z((T, d))
        self.r, self.n2 = z((T, d)), z((T, d))
        self.rstd1, self.rstd2 = z((T,), torch.float32), z((T,), torch.float32)
        self.h, self.a = z((T, f)), z((T, 2 * f))
        self.dh, self.dn2 = z((T, f)), z((T, d))
        self.ws_norm = z((max(ops.rmsnorm_bwd_workspace_size(T, d), 1),), torch.uint8)
        self.optimizer = None

    def init_weights(self, seed=0, std=0.02):
        for i, w in enumerate((self.W1, self.W2, self.We1, self.We2, self.Wr)):
            w.copy_(synth.make_normal_bf16(tuple(w.shape), seed + i, self.device, std))
        self.set_weights()

    def set_weights(self):
        """The MoE sublayer's MXFP8 operands, from its bf16 weights."""
        self.moe.set_weights(self.We1, self.We2)
        self.moe.set_router_weights(self.Wr)

    def make_optimizer(self, lr, weight_decay=0.1, state_bits=32, **kw):
        """AdamW over every weight (no decay on the norms' and the router's)."""
        m = self.moe
        self.optimizer = AdamW([(self.W1, self.dW1), (self.W2, self.dW2), (self.We1, m.dW1), (self.We2, m.dW2),
                                (self.Wr, m.dWr, 0.0), (self.w_norm1, self.dw_norm1, 0.0),
                                (self.w_norm2, self.dw_norm2, 0.0)],
                               lr, weight_decay=weight_decay, state_bits=state_bits, **kw)
        return self.optimizer

    def forward_(self):
        """out from s."""
        m = self.moe
        ops.rmsnorm_residual_fwd(self.s, self.w_norm1, None, self.eps, y=m.x, rstd=self.rstd1)
        m.forward_()
        ops.rmsnorm_residual_fwd(m.out, self.w_norm2, self.s, self.eps, y=self.n2, r=self.r, rstd=self.rstd2)
        ops.gated_ffn_fwd(self.n2, self.W1, self.act, h=self.h, a=self.a, err=m.err)
        ops.linear_fwd(self.h, self.W2, residual=self.r, y=self.out, err=m.err)

    def backward_(self):
        """ds and every weight's gradient from dout."""
        m = self.moe
        ops.linear_bwd(self.dout, self.h, self.W2, dx=self.dh, dw=self.dW2, err=m.err)
        # da takes a's place: nothing reads a afterwards
        ops.gated_ffn_bwd(self.dh, self.a, self.n2, self.W1, self.act, dx=self.dn2, dw1=self.dW1, da=self.a,
                          err=m.err)
        # the gradient of r = s + MoE(n1): through the norm, and dout from the residual
        ops.rmsnorm_residual_bwd(self.dn2, self.r, self.w_norm2, self.rstd2, self.dout, dx=m.dout, dw=self.dw_norm2,
                                 ws=self.ws_norm)
        m.backward_()
        ops.rmsnorm_residual_bwd(m.dx, self.s, self.w_norm1, self.rstd1, m.dout, dx=self.ds, dw=self.dw_norm1,
                                 ws=self.ws_norm)

    def update_(self, grad_scale=None):
        """AdamW, then the MoE sublayer's operands from the new weights."""
        self.optimizer.step_(grad_scale)
        self.set_weights()


def main():
    T, d, E, k, f_moe, f = 1024, 512, 8, 2, 256, 1024
    b = TrainBlock(T, d, E, k, f_moe, f)
    b.init_weights()
    b.make_optimizer(lr=2e-3, state_bits=8)
    b.s.copy_(synth.make_normal_bf16((T, d), 100, b.device))
    target = synth.make_normal_bf16((T, d), 101, b.device).float()
    for step in range(1, 41):
        b.forward_()
        err = b.out.float() - target
        b.dout.copy_(err / T)      # of the loss sum |out - target|^2 / 2T
        b.backward_()
        b.update_()
        if step == 1 or step % 10 == 0:
            print(f"step {step}: loss {0.5 * float(err.square().sum()) / T:.4f}")
    b.moe.check_err()


if __name__ == "__main__":
    main()
