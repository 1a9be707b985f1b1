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

``python -m grouped_gemm_top_gb300.block`` trains one on synthetic data;
``--experts bf16`` with its experts in 16 bits, ``--distill`` under a head that
learns from a teacher's top logits."""
from __future__ import annotations

import argparse

import torch

from . import ops, synth
from .head import DistillHead
from .layer import MoELayer
from .layer_bf16 import MoELayerBF16
from .optim import AdamW


class TrainBlock:
    def __init__(self, T, d, E, k, f_moe, f, act="silu", eps=1e-6, score="softmax", normalize=True, device="cuda:0",
                 experts="mxfp8"):
        """T tokens of width d; an MoE sublayer of E experts of width f_moe,
        top-k, with its router, whose products are in MXFP8 or (experts="bf16")
        in bf16; a dense gated sublayer of width f (f % 8 == 0)."""
        self.T, self.d, self.f, self.act, self.eps = T, d, f, act, eps
        self.device = torch.device(device)
        if experts not in ("mxfp8", "bf16"):
            raise ValueError('experts: "mxfp8" or "bf16"')
        layer = MoELayer if experts == "mxfp8" else MoELayerBF16
        self.moe = layer(T, d, E, k, f_moe, score, normalize, device=device, router=True)

        def z(shape, dtype=torch.bfloat16):
            return torch.zeros(shape, dtype=dtype, device=self.device)

        # parameters (bf16) and their gradients
        self.w_norm1, self.w_norm2 = z((d,)).fill_(1.0), z((d,)).fill_(1.0)
        self.W1, self.W2 = z((d, 2 * f)), z((f, d))
        self.dW1, self.dW2 = z((d, 2 * f)), z((f, d))
        self.dw_norm1, self.dw_norm2 = z((d,), torch.float32), z((d,), torch.float32)
        # the MoE sublayer's bf16 weights (MXFP8: it quantizes its operands from them)
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
        """The MoE sublayer's operands (MXFP8: quantized) from its bf16 weights."""
        self.moe.set_weights(self.We1, self.We2)
        self.moe.set_router_weights(self.Wr)

    def make_optimizer(self, lr, weight_decay=0.1, state_bits=32, others=(), **kw):
        """AdamW over every weight (no decay on the norms' and the router's)
        and `others`, (parameter, gradient, decay) of what is trained with it."""
        m = self.moe
        self.optimizer = AdamW([(self.W1, self.dW1), (self.W2, self.dW2), (self.We1, m.dW1), (self.We2, m.dW2),
                                (self.Wr, m.dWr, 0.0), (self.w_norm1, self.dw_norm1, 0.0),
                                (self.w_norm2, self.dw_norm2, 0.0), *others],
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


def main(argv=None):
    ap = argparse.ArgumentParser(prog="python -m grouped_gemm_top_gb300.block", description="Trains a small block on synthetic data.")
    ap.add_argument("--experts", choices=("mxfp8", "bf16"), default="mxfp8", help="the experts' products")
    ap.add_argument("--distill", action="store_true", help="learn from a teacher's top logits instead of a target")
    ap.add_argument("--steps", type=int, default=40)
    args = ap.parse_args(argv)
    T, d, E, k, f_moe, f, V, top = 1024, 512, 8, 2, 256, 1024, 4000, 16
    b = TrainBlock(T, d, E, k, f_moe, f, experts=args.experts)
    b.init_weights()
    b.s.copy_(synth.make_normal_bf16((T, d), 100, b.device))
    if args.distill:
        head = DistillHead(T, d, V, top, temperature=2.0)
        head.init_weights(200)
        g = torch.Generator(device=b.device).manual_seed(201)
        head.idx.copy_(torch.randint(V, (T, 1), generator=g, device=b.device) + 7 * torch.arange(top, device=b.device))
        head.idx.remainder_(V)
        head.teacher.copy_(4 * torch.randn((T, top), generator=g, device=b.device))
        b.make_optimizer(lr=2e-3, state_bits=8, others=head.parameters())
    else:
        b.make_optimizer(lr=2e-3, state_bits=8)
        target = synth.make_normal_bf16((T, d), 101, b.device).float()
    for step in range(1, args.steps + 1):
        b.forward_()
        if args.distill:
            head.s.copy_(b.out)
            head.forward_backward_()
            b.dout.copy_(head.ds)
        else:
            err = b.out.float() - target
            b.dout.copy_(err / T)      # of the loss sum |out - target|^2 / 2T
        b.backward_()
        b.update_()
        if step == 1 or step % 10 == 0:
            loss = float(head.loss.mean()) if args.distill else 0.5 * float(err.square().sum()) / T
            print(f"step {step}: loss {loss:.4f}")
    b.moe.check_err()
    if args.distill:
        head.check_err()


if __name__ == "__main__":
    main()
