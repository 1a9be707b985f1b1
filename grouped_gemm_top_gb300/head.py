"""DistillHead: the end of a language model that learns from a teacher -- final
norm, projection to the vocabulary, and the distillation loss against the
teacher's top logits:

    n = norm(s),   logits = n W,   loss = distill(logits; idx, teacher)

forward_backward_ makes the loss and its gradient in one pass over the logits,
in their place, so that of [T, V] there is one buffer.  Buffers are sized once;
the calls allocate nothing, never synchronise and can be captured."""
from __future__ import annotations

import torch

from . import ops, synth


class DistillHead:
    def __init__(self, T, d, V, k, temperature=1.0, tail=False, eps=1e-6, device="cuda:0"):
        """T tokens of width d (d % 8 == 0), a vocabulary of V, k teacher
        logits per token.  tail: the teacher's log-sum-exp over its whole
        vocabulary is given too (teacher_lse)."""
        self.T, self.d, self.V, self.temperature, self.eps = T, d, V, float(temperature), eps
        self.device = torch.device(device)
        ops.moe_init(self.device.index or 0)

        def z(shape, dtype=torch.bfloat16):
            return torch.zeros(shape, dtype=dtype, device=self.device)

        wide = (V + 7) // 8 * 8      # rows at multiples of 16 bytes
        self.w_norm, self.W = z((d,)).fill_(1.0), z((d, wide))[:, :V]
        self.dw_norm, self.dW = z((d,), torch.float32), z((d, wide))[:, :V]
        self.s, self.n, self.rstd = z((T, d)), z((T, d)), z((T,), torch.float32)
        self.logits = z((T, wide))[:, :V]
        # the teacher, and each token's weight in the training loss (0: masked)
        self.idx, self.teacher = z((T, k), torch.int32).fill_(-1), z((T, k), torch.float32)
        self.teacher_lse = z((T,), torch.float32) if tail else None
        self.weight = z((T,), torch.float32).fill_(1.0 / T)
        self.loss, self.stats = z((T,), torch.float32), z((T, 3), torch.float32)
        self.dn, self.ds = z((T, d)), z((T, d))
        self.ws_norm = z((max(ops.rmsnorm_bwd_workspace_size(T, d), 1),), torch.uint8)
        self.err = z((1,), torch.int32)

    def init_weights(self, seed=0, std=0.02):
        self.W.copy_(synth.make_normal_bf16((self.d, self.V), seed, self.device, std))

    def parameters(self):
        """(parameter, gradient, weight decay) of each, for AdamW."""
        return [(self.W, self.dW, 0.0), (self.w_norm, self.dw_norm, 0.0)]

    def _logits(self):
        ops.rmsnorm_residual_fwd(self.s, self.w_norm, None, self.eps, y=self.n, rstd=self.rstd)
        ops.linear_fwd(self.n, self.W, y=self.logits, err=self.err)

    def forward_(self):
        """logits, and every token's loss (validation)."""
        self._logits()
        ops.distill_loss_fwd(self.logits, self.idx, self.teacher, self.teacher_lse, self.temperature, loss=self.loss,
                             stats=self.stats, err=self.err)

    def forward_backward_(self):
        """Every token's loss, and ds, dW and dw_norm of the sum of weight * loss;
        logits holds their gradient afterwards."""
        self._logits()
        ops.distill_loss(self.weight, self.logits, self.idx, self.teacher, self.teacher_lse, self.temperature,
                         loss=self.loss, dlogits=self.logits, err=self.err)
        ops.linear_bwd(self.logits, self.n, self.W, dx=self.dn, dw=self.dW, err=self.err)
        ops.rmsnorm_residual_bwd(self.dn, self.s, self.w_norm, self.rstd, None, dx=self.ds, dw=self.dw_norm,
                                 ws=self.ws_norm)

    def check_err(self):
        v = int(self.err.item())
        if v != 0:
            raise ops.MoEError("device", v)
