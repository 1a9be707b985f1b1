"""AdamW: fp32 masters, first and second moments in 32 or 8 bits, and the
bf16 parameters that the layers read, all updated by one launch per gradient
type (ops.adamw_step).  The step count and the learning rate live on the
device, so a captured step counts on when its graph is replayed."""
from __future__ import annotations

import torch

from . import ops


class AdamW:
    def __init__(self, params, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, state_bits=32, seed=0):
        """params: list of (bf16 parameter, gradient) or (bf16 parameter,
        gradient, weight decay); the gradient is the buffer (bf16 or fp32)
        that every backward pass writes.  The masters start as the
        parameters' values.  state_bits: 32, or 8 (E4M3 codes with a scale
        per 256 elements, include/moe.h)."""
        if state_bits not in (32, 8):
            raise ValueError("state_bits: 32 or 8")
        entries = [(p[0], p[1], float(p[2]) if len(p) > 2 else float(weight_decay)) for p in params]
        dev = entries[0][0].device
        ops.moe_init(dev.index or 0)
        self.lr = torch.full((1,), float(lr), dtype=torch.float32, device=dev)
        self.betas, self.eps, self.seed = betas, eps, int(seed)
        self.masters, self.groups = [], []
        for dtype in (torch.bfloat16, torch.float32):
            mine = [e for e in entries if e[1].dtype == dtype]
            if not mine:
                continue
            flat = [(p.detach().reshape(-1), g.reshape(-1)) for p, g, _ in mine]
            masters = [p.float() for p, _ in flat]
            sizes = [p.numel() for p in masters]

            def state():
                if state_bits == 32:
                    return [torch.zeros((n,), dtype=torch.float32, device=dev) for n in sizes], None
                return ([torch.zeros((n,), dtype=torch.uint8, device=dev) for n in sizes],
                        [torch.zeros(((n + 255) // 256,), dtype=torch.float32, device=dev) for n in sizes])

            (m, ms), (v, vs) = state(), state()
            plan = ops.adamw_plan(masters, [g for _, g in flat], m, v, ms, vs, copies=[p for p, _ in flat],
                                  weight_decay=[w for _, _, w in mine])
            self.masters += masters
            self.groups.append((plan, torch.zeros((1,), dtype=torch.int32, device=dev)))

    def step_(self, grad_scale=None):
        """One update from the gradients in their buffers.  grad_scale: fp32
        device tensor, a factor of every gradient (not finite: no update)."""
        for plan, count in self.groups:
            ops.adamw_step(plan, self.lr, self.betas, self.eps, step=count, grad_scale=grad_scale, seed=self.seed)
