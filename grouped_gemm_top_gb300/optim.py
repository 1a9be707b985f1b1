"""AdamW: fp32 masters, first and second moments in 32 or 8 bits, and the
bf16 parameters that the layers read, all updated by one launch per gradient
type (ops.adamw_step).  The step count and the learning rate live on the
device, so a captured step counts on when its graph is replayed."""
from __future__ import annotations

import torch

from . import ops


def _rows(t):
    """t as [rows, n] over its own memory, rows contiguous (a contiguous
    tensor is one row); None when it does not lie that way."""
    if t.is_contiguous():
        return t.view(1, t.numel())
    try:
        t = t.view(-1, t.shape[-1])
    except RuntimeError:
        return None
    return t if t.stride(1) == 1 and t.stride(0) >= t.shape[1] else None


class AdamW:
    def __init__(self, params, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, state_bits=32, seed=0):
        """params: list of (bf16 parameter, gradient) or (bf16 parameter,
        gradient, weight decay); the gradient is the buffer (bf16 or fp32)
        that every backward pass writes.  Both are read and written where
        they lie: contiguous, or in rows with padding between them (as a
        linear layer's weight of odd width has to; one table entry per row).
        The masters start as the parameters' values.  state_bits: 32, or 8
        (E4M3 codes with a scale per 256 elements, include/moe.h)."""
        if state_bits not in (32, 8):
            raise ValueError("state_bits: 32 or 8")
        entries = []
        for p, g, *wd in params:
            p = p.detach()
            rows = _rows(p), _rows(g)
            if p.shape != g.shape and not (p.is_contiguous() and g.is_contiguous()):
                raise ValueError(f"parameter {tuple(p.shape)} and gradient {tuple(g.shape)}")
            if rows[0] is None or rows[1] is None:
                raise ValueError("parameters and gradients: contiguous, or rows with unit stride")
            if p.dtype != torch.bfloat16 or g.dtype not in (torch.bfloat16, torch.float32):
                raise ValueError(f"parameter {p.dtype}, gradient {g.dtype}: bfloat16, and bfloat16 or float32")
            if rows[0].shape != rows[1].shape and p.shape == g.shape:      # one is contiguous, the other is not
                rows = p.view(-1, p.shape[-1]), g.view(-1, p.shape[-1])
            entries.append((*rows, float(wd[0]) if wd else float(weight_decay)))
        if not entries:
            raise ValueError("params: empty")
        dev = entries[0][0].device
        ops.moe_init(dev.index or 0)
        self.lr = torch.full((1,), float(lr), dtype=torch.float32, device=dev)
        self.betas, self.eps, self.seed = betas, eps, int(seed)
        self.masters, self.groups = [], []

        def padded(rows, n, dtype, to):
            """zeros [rows, n], several rows starting at multiples of `to` elements"""
            ld = n if rows == 1 else (n + to - 1) // to * to
            return torch.zeros((rows, ld), dtype=dtype, device=dev)[:, :n]

        def pieces(matrices):
            return None if matrices is None else [row for t in matrices for row in t.unbind(0)]

        counter = 0      # of the 8-bit rounding: every element of the optimizer has its own
        for dtype in (torch.bfloat16, torch.float32):
            mine = [e for e in entries if e[1].dtype == dtype]
            if not mine:
                continue
            shapes = [p.shape for p, _, _ in mine]
            masters = [padded(*s, torch.float32, 8).copy_(p) for s, (p, _, _) in zip(shapes, mine)]

            def state():
                if state_bits == 32:
                    return [padded(*s, torch.float32, 8) for s in shapes], None
                return ([padded(*s, torch.uint8, 16) for s in shapes],
                        [padded(s[0], (s[1] + 255) // 256, torch.float32, 4) for s in shapes])

            (m, ms), (v, vs) = state(), state()
            base = []
            for row in pieces(masters):
                base.append(counter)
                counter += (row.numel() + 255) // 256 * 256
            plan = ops.adamw_plan(pieces(masters), pieces([g for _, g, _ in mine]), pieces(m), pieces(v), pieces(ms),
                                  pieces(vs), copies=pieces([p for p, _, _ in mine]),
                                  weight_decay=[w for p, _, w in mine for _ in range(p.shape[0])], rng_base=base)
            self.masters += [t.view(-1) if len(t) == 1 else t for t in masters]
            self.groups.append((plan, torch.zeros((1,), dtype=torch.int32, device=dev)))

    def step_(self, grad_scale=None):
        """One update from the gradients in their buffers.  grad_scale: fp32
        device tensor, a factor of every gradient (not finite: no update)."""
        for plan, count in self.groups:
            ops.adamw_step(plan, self.lr, self.betas, self.eps, step=count, grad_scale=grad_scale, seed=self.seed)
