"""MoELayerBF16: the MoE layer in 16 bits -- the routing, permutation and
combine of MoELayer around the bf16 products grouped by expert, which take the
groups' real rows out of the padded layout:

    x_perm = permute(x),   h = silu(gate) * up, [gate | up] = x_perm W1   one kernel
    y_perm = h W2,         out = combine(y_perm)

For fine-tuning and for teachers in 16 bits, and as a reference for the MXFP8
layer.  Buffers and calls that it has in common with MoELayer mean the same; it
has no shared experts, row capacity of its own or steps from host inputs, its gate
is silu, and the forward pass always keeps what the backward pass needs (for
decoding call ops.grouped_ffn_fwd and grouped_linear_fwd themselves).  The step
allocates nothing, never synchronises and can be captured in a CUDA graph.  The
weights are read where they lie: nothing is derived from them."""
from __future__ import annotations

import torch

from . import ops

_SCORES = {"softmax": ops.MOE_SCORE_SOFTMAX, "sigmoid": ops.MOE_SCORE_SIGMOID}


def _as_operand(name, w, shape, device):
    """w as the grouped products read it where it lies, or a ValueError."""
    ok = (isinstance(w, torch.Tensor) and w.shape == shape and w.dtype == torch.bfloat16 and w.device == device and
          w.data_ptr() % 16 == 0)
    if ok:
        G, K, N = shape
        gs, ld, one = w.stride()
        ok = (one == 1 or N == 1) and (K == 1 or (ld >= N and ld % 8 == 0))
        ok = ok and (G == 1 or (gs >= (K - 1) * ld + N and gs % 8 == 0))
    if not ok:
        raise ValueError(f"{name}: bfloat16 {tuple(shape)} on {device}, rows at multiples of 16 bytes")
    return w


class MoELayerBF16:
    def __init__(self, T, d, E, k, f, score="softmax", normalize=True, device="cuda:0", router=False):
        """T tokens of width d (d % 8 == 0), E experts of width f (f % 8 == 0),
        top-k.  router: logits = x W_r (T % 128 == 0, E % 8 == 0), with its
        gradients, as in MoELayer."""
        if d % 8 or f % 8:
            raise ValueError("16-bit products: d % 8, f % 8")
        self.T, self.d, self.E, self.k, self.f = T, d, E, k, f
        self.score, self.normalize = _SCORES[score], bool(normalize)
        self.device = torch.device(device)
        ops.moe_init(self.device.index or 0)
        M = self.row_cap = ops.moe_row_capacity(T, E, k)

        def z(shape, dtype=torch.bfloat16):
            return torch.zeros(shape, dtype=dtype, device=self.device)

        self.logits, self.x, self.dout = z((T, E), torch.float32), z((T, d)), z((T, d))
        self.err = z((1,), torch.int32)
        self.topk_idx, self.topk_w = z((T, k), torch.int32), z((T, k), torch.float32)
        self.counts, self.offsets = z((E,), torch.int32), z((E + 1,), torch.int32)
        self.gofs, self.slot_of, self.row_id = z((E + 1,), torch.int32), z((T, k), torch.int32), z((M,), torch.int32)
        self.ws_route = z((ops.moe_route_workspace_size(T, E),), torch.uint8)
        self.ws_perm = z((ops.moe_permute_workspace_size(T, E),), torch.uint8)
        self.x_perm, self.h, self.y_perm, self.out = z((M, d)), z((M, f)), z((M, d)), z((T, d))
        # [gate | up], and their gradient (apart, so that backward_ can be repeated); a is the one
        # that was written last, by forward_ or backward_
        self.gate_up, self.da = z((M, 2 * f)), z((M, 2 * f))
        self.a = self.gate_up
        self.dy_perm, self.dh, self.dx_perm, self.dx = z((M, d)), z((M, f)), z((M, d)), z((T, d))
        self.dw, self.dlogits = z((T, k), torch.float32), z((T, E), torch.float32)
        self.W1 = self.W2 = None
        self.dW1, self.dW2 = z((E, d, 2 * f)), z((E, f, d))
        self.router = bool(router)
        if self.router:
            if T % 128 or d % 8 or E % 8:
                raise ValueError("router GEMMs: T % 128, d % 8, E % 8")
            self.Wr, self.WrT, self.xT = z((d, E)), z((E, d)), z((d, T))
            self.dlogitsT, self.dlogits_bf = z((E, T)), z((T, E))
            self.dx_r, self.dWr = z((T, d), torch.float32), z((d, E), torch.float32)

    def set_weights(self, W1, W2):
        """bf16 W1 [E, d, 2f] and W2 [E, f, d], rows at multiples of 16 bytes;
        they stay the caller's, and the steps read them where they lie."""
        W1 = _as_operand("W1", W1, self.dW1.shape, self.dW1.device)
        self.W1, self.W2 = W1, _as_operand("W2", W2, self.dW2.shape, self.dW2.device)

    def set_router_weights(self, Wr):
        self.Wr.copy_(Wr)
        ops.moe_transpose_bf16(self.Wr, self.WrT)

    def forward_(self):
        err = self.err
        if self.router:
            ops.gemm_bf16_nt(self.x, self.WrT, self.logits, err)
        ops.moe_route_topk(self.logits, self.k, self.score, self.normalize, self.topk_idx, self.topk_w, self.counts,
                           self.offsets, self.ws_route, err)
        ops.moe_permute(self.x, self.topk_idx, self.E, self.row_cap, self.gofs, self.slot_of, self.row_id, self.x_perm,
                        True, self.ws_perm, err)
        self.a = self.gate_up
        ops.grouped_ffn_fwd(self.x_perm, self.W1, self.gofs, self.counts, h=self.h, a=self.gate_up, err=err)
        ops.grouped_linear_fwd(self.h, self.W2, self.gofs, self.counts, y=self.y_perm, err=err)
        ops.moe_unpermute_combine(self.y_perm, self.slot_of, self.topk_w, self.out, err)

    def backward_(self):
        err = self.err
        ops.moe_combine_bwd(self.dout, self.y_perm, self.slot_of, self.topk_w, self.row_id, self.gofs, self.E,
                            self.dy_perm, self.dw, err)
        ops.grouped_linear_bwd(self.dy_perm, self.h, self.W2, self.gofs, self.counts, dx=self.dh, dw=self.dW2, err=err)
        self.a = self.da
        ops.grouped_ffn_bwd(self.dh, self.gate_up, self.x_perm, self.W1, self.gofs, self.counts, dx=self.dx_perm,
                            dw1=self.dW1, da=self.da, err=err)
        ops.moe_route_bwd(self.logits, self.topk_idx, self.dw, self.score, self.normalize, self.dlogits, err)
        if not self.router:
            ops.moe_unpermute_combine(self.dx_perm, self.slot_of, None, self.dx, err)
            return
        ops.moe_transpose_bf16(self.dlogits, self.dlogitsT)
        ops.moe_transpose_bf16(self.dlogitsT, self.dlogits_bf)
        ops.moe_transpose_bf16(self.x, self.xT)
        ops.gemm_bf16_nt(self.dlogits_bf, self.Wr, self.dx_r, err)
        ops.gemm_bf16_nt(self.xT, self.dlogitsT, self.dWr, err)
        ops.moe_unpermute_combine_add(self.dx_perm, self.slot_of, None, self.dx_r, self.dx, err)

    def step_(self):
        """One forward and backward pass over the resident inputs."""
        if self.W1 is None:
            raise RuntimeError("set_weights() first")
        self.forward_()
        self.backward_()

    def check_err(self):
        v = int(self.err.item())
        if v != 0:
            raise ops.MoEError("device", v)
