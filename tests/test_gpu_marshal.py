"""The compiled argument marshalling of the dense operators: it holds on to
no object, refuses what does not fit, and turns misuse into Python errors."""
import sys

import pytest
import torch

from helpers import gpu_ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def bf(*shape):
    return torch.randn(shape, device="cuda").bfloat16()


def test_reference_counts_stay(ops):
    x, w, y, b = bf(4, 64), bf(64, 48), bf(4, 48), bf(48)
    nw, res, rstd = bf(64), bf(4, 64), torch.empty(4, device="cuda")
    codes, scales = torch.empty((128, 64), dtype=torch.uint8, device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda")
    h, a, dw1 = bf(4, 24), bf(4, 48), bf(64, 48)
    db, ws = torch.empty(48, device="cuda"), torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    p, g, m, v = (torch.zeros(300, device="cuda") for _ in range(4))
    lr, step = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = ops.adamw_plan([p], [g], [m], [v])
    side = torch.cuda.Stream()
    out = torch.empty((4, 64), dtype=torch.bfloat16, device="cuda")

    def calls():
        for st in (None, side):
            ops.rmsnorm_residual_fwd(x, nw, res, y=out, r=res, rstd=rstd, codes=None, scales=None, stream=st)
            ops.rmsnorm_residual_bwd(res, x, nw, rstd, res, dx=out, want_dw=False, stream=st)
            ops.linear_fwd(x, w, b, "silu", y, y=y, z=y, stream=st)
            ops.linear_bwd(y, x, w, y, "gelu", dx=out, dw=dw1, dbias=db, ws=ws, stream=st)
            ops.gated_ffn_fwd(x, w, h=h, a=a, stream=st)
            ops.gated_ffn_bwd(h, a, x, w, da=a, dx=out, dw1=dw1, stream=st)
            ops.adamw_step(plan, lr, step=step, grad_scale=lr, stream=st)
        for bad in (lambda: ops.linear_fwd(x.float(), w, y=y), lambda: ops.linear_fwd(x, w, b[:40], y=y),
                    lambda: ops.rmsnorm_residual_fwd(x, nw, res, y=out, r=res, rstd=rstd, codes=codes),
                    lambda: ops.rmsnorm_residual_fwd(x.cpu(), nw, rstd=rstd, want_y=False),
                    lambda: ops.adamw_step(plan, p, step=1)):
            with pytest.raises(ops.MoEError):
                bad()

    held = (x, w, y, b, nw, res, rstd, codes, scales, h, a, dw1, db, ws, lr, step, out, side, torch.bfloat16,
            torch.float32, torch.uint8, torch.int32, None, True, torch.Size)
    calls()
    torch.cuda.synchronize()
    before = [sys.getrefcount(o) for o in held]
    for _ in range(50):
        calls()
    torch.cuda.synchronize()
    after = [sys.getrefcount(o) for o in held]
    # (None, True and the dtypes are shared by everything else that runs: a leak would show 50 and more)
    assert all(abs(j - i) < 25 for i, j in zip(before, after)), list(zip(before, after))


def test_misuse_is_a_python_error(ops):
    from grouped_gemm_top_gb300 import _marshal
    x, w = bf(4, 64), bf(64, 48)
    with pytest.raises(TypeError):
        _marshal.linear_fwd(x, w)
    with pytest.raises(AttributeError):
        _marshal.linear_fwd(x, 7, None, 0, None, x, None, None, None)
    with pytest.raises(TypeError):
        _marshal.linear_fwd(x, w, None, "relu", None, x, None, None, None)
    with pytest.raises(AttributeError):
        ops.linear_fwd(x, w, y=bf(4, 48), stream="side")
    with pytest.raises(ops.MoEError):
        ops.linear_fwd(None, w)
    with pytest.raises(ops.MoEError):
        ops.linear_fwd(x[0], w)
    with pytest.raises(ops.MoEError):
        ops.rmsnorm_residual_fwd(x, None)
