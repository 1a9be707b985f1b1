"""What the norm allocates at odd widths is what the linear layers take."""
import pytest
import torch

from helpers import gpu_ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [41, 4099])
@pytest.mark.parametrize("rtype", [torch.bfloat16, torch.float32])
def test_outputs_start_at_multiples_of_16_bytes(n, rtype):
    ops = gpu_ops()
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn((70, n), generator=g, device="cuda").bfloat16()
    res = torch.randn((70, n), generator=g, device="cuda").to(rtype)
    w = torch.ones((n,), device="cuda")
    y, r, rstd, _, _ = ops.rmsnorm_residual_fwd(x, w, res)
    dx, _ = ops.rmsnorm_residual_bwd(y, r, w, rstd)
    for t in (y, r, dx):
        assert t.shape == (70, n) and t.stride(0) * t.element_size() % 16 == 0 and t.data_ptr() % 16 == 0
    # the same values as in rows without padding
    y2, r2, dx2 = (torch.empty((70, n), dtype=t.dtype, device="cuda") for t in (y, r, dx))
    ops.rmsnorm_residual_fwd(x, w, res, y=y2, r=r2)
    ops.rmsnorm_residual_bwd(y, r, w, rstd, dx=dx2)
    assert torch.equal(y, y2) and torch.equal(r, r2) and torch.equal(dx, dx2)
    p = torch.randn((n, 48), generator=g, device="cuda").mul_(n ** -0.5).bfloat16()
    out = ops.linear_fwd(y, p)
    want = y.double() @ p.double()
    size = y.double().abs() @ p.double().abs()
    assert bool(((out.double() - want).abs() <= (n / 16 + 8) * 2.0 ** -23 * size + want.abs() * 2.0 ** -8).all())
