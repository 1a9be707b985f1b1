"""The compiled argument marshalling without a GPU: a stand-in for the current
device, calls that are refused or have nothing to do."""
import pytest
import torch

from helpers import build_lib


@pytest.fixture
def marshal():
    build_lib()
    from grouped_gemm_top_gb300 import _marshal, ops

    def setup(*device_and_stream):
        _marshal.setup(torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn, torch.int32, *device_and_stream)

    setup(lambda: 0, lambda device: 0)
    yield _marshal, ops
    setup(torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)


def test_a_plan_of_another_device_is_refused(marshal):
    m, ops = marshal

    def step(device, **k):
        table = torch.zeros(64, dtype=torch.int64)
        plan = ops.AdamWPlan(table, 1, 0, ops.MOE_TYPE_F32, ops.MOE_TYPE_F32, 32, ())      # no tiles: nothing to launch
        assert plan.args[1] == table.get_device()
        plan.args = (4096, device) + plan.args[2:]
        return ops.adamw_step(plan, 1e-3, step=1)

    for device in (1, 7, -1):
        with pytest.raises(ops.MoEError) as e:
            step(device)
        assert e.value.status == ops.MOE_ERR_INVALID_ARG, device
    try:
        step(0)
    except ops.MoEError as e:
        assert e.status == ops.MOE_ERR_NOT_INITIALIZED      # past the marshalling; the library has no device here


def test_a_python_error_is_raised_before_anything_else_is_looked_at(marshal):
    m, ops = marshal
    m.setup(torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn, torch.int32, lambda: -1, lambda device: 0)
    x, w = torch.zeros((4, 8)), torch.zeros(8)                 # host memory is "on" device -1
    with pytest.raises(TypeError):
        m.rmsnorm_residual_fwd(x, w, None, "eps", x[:3], None, None, None, None, 0, None)
    plan = (4096, -1, 1, 0, 1, 1, 32)
    with pytest.raises(OverflowError):
        m.adamw_step(*plan, 10 ** 400, 0.9, 0.999, 1e-8, x, None, 0, None)
    with pytest.raises(OverflowError):
        m.adamw_step(*plan, 1e-3, 0.9, 0.999, 1e-8, 10 ** 40, x, 0, None)
