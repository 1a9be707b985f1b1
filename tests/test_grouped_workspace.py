"""The grouped products take a workspace as the dense operators do: no bytes are
needed, one may be given, and something else in its place is refused."""
import inspect

import pytest
import torch

from helpers import build_lib, gpu_ops

BF = torch.bfloat16
CALLS = ("grouped_linear_fwd", "grouped_linear_bwd", "grouped_ffn_fwd", "grouped_ffn_bwd")


@pytest.fixture
def host():
    """The calls on host memory, up to the library's own checks."""
    build_lib()
    from grouped_gemm_top_gb300 import _marshal, ops

    def setup(*device_and_stream):
        _marshal.setup(BF, torch.float32, torch.uint8, torch.float8_e4m3fn, torch.int32, *device_and_stream)

    setup(lambda: -1, lambda device: 0)
    yield ops
    setup(torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)


def calls(ops, x, dy, w, offsets, **k):
    """each call over f = N / 2"""
    n = w.shape[2] // 2
    return {"grouped_linear_fwd": lambda: ops.grouped_linear_fwd(x, w, offsets, **k),
            "grouped_linear_bwd": lambda: ops.grouped_linear_bwd(dy, x, w, offsets, **k),
            "grouped_ffn_fwd": lambda: ops.grouped_ffn_fwd(x, w, offsets, **k),
            "grouped_ffn_bwd": lambda: ops.grouped_ffn_bwd(dy[:, :n], dy, x, w, offsets, **k)}


def test_sizes(host):
    assert [host.grouped_workspace_size(g) for g in (1, 256, 65536)] == [0, 0, 0]
    assert [host.grouped_workspace_size(g) for g in (0, -1, 65537)] == [-1, -1, -1]
    for name in CALLS:
        assert inspect.signature(getattr(host, name)).parameters["ws"].default is None


@pytest.mark.parametrize("name", CALLS)
def test_taken_or_refused(host, name):
    x, dy, w = torch.zeros((0, 64), dtype=BF), torch.zeros((0, 48), dtype=BF), torch.zeros((3, 64, 48), dtype=BF)
    offsets = torch.zeros(4, dtype=torch.int32)

    def status(ws):
        try:
            calls(host, x, dy, w, offsets, ws=ws)[name]()
        except host.MoEError as e:
            return e.status
        return host.MOE_OK

    # (the backward calls write zeros to dw, for which there is no device here)
    past = host.MOE_OK if name.endswith("fwd") else host.MOE_ERR_NOT_INITIALIZED
    assert status(None) == past
    assert status(torch.empty((host.grouped_workspace_size(3),), dtype=torch.uint8)) == past
    for ws in (torch.empty((16,)), torch.empty((16,), dtype=torch.uint8, device="meta"), 4096):
        assert status(ws) == host.MOE_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_the_same_bits(name):
    ops = gpu_ops()
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy = (torch.randn((100, n), generator=g, device="cuda").to(BF) for n in (64, 48))
    w = torch.randn((3, 64, 48), generator=g, device="cuda").to(BF)
    offsets = torch.tensor([0, 33, 33, 100], dtype=torch.int32, device="cuda")
    ws = torch.empty((ops.grouped_workspace_size(3),), dtype=torch.uint8, device="cuda")
    p, q = (calls(ops, x, dy, w, offsets, ws=t)[name]() for t in (None, ws))
    for a, b in zip(p if isinstance(p, tuple) else (p,), q if isinstance(q, tuple) else (q,)):
        assert torch.equal(a, b)
