"""Which memory optim.AdamW takes for a parameter and its gradient: their own,
never a copy, or it says so."""
import pytest
import torch

from helpers import build_lib


@pytest.fixture(scope="module")
def optim():
    build_lib()
    from grouped_gemm_top_gb300 import optim
    return optim


def padded(m, n, pad=7, dtype=torch.bfloat16):
    return torch.zeros((m, n + pad), dtype=dtype)[:, :n]


def test_rows_are_the_tensors_own_memory(optim):
    cube = torch.zeros((3, 5, 16))[:, :, :9]
    for t, shape in ((torch.zeros(12), (1, 12)), (torch.zeros((3, 4)), (1, 12)), (torch.zeros(()), (1, 1)),
                     (torch.zeros((0, 4)), (1, 0)), (padded(5, 41), (5, 41)), (padded(1, 41), (1, 41)), (cube, (15, 9))):
        rows = optim._rows(t)
        assert tuple(rows.shape) == shape and rows.data_ptr() == t.data_ptr()
        assert all(r.is_contiguous() for r in rows.unbind(0))
        if t.numel():
            rows[-1, -1] = 5
            assert t.reshape(-1)[-1] == 5


def test_what_does_not_lie_in_rows_is_refused(optim):
    w = torch.zeros((4, 6), dtype=torch.bfloat16)
    for t in (w.t(), torch.zeros((4, 12), dtype=torch.bfloat16)[:, ::2], torch.zeros((1, 6)).expand(4, 6),
              torch.zeros((2, 4, 16))[:, :3, :5], torch.zeros(12)[::2]):
        assert optim._rows(t) is None
    for p, g in ((w.t(), w.t()), (w, torch.zeros((6, 4), dtype=torch.bfloat16).t()), (padded(4, 6), torch.zeros((6, 4)))):
        with pytest.raises(ValueError):
            optim.AdamW([(p, g)], 1e-3)


def test_types_that_no_plan_takes_are_refused(optim):
    """A gradient of another type has no plan and would never be applied."""
    w = torch.zeros((4, 8), dtype=torch.bfloat16)
    for p, g in ((w, w.half()), (w, w.double()), (w.float(), w), (w.half(), w)):
        with pytest.raises(ValueError):
            optim.AdamW([(w, w), (p, g)], 1e-3)
    with pytest.raises(ValueError):
        optim.AdamW([], 1e-3)


def test_every_element_has_its_own_rounding_counter(optim, monkeypatch):
    """Over the plans of both gradient types, padded rows among them."""
    plans = []

    def plan(params, grads, m, v, m_scales, v_scales, copies, weight_decay, rng_base=None):
        base = 0
        for i, t in enumerate(params):      # the default: one tensor after the other
            plans.append((base if rng_base is None else rng_base[i], t.numel()))
            base += (t.numel() + 255) // 256 * 256

    monkeypatch.setattr(optim.ops, "adamw_plan", plan)
    monkeypatch.setattr(optim.ops, "moe_init", lambda device: None)
    w = [torch.zeros(s, dtype=torch.bfloat16) for s in ((4, 300), (1000,), (512,), (3, 5))] + [padded(5, 41)]
    optim.AdamW([(t, torch.zeros_like(t, dtype=d)) for t, d in zip(w, [torch.float32, torch.bfloat16] * 3)], 1e-3,
                state_bits=8)
    assert len(plans) == 9 and all(b % 256 == 0 for b, _ in plans)
    taken = sorted((b, b + n) for b, n in plans)
    assert all(x[1] <= y[0] for x, y in zip(taken, taken[1:])), taken
