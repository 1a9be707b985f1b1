"""8-bit states of tensors with more whole tiles than the ring of stages holds:
stages refilled and reused over several turns, whole tiles between ragged and
unaligned tensors in one CTA's share."""
import numpy as np
import pytest
import torch

from helpers import gpu_ops
from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu

LR, B1, B2, EPS, WD = 1e-3, 0.9, 0.999, 1e-8, 0.1
BF, F = torch.bfloat16, torch.float32
CTAS, STAGES = 4, 4                     # at most, of an SM and of a CTA


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def f64(t):
    return t.double().cpu().numpy()


def states(n, seed, off=0):
    """codes and scales of m, of v's root: [n + off] bytes from `off` on"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = (n + 255) // 256
    m = torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.int32)
    m = torch.where(m & 0x7F == 0x7F, m - 1, m).to(torch.uint8)          # (no NaN codes)
    v = torch.randint(1, 0x7F, (n,), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    ms = torch.rand((nb,), generator=g, device="cuda").add_(0.5).mul_(1e-6)
    vs = torch.rand((nb,), generator=g, device="cuda").add_(0.5).mul_(4e-6)
    return m, v, ms, vs


def shifted(t, off):
    """A copy that starts `off` elements into its memory."""
    out = torch.empty((t.numel() + off,), dtype=t.dtype, device="cuda")[off:]
    return out.copy_(t)


@pytest.mark.parametrize("pt,gt,copy", [(BF, BF, False), (F, BF, True), (F, F, False), (BF, F, True)])
def test_ring_over_many_turns(ops, pt, gt, copy):
    tile = 4096 if (pt, gt) == (BF, BF) else 2048
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    whole = sms * CTAS * (STAGES + 2)
    # long ones (each CTA's share: several whole tiles in a row), then a mixture
    sizes = [tile * (whole // 2 + 3), 3, tile * (whole // 2) + 77] + [tile * (1 + i % 3) + (0, 1, 255, 900)[i % 4] for i in range(300)]
    offs = [0, 0, 0] + [i % 5 == 4 for i in range(300)]                 # some start at odd addresses
    assert sum(n // tile for n, o in zip(sizes, offs) if not o) > whole
    g = torch.Generator(device="cuda").manual_seed(5)
    p0 = [torch.randn((n,), generator=g, device="cuda").mul_(0.02).to(pt) for n in sizes]
    g0 = [torch.randn((n,), generator=g, device="cuda").mul_(1e-3).to(gt) for n in sizes]
    s0 = [states(n, i) for i, n in enumerate(sizes)]
    base = np.concatenate([[0], np.cumsum([(n + 255) // 256 * 256 for n in sizes])]).tolist()

    def build(off):
        p = [shifted(t, o) for t, o in zip(p0, off)]
        gr = [shifted(t, o) for t, o in zip(g0, off)]
        m, v = ([shifted(s[j], o) for s, o in zip(s0, off)] for j in (0, 1))
        ms, vs = ([s[j].clone() for s in s0] for j in (2, 3))
        c = [torch.zeros((n + 8,), dtype=BF, device="cuda")[8 - 7 * o:][:n] for n, o in zip(sizes, off)] if copy else None
        return (p, m, v, ms, vs) + ((c,) if copy else ()), ops.adamw_plan(p, gr, m, v, ms, vs, copies=c, weight_decay=WD,
                                                                          rng_base=base[:-1])

    a, plan_a = build(offs)
    b, plan_b = build([1] * len(sizes))                 # the same with no tile in the ring
    for t in (1, 2, 3):
        if t == 3:
            old = [[x.clone() for x in lst] for lst in a]
        ops.adamw_step(plan_a, LR, (B1, B2), EPS, step=t, seed=11)
        ops.adamw_step(plan_b, LR, (B1, B2), EPS, step=t, seed=11)
        for x, y in zip(a, b):
            for i, (s, u) in enumerate(zip(x, y)):
                assert torch.equal(s, u), (t, i)
    # the last step against the definition: blocks of every tensor, spread over its tiles
    differ = total = 0
    for i, n in enumerate(sizes):
        nb = (n + 255) // 256
        blocks = np.unique(np.r_[0, nb - 1, np.arange(0, nb, max(nb // 40, 1))])
        at = np.concatenate([np.arange(k * 256, min((k + 1) * 256, n)) for k in blocks])
        pick = torch.from_numpy(at).cuda()
        dec = lambda codes, sc: f64(codes[pick].view(torch.float8_e4m3fn).float()) * f64(sc)[at // 256]  # noqa: E731
        p, m, v, ms, vs = (lst[i] for lst in old[:5])
        was = f64(p[pick]), f64(g0[i][pick]), dec(m, ms), dec(v, vs) ** 2
        wp, wm, wv = D.adamw(*was, 3, LR, B1, B2, EPS, WD)
        size = np.abs(was[0] * 0), np.abs(was[1]), np.abs(was[2]), was[3]
        upd = np.abs(D.adamw(*size, 3, LR, B1, B2, EPS, 0.0)[0])
        tol = np.abs(wp) * (2.0 ** -22 + (2.0 ** -8 if pt == BF else 0)) + upd * 2.0 ** -18 + np.abs(was[0]) * 2.0 ** -22
        assert np.all(np.abs(f64(a[0][i][pick]) - wp) <= tol), i
        if copy:
            assert torch.equal(a[5][i], a[0][i].to(BF)), i
        bits = D.dither_bits(at + base[i], 11, 3)
        for codes, scale, want, r in ((a[1][i], a[3][i], wm, bits & 0xFFFF), (a[2][i], a[4][i], np.sqrt(wv), bits >> 16)):
            top = np.zeros(nb)
            np.maximum.at(top, at // 256, np.abs(want))
            assert np.all(np.abs(f64(scale) - top / 448)[blocks] <= top[blocks] / 448 * 2.0 ** -20), i
            x = want / f64(scale)[at // 256]
            got = f64(codes[pick].view(torch.float8_e4m3fn).float())
            step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(x) * (1 + 2.0 ** -18), 1e-30))) - 3, -9))
            assert np.all(np.abs(got - x) <= step * (1 + 2.0 ** -10)), i
            differ += int(np.sum(got != D.e4m3_dither(x, r)))
            total += len(at)
    # (as in test_gpu_adamw.py: fp32 falls on the other side of a border for one in 2^16)
    assert differ <= 20 + total * 2.0 ** -12
