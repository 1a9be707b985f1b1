"""AdamW over many tensors, states in 32 and 8 bits, against the fp64 step.

Tolerances, from the roundings alone: fp32 chains of up to eight operations
(m, v: 2^-21 of the terms' sizes; the update lr m^ / (sqrt(v^) + eps): 2^-18 of
what it would be if the two terms of m did not cancel; p: 2^-22 of itself
besides); bf16 stores add 2^-8.  An 8-bit state is
rounded down or up, so it is less than one E4M3 step off."""
import numpy as np
import pytest
import torch

from helpers import gpu_ops
from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu

LR, B1, B2, EPS, WD = 1e-3, 0.9, 0.999, 1e-8, 0.1
BF, F = torch.bfloat16, torch.float32
SIZES = [1, 7, 8, 255, 256, 257, 2048, 2049, 0, 5000, 1, 100003]


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def f64(t):
    return t.double().cpu().numpy()


def rnd(n, seed, std=1.0, dtype=F, off=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((n + off,), generator=g, device="cuda").mul_(std).to(dtype)[off:]


def make(sizes, pt, gt, off=0, copy=False):
    p = [rnd(n, 10 + i, 0.02, pt, off) for i, n in enumerate(sizes)]
    g = [rnd(n, 50 + i, 1e-3, gt, off) for i, n in enumerate(sizes)]
    m = [rnd(n, 90 + i, 3e-4, F, off) for i, n in enumerate(sizes)]
    v = [rnd(n, 130 + i, 1e-3, F, off).square() for i, n in enumerate(sizes)]
    c = [torch.zeros((n + off,), dtype=BF, device="cuda")[off:] for n in sizes] if copy else None
    return p, g, m, v, c


def check_p(got, want, old, t, dtype):
    before, g, m, v = old
    size = np.abs(before * 0), np.abs(g), np.abs(m), v
    upd = np.abs(D.adamw(*size, t, LR, B1, B2, EPS, 0.0)[0])
    tol = np.abs(want) * (2.0 ** -22 + (2.0 ** -8 if dtype == BF else 0)) + upd * 2.0 ** -18 + np.abs(before) * 2.0 ** -22
    assert np.all(np.abs(f64(got) - want) <= tol)


@pytest.mark.parametrize("pt,gt,off,copy", [(F, F, 0, False), (F, BF, 0, True), (BF, BF, 0, False), (BF, F, 1, False),
                                            (F, BF, 3, True)])
def test_states_in_32_bits(ops, pt, gt, off, copy):
    p, g, m, v, c = make(SIZES, pt, gt, off, copy)
    wd = [WD if i % 2 else 0.0 for i in range(len(SIZES))]
    plan = ops.adamw_plan(p, g, m, v, copies=c, weight_decay=wd)
    for t in (1, 2, 1000):
        old = [[f64(a) for a in lst] for lst in (p, g, m, v)]
        ops.adamw_step(plan, LR, (B1, B2), EPS, step=t)
        for i in range(len(SIZES)):
            wp, wm, wv = D.adamw(*(o[i] for o in old), t, LR, B1, B2, EPS, wd[i])
            assert np.all(np.abs(f64(m[i]) - wm) <= (np.abs(old[2][i]) + np.abs(old[1][i])) * 2.0 ** -21)
            assert np.all(np.abs(f64(v[i]) - wv) <= (old[3][i] + old[1][i] ** 2) * 2.0 ** -21 + 1e-44)
            check_p(p[i], wp, [o[i] for o in old], t, pt)
            if c is not None:
                assert torch.equal(c[i], p[i].to(BF))


def decode(codes, scale):
    n = codes.numel()
    return f64(codes.view(torch.float8_e4m3fn).float()) * f64(scale).repeat(256)[:n]


def states8(sizes, seed=0):
    def one(std, s, pos):
        codes, scales = [], []
        for i, n in enumerate(sizes):
            t = rnd(n, s + i, std)
            t = t.abs() if pos else t
            pad = torch.nn.functional.pad(t, (0, -n % 256)).view(-1, 256)
            sc = pad.abs().amax(1) / 448 if n else pad.new_zeros((0,))
            q = torch.where(sc[:, None] > 0, pad / sc[:, None], 0.0).to(torch.float8_e4m3fn).view(-1)[:n]
            codes.append(q.view(torch.uint8).clone())
            scales.append(sc)
        return codes, scales
    return one(3e-4, 300 + seed, False) + one(1e-3, 400 + seed, True)


@pytest.mark.parametrize("pt,gt,copy", [(BF, BF, False), (F, BF, True), (F, F, False)])
def test_states_in_8_bits(ops, pt, gt, copy):
    p, g, _, _, c = make(SIZES, pt, gt, 0, copy)
    m, ms, v, vs = states8(SIZES)
    plan = ops.adamw_plan(p, g, m, v, ms, vs, copies=c, weight_decay=WD)
    base = np.concatenate([[0], np.cumsum([(n + 255) // 256 * 256 for n in SIZES])])
    for t in (7, 8):
        old = [(f64(p[i]), f64(g[i]), decode(m[i], ms[i]), decode(v[i], vs[i]) ** 2) for i in range(len(SIZES))]
        ops.adamw_step(plan, LR, (B1, B2), EPS, step=t, seed=99)
        differ = total = 0
        for i, n in enumerate(SIZES):
            if n == 0:
                continue
            wp, wm, wv = D.adamw(*old[i], t, LR, B1, B2, EPS, WD)
            check_p(p[i], wp, old[i], t, pt)
            bits = D.dither_bits(np.arange(n) + base[i], 99, t)
            for codes, scale, want, b in ((m[i], ms[i], wm, bits & 0xFFFF), (v[i], vs[i], np.sqrt(wv), bits >> 16)):
                pad = np.pad(np.abs(want), (0, -n % 256)).reshape(-1, 256)
                top = pad.max(1)
                assert np.all(np.abs(f64(scale) - top / 448) <= top / 448 * 2.0 ** -20)
                sc = f64(scale).repeat(256)[:n]
                x = want / sc
                got = f64(codes.view(torch.float8_e4m3fn).float())
                step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(x) * (1 + 2.0 ** -18), 1e-30))) - 3, -9))
                assert np.all(np.abs(got - x) <= step * (1 + 2.0 ** -10))
                differ += int(np.sum(got != D.e4m3_dither(x, b)))
                total += n
        # the same codes as the definition's, but where fp32 falls on the other side of a border:
        # an error of 2^-20 of a value of up to 16 steps moves one in 2^16 of them
        assert differ <= 20 + total * 2.0 ** -12


def test_8_bit_rounding_keeps_the_mean_and_v_moves(ops):
    """States decay by b a step, far below half a code; the mean over many
    equal elements follows all the same (each block's largest element stays
    what it is, and the scale with it).  The same call gives the same codes."""
    n = 1 << 18
    p, g = torch.zeros((n,), device="cuda"), torch.zeros((n,), device="cuda")
    m, v = torch.full((n,), 0x40, dtype=torch.uint8, device="cuda"), torch.full((n,), 0x44, dtype=torch.uint8, device="cuda")
    m[::256], v[::256], g[::256] = 0x7E, 0x7E, 448.0
    ms, vs = torch.ones((n // 256,), device="cuda"), torch.ones((n // 256,), device="cuda")
    plan = ops.adamw_plan([p], [g], [m], [v], [ms], [vs])
    twin = [t.clone() for t in (m, v)], [t.clone() for t in (ms, vs)]
    ops.adamw_step(plan, 0.0, (0.99, 0.999), EPS, step=3, seed=5)
    for codes, scale, code, b in ((m, ms, 2.0, 0.99), (v, vs, 3.0, 0.999 ** 0.5)):
        val = decode(codes, scale).reshape(-1, 256)[:, 1:]
        # steps of E4M3 are 1/8 and 1/4 here, so one code's deviation is at most 1/8, that of the mean of
        # 2^18 of them 2^-12
        assert abs(val.mean() - code * b) <= 6 * 2.0 ** -12 + 1e-6
        kept = f64(codes.view(torch.float8_e4m3fn).float()).reshape(-1, 256)[:, 1:] == code
        assert 0 < np.mean(kept) < 1
        assert np.all(np.abs(f64(scale) - 1) < 1e-6)
    plan2 = ops.adamw_plan([p.clone()], [g], [twin[0][0]], [twin[0][1]], [twin[1][0]], [twin[1][1]])
    ops.adamw_step(plan2, 0.0, (0.99, 0.999), EPS, step=3, seed=5)
    assert torch.equal(m, twin[0][0]) and torch.equal(v, twin[0][1])


def test_8_bit_second_moment_is_never_rounded_to_zero(ops):
    n = 512
    g = torch.zeros((n,), device="cuda")
    g[0], g[1:128], g[128:256], g[256:] = 1.0, 1e-9, 1e-15, 0.0
    m, v = (torch.zeros((n,), dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = torch.zeros((2,), device="cuda"), torch.zeros((2,), device="cuda")
    p = torch.zeros((n,), device="cuda")
    plan = ops.adamw_plan([p], [g], [m], [v], [ms], [vs])
    for t in (1, 2, 3):
        ops.adamw_step(plan, LR, (B1, B2), EPS, step=t)
        assert torch.isfinite(p).all() and p.abs().max() <= 4 * LR
    assert (v[:256] > 0).all() and not v[256:].any() and vs[1] == 0 and ms[1] == 0


def test_device_step_lr_scale_and_graph(ops):
    """Step count and learning rate on the device, gradient scale, a graph
    that counts on, and the step that is not taken."""
    def fresh():
        p, g, m, v, _ = make([300, 4096, 10001], F, BF)
        return p, g, m, v, ops.adamw_plan(p, g, m, v, weight_decay=WD)
    a, b = fresh(), fresh()
    step = torch.zeros((1,), dtype=torch.int32, device="cuda")
    lr = torch.full((1,), LR, device="cuda")
    scale = torch.full((1,), 0.5, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.adamw_step(a[4], lr, (B1, B2), EPS, step=step, grad_scale=scale)
    for t in (1, 2, 3):
        graph.replay()
        ops.adamw_step(b[4], LR, (B1, B2), EPS, step=t, grad_scale=scale)
        torch.cuda.synchronize()
        assert int(step) == t
        for x, y in zip(a[0] + a[2] + a[3], b[0] + b[2] + b[3]):
            assert np.all(np.abs(f64(x) - f64(y)) <= np.abs(f64(y)) * 2.0 ** -22 + LR * 2.0 ** -18)
    keep = [t.clone() for t in a[0] + a[2] + a[3]]
    for bad in (float("nan"), float("inf"), float("-inf")):
        scale.fill_(bad)
        graph.replay()
    torch.cuda.synchronize()
    assert int(step) == 3 and all(torch.equal(x, y) for x, y in zip(keep, a[0] + a[2] + a[3]))


def test_many_tensors(ops):
    sizes = [(i * 37) % 700 for i in range(500)]
    p, g, m, v, _ = make(sizes, F, F)
    old = [[f64(t) for t in lst] for lst in (p, g, m, v)]
    ops.adamw_step(ops.adamw_plan(p, g, m, v, weight_decay=WD), LR, (B1, B2), EPS, step=4)
    for i in range(0, len(sizes), 7):
        check_p(p[i], D.adamw(*(o[i] for o in old), 4, LR, B1, B2, EPS, WD)[0], [o[i] for o in old], 4, F)


def test_refusals(ops):
    p, g, m, v, _ = make([256, 300], F, BF)

    def refused(status, fn, *a, **k):
        with pytest.raises(ops.MoEError) as e:
            fn(*a, **k)
        assert e.value.status == status

    bad = ops.MOE_ERR_INVALID_ARG
    refused(bad, ops.adamw_plan, [], [], [], [])
    refused(bad, ops.adamw_plan, p, g[:1], m, v)
    refused(bad, ops.adamw_plan, [t.cpu() for t in p], g, m, v)
    refused(bad, ops.adamw_plan, p, g, m, [v[0], v[1][:299]])
    refused(bad, ops.adamw_plan, [t.half() for t in p], g, m, v)
    refused(bad, ops.adamw_plan, [p[0], torch.zeros((600,), device="cuda")[::2]], g, m, v)
    u = [torch.zeros((n,), dtype=torch.uint8, device="cuda") for n in (256, 300)]
    s = [torch.zeros((n,), device="cuda") for n in (1, 2)]
    refused(bad, ops.adamw_plan, p, g, u, u)
    refused(bad, ops.adamw_plan, p, g, u, u, s, [s[0], s[0]])
    refused(bad, ops.adamw_plan, p, g, u, u, s, s, rng_base=[0, 100])
    plan = ops.adamw_plan(p, g, m, v)
    refused(bad, ops.adamw_step, plan, LR, step=0)
    refused(bad, ops.adamw_step, plan, LR, betas=(1.0, 0.9))
    refused(bad, ops.adamw_step, plan, LR, eps=-1e-8)
    refused(bad, ops.adamw_step, plan, torch.zeros((1,)), step=1)


def test_whole_tiles_partial_tiles_and_odd_addresses_in_one_plan(ops):
    """Tensors of many whole tiles of 2,048 elements (which come through the
    ring) between small, ragged and unaligned ones."""
    sizes = [2048 * 700, 3, 2048 * 3 + 1, 100, 2048, 4095, 2048 * 50 + 2047, 7]
    offs = [0, 0, 0, 1, 0, 3, 0, 0]
    mk = lambda s, std, dt: [rnd(n, s + i, std, dt, o) for i, (n, o) in enumerate(zip(sizes, offs))]  # noqa: E731
    p, g, m = mk(10, 0.02, F), mk(50, 1e-3, BF), mk(90, 3e-4, F)
    v = [t.square() if o == 0 else torch.cat([t.new_zeros(o), t.square()])[o:] for t, o in zip(mk(130, 1e-3, F), offs)]
    plan = ops.adamw_plan(p, g, m, v, weight_decay=WD)
    for t in (1, 2):
        old = [[f64(a) for a in lst] for lst in (p, g, m, v)]
        ops.adamw_step(plan, LR, (B1, B2), EPS, step=t)
        for i in range(len(sizes)):
            o = [x[i] for x in old]
            wp, wm, wv = D.adamw(*o, t, LR, B1, B2, EPS, WD)
            assert np.all(np.abs(f64(m[i]) - wm) <= (np.abs(o[2]) + np.abs(o[1])) * 2.0 ** -21)
            assert np.all(np.abs(f64(v[i]) - wv) <= (o[3] + o[1] ** 2) * 2.0 ** -21 + 1e-44)
            check_p(p[i], wp, o, t, F)


@pytest.mark.parametrize("bits", [32, 8])
def test_non_finite_gradients_stay_with_their_elements(ops, bits):
    """NaN and infinite gradients, and one whose square overflows, in one
    block of one tensor (8 bits: its block's states are lost with it)."""
    n = 4096 + 300
    p, g = rnd(n, 1, 0.02), rnd(n, 2, 1e-3)
    g[5], g[300], g[4100] = float("nan"), float("inf"), 1e25
    keep = p.clone()
    if bits == 32:
        st = [torch.zeros((n,), device="cuda") for _ in range(2)]
        plan = ops.adamw_plan([p], [g], [st[0]], [st[1]])
    else:
        nb = (n + 255) // 256
        st = [torch.zeros((n,), dtype=torch.uint8, device="cuda") for _ in range(2)]
        plan = ops.adamw_plan([p], [g], [st[0]], [st[1]], [torch.zeros((nb,), device="cuda")], [torch.zeros((nb,), device="cuda")])
    ops.adamw_step(plan, LR, (B1, B2), EPS, step=1)
    bad = torch.zeros((n,), dtype=torch.bool, device="cuda")
    bad[[5, 300]] = True
    assert torch.isnan(p[bad]).all() and torch.isfinite(p[~bad]).all()
    assert p[4100] == keep[4100]                   # m / sqrt(inf) = 0
    zero = torch.zeros_like(keep)
    fine = ~bad
    fine[4100] = False
    want = D.adamw(f64(keep), f64(g), f64(zero), f64(zero), 1, LR, B1, B2, EPS, 0.0)[0]
    f = fine.cpu().numpy()
    assert np.all(np.abs(f64(p)[f] - want[f]) <= 2.0 ** -21 * np.abs(want[f]) + LR * 2.0 ** -18)
