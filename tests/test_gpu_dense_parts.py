"""Dense products whose depth is split over the pairs of a cluster: every form
(tile width, parts) that some size reaches on this device, each product and
epilogue, against 64-bit products, and the same bits on every run.

Tolerances as in test_gpu_dense.py: the accumulators (K / 16 + 8) 2^-23 of the
sum of the terms' magnitudes (the 8 covers the additions of up to four parts),
2^-18 of what an activation handles, half a step of each bf16 store."""
import pytest
import torch

from helpers import gpu_ops

pytestmark = pytest.mark.gpu

HALF, WORK = 2.0 ** -8, 2.0 ** -18
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def reached(ops, product):
    """{(tile columns, parts): the cheapest (M, N, K) of a grid}, sizes made ragged."""
    gated, best = product == ops.MOE_DENSE_GATED, {}
    for m in (256, 300, 512, 1024, 2048, 4096):
        for n in list(range(64, 2048, 64)) + list(range(2048, 10240, 128)):
            for k in (512, 2048, 4096, 8192, 10752, 12288, 16384, 32768):
                size = (m - 7, n - (8 if gated else 3), k - 1)
                p = ops.moe_selftest_dense_plan(product, *size)
                if p.parts > 1:
                    key, cost = (p.tile_cols, p.parts), m * n * k
                    if key not in best or cost < best[key][0]:
                        best[key] = (cost, size)
    assert {parts for _, parts in best} == {2, 3, 4}
    return sorted((key, size) for key, (_, size) in best.items())


def mat(m, n, seed, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn((m, (n + 7) // 8 * 8 + 8), generator=g, device="cuda").mul_(std).to(dtype)
    buf[:, n:] = float("nan")             # nothing between the rows is used
    return buf[:, :n]


def acc(k):
    return (k / 16 + 8) * 2.0 ** -23


def product(a, b):
    """The 64-bit product and the sum of its terms' magnitudes."""
    return a.double() @ b.double(), a.double().abs() @ b.double().abs()


def close(got, want, tol, what):
    off = (got.double() - want).abs() - tol
    assert bool((off <= 1e-30).all()), (what, float(off.nan_to_num(1e30).max()))
    assert float((got.double() - want).norm()) <= HALF * float(want.norm()), what


def untouched(t):
    return bool(torch.isnan(t._base[:, t.shape[1]:]).all())


ACTS = {"none": lambda z: z, "relu": lambda z: z.clamp(min=0),
        "silu": lambda z: z / (1 + torch.exp(-z)),
        "gelu": lambda z: 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))}


def test_gated_forward(ops):
    for i, ((cols, parts), (m, f, d)) in enumerate(reached(ops, ops.MOE_DENSE_GATED)):
        what = (cols, parts, m, f, d)
        act = ("silu", "gelu", "relu", "none")[i % 4]
        x, w1 = mat(m, d, 1), mat(d, 2 * f, 2, d ** -0.5)
        h, a, err = mat(m, f, 3), mat(m, 2 * f, 4), torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.gated_ffn_fwd(x, w1, act, h=h, a=a, err=err)
        wa, size = product(x, w1)
        ea = acc(d) * size
        close(a, wa, ea + wa.abs() * HALF, ("a", what))
        g, u, eg, eu = wa[:, :f], wa[:, f:], ea[:, :f], ea[:, f:]
        wh = ACTS[act](g) * u
        close(h, wh, 1.2 * eg * (u.abs() + eu) + ACTS[act](g).abs() * eu + (g * u).abs() * WORK + wh.abs() * HALF, ("h", what))
        assert untouched(h) and untouched(a), what
        first = h.clone(), a.clone()
        for _ in range(8):
            assert torch.equal(ops.gated_ffn_fwd(x, w1, act, h=h), first[0]), what
            ops.gated_ffn_fwd(x, w1, act, h=h, a=a, err=err)
            assert torch.equal(h, first[0]) and torch.equal(a, first[1]), what
        assert int(err) == 0


def test_linear_forward(ops):
    for i, ((cols, parts), (m, n, k)) in enumerate(reached(ops, ops.MOE_DENSE_FWD)):
        what = (cols, parts, m, n, k)
        act = ("gelu", "silu", "none", "relu")[i % 4]
        x, w, b, r = mat(m, k, 1), mat(k, n, 2, k ** -0.5), mat(1, n, 3)[0], mat(m, n, 4)
        y, z, err = mat(m, n, 5), mat(m, n, 6), torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.linear_fwd(x, w, b, act, r, y=y, z=z, err=err)
        plain, size = product(x, w)
        wz = plain + b.double()
        ez = acc(k) * (size + b.double().abs())
        close(z, wz, ez + wz.abs() * HALF, ("z", what))
        wy = ACTS[act](wz) + r.double()
        work = 0 if act == "none" else wz.abs() * WORK
        close(y, wy, 1.2 * ez + work + r.double().abs() * 2.0 ** -22 + wy.abs() * (HALF + 2.0 ** -22), ("y", what))
        assert untouched(y) and untouched(z), what
        p = mat(m, n, 7)
        ops.linear_fwd(x, w, y=p, err=err)
        close(p, plain, acc(k) * size + plain.abs() * HALF, ("plain", what))
        assert untouched(p), what
        first = y.clone(), z.clone(), p.clone()
        for _ in range(4):
            ops.linear_fwd(x, w, b, act, r, y=y, z=z, err=err)
            ops.linear_fwd(x, w, y=p, err=err)
            assert all(torch.equal(s, t) for s, t in zip(first, (y, z, p))), what
        ops.linear_fwd(x, w, b, act, r, y=r, err=err)          # the residual's place
        assert torch.equal(r, first[0]) and int(err) == 0, what


def test_input_gradient(ops):
    """dx[M, K] = dy W^T alone; its depth is dy's width."""
    for (cols, parts), (m, k, n) in reached(ops, ops.MOE_DENSE_DGRAD):
        what = (cols, parts, m, k, n)
        dy, w, x, dx = mat(m, n, 1), mat(k, n, 2, n ** -0.5), mat(m, k, 3), mat(m, k, 4)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.linear_bwd(dy, x, w, want_dw=False, dx=dx, err=err)
        want, size = product(dy, w.t())
        close(dx, want, acc(n) * size + want.abs() * HALF, what)
        first = dx.clone()
        for _ in range(4):
            ops.linear_bwd(dy, x, w, want_dw=False, dx=dx, err=err)
            assert torch.equal(dx, first), what
        assert untouched(dx) and int(err) == 0, what


@pytest.mark.parametrize("dtype", [BF, F])
def test_weight_gradient(ops, dtype):
    """dw[K, N] = x^T dy alone; its depth is the number of rows."""
    for (cols, parts), (k, n, m) in reached(ops, ops.MOE_DENSE_WGRAD):
        what = (cols, parts, k, n, m)
        x, dy, w, dw = mat(m, k, 1), mat(m, n, 2, m ** -0.5), mat(k, n, 3), mat(k, n, 4, dtype=dtype)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.linear_bwd(dy, x, w, want_dx=False, dw=dw, err=err)
        want, size = product(x.t(), dy)
        close(dw, want, acc(m) * size + want.abs() * (HALF if dtype == BF else 0), what)
        first = dw.clone()
        for _ in range(4):
            ops.linear_bwd(dy, x, w, want_dx=False, dw=dw, err=err)
            assert torch.equal(dw, first), what
        assert untouched(dw) and int(err) == 0, what


def test_both_gradients_in_one_launch(ops):
    """Every tile width of the launch that computes dx and dw."""
    best = {}
    for m in (256, 300, 512, 1024, 2048, 4096, 8192):
        for n in (64, 320, 512, 1024, 1536, 2048, 4096, 7168):
            for k in (64, 320, 512, 1024, 1536, 2048, 4096):
                size = (m - 7, n - 3, k - 1)
                w = ops.moe_selftest_dense_plan(ops.MOE_DENSE_BACKWARD, *size).tile_cols
                if w and (w not in best or m * n * k < best[w][0]):
                    best[w] = (m * n * k, size)
    assert {64, 128, 256} <= set(best)
    for w, (_, (m, n, k)) in sorted(best.items()):
        for dtype in (BF, F):
            what = (w, m, n, k, dtype)
            dy, x, wt = mat(m, n, 1), mat(m, k, 2), mat(k, n, 3, n ** -0.5)
            dx, dw, err = mat(m, k, 4), mat(k, n, 5, dtype=dtype), torch.zeros(1, dtype=torch.int32, device="cuda")
            ops.linear_bwd(dy, x, wt, dx=dx, dw=dw, err=err)
            want, size = product(dy, wt.t())
            close(dx, want, acc(n) * size + want.abs() * HALF, ("dx", what))
            want, size = product(x.t(), dy)
            close(dw, want, acc(m) * size + want.abs() * (HALF if dtype == BF else 0), ("dw", what))
            first = dx.clone(), dw.clone()
            for _ in range(4):
                ops.linear_bwd(dy, x, wt, dx=dx, dw=dw, err=err)
                assert torch.equal(dx, first[0]) and torch.equal(dw, first[1]), what
            assert untouched(dx) and untouched(dw) and int(err) == 0, what


@pytest.mark.parametrize("m", [1, 13, 64, 128])
def test_few_rows_in_every_number_of_parts(ops, m):
    seen = {"f": set(), "g": set(), "d": set()}
    for k in (63, 511, 1023, 4095):
        for n in (120, 4099):
            what = (m, n, k)
            x, w, b, r, y, z = mat(m, k, 1), mat(k, n, 2, k ** -0.5), mat(1, n, 3)[0], mat(m, n, 4), mat(m, n, 5), mat(m, n, 6)
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            plain, size = product(x, w)
            wz, ez = plain + b.double(), acc(k) * (size + b.double().abs())
            wy = ACTS["gelu"](wz) + r.double()
            ops.linear_fwd(x, w, b, "gelu", r, y=y, z=z, err=err)
            close(z, wz, ez + wz.abs() * HALF, ("z", what))
            close(y, wy, 1.2 * ez + wz.abs() * WORK + r.double().abs() * 2.0 ** -22 + wy.abs() * (HALF + 2.0 ** -22), ("y", what))
            seen["f"].add(ops.moe_selftest_dense_plan(ops.MOE_DENSE_FWD, m, n, k).few_parts)
            f = n // 8 * 8
            w1, h, a = mat(k, 2 * f, 7, k ** -0.5), mat(m, f, 8), mat(m, 2 * f, 9)
            ops.gated_ffn_fwd(x, w1, h=h, a=a, err=err)
            wa, size = product(x, w1)
            ea = acc(k) * size
            close(a, wa, ea + wa.abs() * HALF, ("a", what))
            g, u, eg, eu = wa[:, :f], wa[:, f:], ea[:, :f], ea[:, f:]
            wh = ACTS["silu"](g) * u
            close(h, wh, 1.2 * eg * (u.abs() + eu) + ACTS["silu"](g).abs() * eu + (g * u).abs() * WORK + wh.abs() * HALF, ("h", what))
            seen["g"].add(ops.moe_selftest_dense_plan(ops.MOE_DENSE_GATED, m, f, k).few_parts)
            # the input gradient's depth is dy's width: n outputs from depth k
            dy, wt, dx = mat(m, k, 10), mat(n, k, 11, k ** -0.5), mat(m, n, 12)
            ops.linear_bwd(dy, mat(m, n, 13), wt, want_dw=False, dx=dx, err=err)
            want, size = product(dy, wt.t())
            close(dx, want, acc(k) * size + want.abs() * HALF, ("dx", what))
            seen["d"].add(ops.moe_selftest_dense_plan(ops.MOE_DENSE_DGRAD, m, n, k).few_parts)
            assert all(untouched(t) for t in (y, z, h, a, dx)) and int(err) == 0, what
    if m <= 13:
        assert all(s == {1, 2, 4, 8} for s in seen.values()), seen
