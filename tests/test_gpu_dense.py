"""The dense bf16 layers (linear, gated feed-forward) and their backward
passes against the fp64 definitions.

Tolerances, from the roundings alone: the tensor core adds 16 products at a
time to an fp32 accumulator, so a product over K is off by at most
(K / 16 + 8) 2^-23 of the sum of its terms' magnitudes; the activations' fp32
work by 2^-18 of the magnitudes it handles, and their slopes are below 1.2;
each bf16 store by half a step, 2^-8 of the value.  Rounded operands of the
backward products (da, dz) pass their half step on through the sum of the magnitudes.
Besides, the Frobenius norm of the error of results of 256 elements and more
stays below 2^-8 of the result's (two independent roundings of 2^-8 / sqrt(3)
at most each)."""
import numpy as np
import pytest
import torch

from helpers import gpu_ops
from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu

HALF, WORK = 2.0 ** -8, 2.0 ** -18
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def up8(n):
    return (n + 7) // 8 * 8


def mat(m, n, seed, std=1.0, pad=0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn((m, up8(n) + pad), generator=g, device="cuda").mul_(std).to(dtype)
    buf[:, n:] = float("nan")             # nothing between the rows is used
    return buf[:, :n]


def f64(t):
    return t.double().cpu().numpy()


def acc(k):
    return (k / 16 + 8) * 2.0 ** -23


def close(got, want, tol, what=""):
    g = f64(got)
    assert np.all(np.isfinite(g)), what
    off = np.abs(g - want) - tol
    assert np.all(off <= 1e-30), (what, float(off.max()), np.argwhere(off > 0)[:3].tolist())
    n = np.linalg.norm(want)
    if want.size >= 256:
        assert np.linalg.norm(g - want) <= HALF * n, (what, np.linalg.norm(g - want) / n)


def linear_tol(x, w, b, act, res, want, z):
    size = np.abs(x) @ np.abs(w) + (0 if b is None else np.abs(b))
    t = 1.2 * acc(x.shape[1]) * size + np.abs(want) * (HALF + 2.0 ** -22) + (np.abs(z) * WORK if act != "none" else 0)
    return t if res is None else t + np.abs(res) * 2.0 ** -22


# (M, N, K): one tile, ragged everywhere, several tiles per pair, one row, one column, one deep
SIZES = [(256, 256, 64), (1, 1, 1), (1, 4096, 256), (3, 257, 65), (16, 520, 1000), (127, 128, 129), (255, 300, 8),
         (257, 513, 777), (200, 1030, 900), (384, 520, 1000), (1000, 1001, 130), (2049, 264, 4099), (5000, 4100, 70), (64, 24, 14336)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_plain(ops, m, n, k):
    x, w = mat(m, k, 1), mat(k, n, 2, 0.05)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ops.linear_fwd(x, w, err=err)
    want, z = D.linear(f64(x), f64(w))
    close(y, want, linear_tol(f64(x), f64(w), None, "none", None, want, z))
    assert int(err) == 0


@pytest.mark.parametrize("m,n,k", [(1, 300, 100), (5, 4096, 512), (300, 513, 200), (1025, 776, 96)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("bias,res", [(True, False), (False, True), (True, True)])
def test_linear_epilogue(ops, m, n, k, act, bias, res):
    x, w = mat(m, k, 1, pad=8), mat(k, n, 2, 0.1, pad=16)
    b = mat(1, n, 3)[0] if bias else None
    r = mat(m, n, 4, pad=24) if res else None
    out = mat(m, n, 5, pad=8)
    y, z = ops.linear_fwd(x, w, b, act, r, y=out, want_z=True)
    bn, rn = (f64(b) if bias else None), (f64(r) if res else None)
    want, wz = D.linear(f64(x), f64(w), bn, act, rn)
    close(y, want, linear_tol(f64(x), f64(w), bn, act, rn, want, wz), "y")
    close(z, wz, linear_tol(f64(x), f64(w), bn, "none", None, wz, wz), "z")
    base = out._base
    assert torch.isnan(base[:, n:]).all()                 # nothing between the rows is written
    if res:                                               # residual in place
        y2 = ops.linear_fwd(x, w, b, act, r, y=r)
        assert torch.equal(y2, y)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("act,dw_dtype", [("none", BF), ("silu", BF), ("gelu", F), ("relu", F)])
def test_linear_backward(ops, m, n, k, act, dw_dtype):
    x, w, dy = mat(m, k, 1, pad=8), mat(k, n, 2, 0.05), mat(m, n, 3, pad=16)
    z = mat(m, n, 4, pad=8) if act != "none" else None
    dx, dw, db = ops.linear_bwd(dy, x, w, z, act, want_dbias=True, dw_dtype=dw_dtype)
    wdx, wdw, wdb, dz = D.linear_bwd(f64(dy), f64(x), f64(w), None if z is None else f64(z), act)
    slack = np.abs(f64(dy)) * WORK
    rnd = (0 if act == "none" else HALF * np.abs(dz)) + (0 if act == "none" else slack)
    aw, ax = np.abs(f64(w)), np.abs(f64(x))
    close(dx, wdx, np.abs(wdx) * HALF + (rnd + acc(n) * np.abs(dz) + 0 * dz) @ aw.T, "dx")
    close(dw, wdw, np.abs(wdw) * (HALF if dw_dtype == BF else 0) + ax.T @ (rnd + acc(m) * np.abs(dz)), "dw")
    # a column's sum: at most m / (8 * parts) + 8 + parts / 32 + 8 additions in a chain
    tol = (m / 8 / min(-(-m // 32), 256) + 32) * 2.0 ** -24 * np.sum(np.abs(dz), 0) + np.sum(slack, 0)
    assert np.all(np.abs(f64(db) - wdb) <= tol)
    again = ops.linear_bwd(dy, x, w, z, act, want_dbias=True, dw_dtype=dw_dtype)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1]) and torch.equal(db, again[2])


@pytest.mark.parametrize("m,n,k", [(300, 520, 1000), (1000, 1001, 130), (130, 136, 5000)])
@pytest.mark.parametrize("dw_dtype", [BF, F])
def test_linear_backward_one_gradient(ops, m, n, k, dw_dtype):
    x, w, dy = mat(m, k, 1), mat(k, n, 2, 0.05, pad=8), mat(m, n, 3)
    wdx, wdw, _, dz = D.linear_bwd(f64(dy), f64(x), f64(w), None, "none")
    dx, none, _ = ops.linear_bwd(dy, x, w, want_dw=False)
    assert none is None
    close(dx, wdx, np.abs(wdx) * HALF + acc(n) * (np.abs(dz) @ np.abs(f64(w)).T), "dx")
    none, dw, _ = ops.linear_bwd(dy, x, w, want_dx=False, dw_dtype=dw_dtype)
    assert none is None
    close(dw, wdw, np.abs(wdw) * (HALF if dw_dtype == BF else 0) + acc(m) * (np.abs(f64(x)).T @ np.abs(dz)), "dw")


@pytest.mark.parametrize("n", list(range(1, 35)) + [63, 121, 127, 250, 253, 287])
def test_every_width_of_the_last_columns(ops, n):
    m, k = 400, 72
    x, w, b, r = mat(m, k, 1, pad=8), mat(k, n, 2, 0.1), mat(1, n, 3)[0], mat(m, n, 4)
    out = mat(m, n, 5, pad=8)
    y, z = ops.linear_fwd(x, w, b, "relu", r, y=out, want_z=True)
    want, wz = D.linear(f64(x), f64(w), f64(b), "relu", f64(r))
    close(y, want, linear_tol(f64(x), f64(w), f64(b), "relu", f64(r), want, wz), "y")
    close(z, wz, linear_tol(f64(x), f64(w), f64(b), "none", None, wz, wz), "z")
    assert torch.isnan(out._base[:, n:]).all()
    for dtype in (BF, F):
        dw = torch.full((m, up8(n) + 8), float("nan"), dtype=dtype, device="cuda")
        ops.linear_bwd(mat(k, n, 6), mat(k, m, 7), mat(m, n, 8), want_dx=False, dw=dw[:, :n])
        g, h = f64(mat(k, m, 7)).T, f64(mat(k, n, 6))
        close(dw[:, :n], g @ h, np.abs(g @ h) * (HALF if dtype == BF else 0) + acc(k) * (np.abs(g) @ np.abs(h)), "dw")
        assert torch.isnan(dw[:, n:]).all()


# (M, f, d)
GLU_SIZES = [(1, 8, 1), (1, 4096, 256), (4, 520, 1000), (128, 128, 64), (130, 136, 129), (257, 264, 777),
             (1000, 1000, 65), (2049, 128, 2050), (33, 3000, 72)]


@pytest.mark.parametrize("m,f,d", GLU_SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_ffn_forward(ops, m, f, d, act):
    x, w1 = mat(m, d, 1, pad=8), mat(d, 2 * f, 2, 0.1, pad=8)
    h, a = ops.gated_ffn_fwd(x, w1, act, want_a=True)
    wh, wa = D.gated_ffn(f64(x), f64(w1), act)
    ea = acc(d) * (np.abs(f64(x)) @ np.abs(f64(w1)))
    close(a, wa, ea + np.abs(wa) * HALF, "a")
    g, u = wa[:, :f], wa[:, f:]
    tol = 1.2 * ea[:, :f] * (np.abs(u) + ea[:, f:]) + np.abs(D.act(g, act)) * ea[:, f:] + np.abs(g * u) * WORK + np.abs(wh) * HALF
    close(h, wh, tol, "h")
    assert torch.equal(ops.gated_ffn_fwd(x, w1, act), h)


@pytest.mark.parametrize("m,f,d", GLU_SIZES)
@pytest.mark.parametrize("act,dw_dtype", [("silu", BF), ("gelu", F), ("relu", BF)])
def test_gated_ffn_backward(ops, m, f, d, act, dw_dtype):
    x, w1, dh, a = mat(m, d, 1, pad=8), mat(d, 2 * f, 2, 0.1), mat(m, f, 3, pad=8), mat(m, 2 * f, 4, pad=16)
    wdx, wdw, wda = D.gated_ffn_bwd(f64(dh), f64(a), f64(x), f64(w1), act)
    size = np.concatenate([np.abs(f64(dh) * f64(a)[:, f:]), np.abs(f64(dh) * f64(a)[:, :f])], 1)
    rnd = np.abs(wda) * HALF + size * WORK * 2
    dx, dw1 = ops.gated_ffn_bwd(dh, a, x, w1, act, dw_dtype=dw_dtype)
    close(dx, wdx, np.abs(wdx) * HALF + (rnd + acc(2 * f) * np.abs(wda)) @ np.abs(f64(w1)).T, "dx")
    close(dw1, wdw, np.abs(wdw) * (HALF if dw_dtype == BF else 0) +
          np.abs(f64(x)).T @ (rnd + acc(m) * np.abs(wda)), "dw1")
    dx2, dw2 = ops.gated_ffn_bwd(dh, a, x, w1, act, da=a, dw_dtype=dw_dtype)          # da in a's place
    assert torch.equal(dx, dx2) and torch.equal(dw1, dw2)
    close(a, wda, rnd, "da")


def test_gradients_against_differences(ops):
    """The kernels' gradients against central differences of the fp64
    definitions: the bf16 roundings of the operands and results bound how
    near they come (2^-6 of the gradient's largest element)."""
    m, f, d = 5, 16, 24
    x, w1, dh = mat(m, d, 1), mat(d, 2 * f, 2, 0.3), mat(m, f, 3)
    _, a = ops.gated_ffn_fwd(x, w1, want_a=True)
    dx, dw = ops.gated_ffn_bwd(dh, a, x, w1)
    loss = lambda p, q: float(np.sum(D.gated_ffn(p, q)[0] * f64(dh)))  # noqa: E731
    h = 1e-5
    for grad, at in ((dx, 0), (dw, 1)):
        args = [f64(x), f64(w1)]
        for i, j in [(0, 0), (2, 7), (4, 23)]:
            e = np.zeros_like(args[at])
            e[i, j] = h
            up, dn = list(args), list(args)
            up[at], dn[at] = args[at] + e, args[at] - e
            assert abs((loss(*up) - loss(*dn)) / (2 * h) - float(grad[i, j])) <= 2.0 ** -6 * float(grad.abs().max())


def test_no_rows(ops):
    x, w = torch.empty((0, 64), dtype=BF, device="cuda"), mat(64, 48, 1)
    assert ops.linear_fwd(x, w).shape == (0, 48)
    dy = torch.empty((0, 48), dtype=BF, device="cuda")
    dw, db = torch.ones((64, 48), dtype=BF, device="cuda"), torch.ones((48,), device="cuda")
    dx, dw, db = ops.linear_bwd(dy, x, w, z=dy, act="silu", dw=dw, dbias=db)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    h, a = ops.gated_ffn_fwd(x, w, want_a=True)
    assert h.shape == (0, 24)
    dx, dw = ops.gated_ffn_bwd(h, a, x, w, dw_dtype=F)
    assert dx.shape == (0, 64) and not dw.any()


def test_non_finite_values_stay_in_their_rows(ops):
    m, n, k = 300, 520, 200
    x, w = mat(m, k, 1), mat(k, n, 2, 0.1)
    want = ops.linear_fwd(x, w, act="silu")
    x[7, 3], x[260, 199] = float("nan"), float("inf")
    y = ops.linear_fwd(x, w, act="silu")
    keep = [i for i in range(m) if i not in (7, 260)]
    assert torch.isnan(y[7]).all() and not torch.isfinite(y[260]).any()
    assert torch.equal(y[keep], want[keep])


def test_stream_and_graph(ops):
    m, f, d = 200, 264, 136
    x, w1, dh, w2 = mat(m, d, 1), mat(d, 2 * f, 2, 0.1), mat(m, f, 3), mat(f, d, 4, 0.1)

    def step(stream=None, **o):
        h, a = ops.gated_ffn_fwd(x, w1, want_a=True, stream=stream, h=o.get("h"), a=o.get("a"))
        y = ops.linear_fwd(h, w2, residual=x, stream=stream, y=o.get("y"))
        dx, dw1 = ops.gated_ffn_bwd(dh, a, x, w1, stream=stream, dx=o.get("dx"), dw1=o.get("dw1"), da=o.get("da"))
        gx, gw, gb = ops.linear_bwd(y, h, w2, want_dbias=True, stream=stream, dx=o.get("gx"), dw=o.get("gw"), dbias=o.get("gb"),
                                    ws=o.get("ws"))
        return dict(h=h, a=a, y=y, dx=dx, dw1=dw1, gx=gx, gw=gw, gb=gb)

    base = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(base[k], other[k]) for k in base)
    outs = {k: torch.zeros_like(v) for k, v in base.items()}
    extra = dict(da=torch.empty_like(base["a"]),
                 ws=torch.empty((ops.linear_bwd_workspace_size(m, d),), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(**outs, **extra)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(base[k], outs[k]) for k in base)


def test_refusals(ops):
    x, w = mat(16, 64, 1), mat(64, 48, 2)

    def refused(status, fn, *a, **k):
        with pytest.raises(ops.MoEError) as e:
            fn(*a, **k)
        assert e.value.status == status

    bad, ali = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_ALIGNMENT
    refused(bad, ops.linear_fwd, x.cpu(), w)
    refused(bad, ops.linear_fwd, x.float(), w)
    refused(bad, ops.linear_fwd, x, w[:60])
    refused(bad, ops.linear_fwd, x, w, mat(1, 40, 3)[0])
    refused(bad, ops.linear_fwd, x, w, act="tanh")
    refused(bad, ops.linear_fwd, x, w, act=7)
    refused(bad, ops.linear_fwd, x, w.t().contiguous().t())
    refused(bad, ops.linear_fwd, x, w, residual=x)
    refused(ali, ops.linear_fwd, torch.zeros((4, 65), dtype=BF, device="cuda")[:, :64], w)
    refused(ali, ops.linear_fwd, torch.zeros((4, 72), dtype=BF, device="cuda")[:, 1:65], w)
    dy = mat(16, 48, 3)
    refused(bad, ops.linear_bwd, dy, x, w, act="silu")                     # no z
    refused(ops.MOE_ERR_WORKSPACE, ops.linear_bwd, dy, x, w, z=dy, act="silu",
            ws=torch.empty((64,), dtype=torch.uint8, device="cuda"))
    refused(bad, ops.linear_bwd, dy[:15], x, w)
    refused(bad, ops.linear_bwd, dy, x, w, want_dx=False, want_dw=False)
    refused(bad, ops.gated_ffn_fwd, x, mat(64, 47, 2))
    refused(ops.MOE_ERR_UNSUPPORTED, ops.gated_ffn_fwd, x, mat(64, 40, 2), h=mat(16, 20, 2))
    refused(bad, ops.gated_ffn_bwd, mat(16, 24, 3), mat(16, 40, 3), x, w)
