"""RMS norm with the residual's addition, its MXFP8 output and its backward
pass against the fp64 definition.

Tolerances, from the roundings alone: fp32 work between load and store leaves
a relative error below 2^-17 (a chain of at most 64 additions and a handful of
products at 2^-24 each); storing adds half a step of the output type (bf16
2^-8, E4M3 2^-4 or half its smallest step 2^-9)."""
import numpy as np
import pytest
import torch

from helpers import atoms_to_rowmajor, gpu_ops
from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -17
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}
EPS = 1e-6


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def mat(m, n, seed, dtype=torch.bfloat16, std=1.0, ld=None, off=0):
    """[m, n] inside a buffer of rows of ld elements, `off` elements in."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = ld or n
    flat = torch.randn((m * ld + off + 8,), generator=g, device="cuda").mul_(std).to(dtype)
    return flat[off:off + m * ld].view(m, ld)[:, :n]


def f64(t):
    return t.double().cpu().numpy()


def check_rows(got, want, dtype, what):
    g = f64(got)
    tol = np.abs(want) * (HALF[dtype] + F32) + 1e-30
    assert np.all(np.abs(g - want) <= tol), (what, np.max(np.abs(g - want) - tol))


def check_mx(ops, codes, scales, y, M, N, layout):
    """Scale bytes by the rule (either side when the block's largest value is
    within 2^-16 of a border) and codes within half a step of y."""
    rows = codes.shape[0]
    sc = scales.cpu().numpy()
    sc = atoms_to_rowmajor(sc, rows, N) if layout == ops.MOE_SF_ATOMS else sc.reshape(rows, N // 32)
    top = np.abs(y).reshape(M, N // 32, 32).max(2)
    lo, hi = D.e8m0_byte(top * (1 - 2 * F32)), D.e8m0_byte(top * (1 + 2 * F32))
    assert np.all((sc[:M] == lo) | (sc[:M] == hi))
    step = np.exp2(sc[:M].astype(np.float64) - 127).repeat(32, axis=1)
    val = f64(codes.view(torch.float8_e4m3fn).float()[:M]) * step
    tol = np.maximum(np.abs(y) * 2.0 ** -4, step * 2.0 ** -10) + np.abs(y) * F32
    assert np.all(np.abs(val - y) <= tol)
    assert not codes[M:].any() and not sc[M:].any()


SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 64), (33, 129), (130, 1000), (7, 1024), (9, 1025), (200, 2048), (17, 4099),
          (4, 7168), (3, 16384), (2, 20001), (2, 32768)]


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("xt,rt", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                   (torch.float32, torch.bfloat16), (torch.float32, torch.float32)])
def test_forward(ops, m, n, xt, rt):
    x, res, w = mat(m, n, 1, xt), mat(m, n, 2, rt, 3.0), mat(1, n, 3, torch.bfloat16)[0]
    y, r, rstd, _, _ = ops.rmsnorm_residual_fwd(x, w, res, EPS, y_dtype=xt)
    wr, wrstd, wy = D.rmsnorm_residual(f64(x), f64(res), f64(w), EPS)
    check_rows(r, wr, rt, "r")
    check_rows(y, wy, xt, "y")
    check_rows(rstd[:, None], wrstd[:, None], torch.float32, "rstd")


@pytest.mark.parametrize("m,n", [(5, 1000), (12, 4096), (3, 4099)])
@pytest.mark.parametrize("pad,off", [(8, 0), (3, 0), (8, 1), (5, 3)])
def test_strides_and_offsets(ops, m, n, pad, off):
    x, res = mat(m, n, 1, ld=n + pad, off=off), mat(m, n, 2, ld=n + pad, off=off)
    w = mat(1, n, 3, torch.float32, off=off)[0]
    y, r = mat(m, n, 4, ld=n + pad, off=off), mat(m, n, 5, ld=n + pad, off=off)
    keep = torch.as_strided(y, (m - 1, pad), (n + pad, 1), y.storage_offset() + n).clone()
    ops.rmsnorm_residual_fwd(x, w, res, EPS, y=y, r=r)
    wr, _, wy = D.rmsnorm_residual(f64(x), f64(res), f64(w), EPS)
    check_rows(r, wr, torch.bfloat16, "r")
    check_rows(y, wy, torch.bfloat16, "y")
    assert torch.equal(keep, torch.as_strided(y, (m - 1, pad), (n + pad, 1), y.storage_offset() + n))


def test_no_residual_and_in_place(ops):
    m, n = 37, 2048
    x, w = mat(m, n, 1), mat(1, n, 3)[0]
    y, r, _, _, _ = ops.rmsnorm_residual_fwd(x, w, None, EPS)
    assert r is None
    check_rows(y, D.rmsnorm_residual(f64(x), None, f64(w), EPS)[2], torch.bfloat16, "y")
    res = mat(m, n, 2, torch.float32)
    wr, _, wy = D.rmsnorm_residual(f64(x), f64(res), f64(w), EPS)
    y, r, _, _, _ = ops.rmsnorm_residual_fwd(x, w, res, EPS, r=res, y=x)
    assert r is res and y is x
    check_rows(res, wr, torch.float32, "r")
    check_rows(x, wy, torch.bfloat16, "y")


@pytest.mark.parametrize("m,n,layout", [(1, 128, "atoms"), (3, 4096, "atoms"), (128, 256, "atoms"), (129, 7168, "atoms"),
                                        (300, 1152, "atoms"), (1, 32, "canonical"), (5, 96, "canonical"),
                                        (131, 2080, "canonical"), (7, 4096, "canonical")])
def test_mxfp8_output(ops, m, n, layout):
    layout = ops.MOE_SF_ATOMS if layout == "atoms" else ops.MOE_SF_CANONICAL
    x, res, w = mat(m, n, 1), mat(m, n, 2), mat(1, n, 3)[0]
    x[0, :32] = 0
    res[0, :32] = 0                               # a block of zeros
    y, r, _, codes, scales = ops.rmsnorm_residual_fwd(x, w, res, EPS, want_codes=True, sf_layout=layout)
    wy = D.rmsnorm_residual(f64(x), f64(res), f64(w), EPS)[2]
    check_rows(y, wy, torch.bfloat16, "y")
    check_mx(ops, codes, scales, wy, m, n, layout)
    only = ops.rmsnorm_residual_fwd(x, w, res, EPS, want_y=False, want_r=False, want_codes=True, sf_layout=layout)
    assert only[0] is None and only[1] is None
    assert torch.equal(only[3], codes) and torch.equal(only[4], scales)


def test_mxfp8_scale_borders(ops):
    """Blocks whose largest value is exactly 1.75 * 2^q take e = q - 8, and
    the next fp32 value above e = q - 7.  (A row of +-1 has rstd = 1 with
    eps = 0, so y is the weight.)"""
    n = 128
    x = torch.ones((1, n), device="cuda")
    w = torch.full((n,), 0.25, device="cuda")
    w[0], w[32], w[64], w[96] = 1.75, 1.7500001192092896, 448.0, 2.0 ** -100
    w[97:] = 0
    _, _, _, _, s = ops.rmsnorm_residual_fwd(x, w, None, 0.0, want_codes=True, sf_layout=ops.MOE_SF_CANONICAL)
    assert s.tolist() == [127 - 8, 127 - 7, 127, 127 - 108]


def test_codes_feed_the_grouped_gemm(ops):
    """The codes and scales are an operand of the grouped GEMM as they are."""
    m, k, n = 200, 512, 256
    x, w = mat(m, k, 1), mat(1, k, 3)[0]
    _, _, _, codes, scales = ops.rmsnorm_residual_fwd(x, w, None, EPS, want_codes=True)
    b = mat(n, k, 4)
    bq, bs = ops.mxfp8_group_quantize(b, ops.MOE_QUANT_ROWWISE)
    gofs = torch.tensor([0, 256], dtype=torch.int32, device="cuda")
    d = ops.grouped_gemm_mxfp8(ops.MOE_GEMM_FWD, codes, scales, bq, bs, ops.MOE_B_GNK, gofs, 1, 256, n, k)
    deq = lambda q, s, rows: (q.view(torch.float8_e4m3fn).float().double().cpu().numpy() *  # noqa: E731
                              np.exp2(atoms_to_rowmajor(s.cpu().numpy(), rows, k).astype(float) - 127).repeat(32, 1))
    want = deq(codes, scales, 256) @ deq(bq, bs, n).T
    scale = np.abs(deq(codes, scales, 256)) @ np.abs(deq(bq, bs, n)).T
    assert np.all(np.abs(f64(d) - want) <= np.abs(want) * 2.0 ** -8 + scale * 2.0 ** -14)


def test_non_finite_rows_stay_in_their_rows(ops):
    m, n = 6, 4096
    x, w = mat(m, n, 1), mat(1, n, 3)[0]
    x[1, 5], x[3, 7], x[4] = float("nan"), float("inf"), 0.0
    y, _, rstd, codes, _ = ops.rmsnorm_residual_fwd(x, w, None, EPS, want_codes=True)
    good = [0, 2, 5]
    check_rows(y[good], D.rmsnorm_residual(f64(x[good]), None, f64(w), EPS)[2], torch.bfloat16, "y")
    assert torch.isnan(y[1]).all() and rstd[3] == 0 and torch.isnan(y[3, 7]) and not y[4].any()
    assert not (codes[4] & 0x7F).any()            # zeros, signs kept


def bwd_tol(dy, r, w, rstd, dres, dtype, want):
    xhat = np.abs(r * rstd[:, None])
    t = np.abs(dy * w)
    size = rstd[:, None] * (t + xhat * np.mean(t * xhat, axis=1, keepdims=True)) + (0 if dres is None else np.abs(dres))
    return np.abs(want) * HALF[dtype] + size * F32


@pytest.mark.parametrize("m,n", SHAPES + [(3000, 64), (1500, 4096)])
@pytest.mark.parametrize("yt,rt,dres", [(torch.bfloat16, torch.bfloat16, True), (torch.bfloat16, torch.float32, True),
                                        (torch.float32, torch.bfloat16, False), (torch.float32, torch.float32, True)])
def test_backward(ops, m, n, yt, rt, dres):
    r, dy, w = mat(m, n, 1, rt, 3.0), mat(m, n, 2, yt), mat(1, n, 3)[0]
    dr = mat(m, n, 4, rt) if dres else None
    rstd = torch.rsqrt(r.double().square().mean(1) + EPS).float()
    dx, dw = ops.rmsnorm_residual_bwd(dy, r, w, rstd, dr)
    drn = f64(dr) if dres else None
    want, wdw = D.rmsnorm_residual_bwd(f64(dy), f64(r), f64(w), f64(rstd), drn)
    assert np.all(np.abs(f64(dx) - want) <= bwd_tol(f64(dy), f64(r), f64(w), f64(rstd), drn, rt, want) + 1e-30)
    size = np.sum(np.abs(f64(dy) * f64(r) * f64(rstd)[:, None]), axis=0)
    # at most m / 608 + 608 / 32 + 16 additions of a column one after the other
    assert np.all(np.abs(f64(dw) - wdw) <= size * (m / 608 + 40) * 2.0 ** -24 + 1e-30)
    again = ops.rmsnorm_residual_bwd(dy, r, w, rstd, dr)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("pad,off", [(8, 0), (3, 0), (5, 3)])
def test_backward_strides(ops, pad, off):
    m, n = 50, 1501
    r, dy, dr = (mat(m, n, s, ld=n + pad, off=off) for s in (1, 2, 3))
    w, rstd = mat(1, n, 4, off=off)[0], torch.rsqrt(r.double().square().mean(1) + EPS).float()
    want, _ = D.rmsnorm_residual_bwd(f64(dy), f64(r), f64(w), f64(rstd), f64(dr))
    tol = bwd_tol(f64(dy), f64(r), f64(w), f64(rstd), f64(dr), torch.bfloat16, want)
    dx, dw = ops.rmsnorm_residual_bwd(dy, r, w, rstd, dr, dx=dr, want_dw=False)      # in place
    assert dx is dr and dw is None
    assert np.all(np.abs(f64(dx) - want) <= tol)


def test_gradients_against_differences(ops):
    """dx and dw against central differences of the fp64 definition."""
    m, n = 3, 40
    x, res, w = mat(m, n, 1, torch.float32), mat(m, n, 2, torch.float32), mat(1, n, 3, torch.float32)[0]
    dy = mat(m, n, 4, torch.float32)
    _, r, rstd, _, _ = ops.rmsnorm_residual_fwd(x, w, res, EPS, y_dtype=torch.float32)
    dx, dw = ops.rmsnorm_residual_bwd(dy, r, w, rstd)
    loss = lambda a, b: float(np.sum(D.rmsnorm_residual(a, f64(res), b, EPS)[2] * f64(dy)))  # noqa: E731
    h = 1e-5
    for i, j in [(0, 0), (1, 17), (2, 39)]:
        e = np.zeros((m, n))
        e[i, j] = h
        assert abs((loss(f64(x) + e, f64(w)) - loss(f64(x) - e, f64(w))) / (2 * h) - float(dx[i, j])) < 1e-4
        assert abs((loss(f64(x), f64(w) + e[i]) - loss(f64(x), f64(w) - e[i])) / (2 * h) - float(dw[j])) < 1e-4


def test_no_rows(ops):
    x, w = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), mat(1, 256, 3)[0]
    y, r, rstd, codes, scales = ops.rmsnorm_residual_fwd(x, w, x, EPS, want_codes=True)
    assert y.shape == (0, 256) and codes.numel() == 0
    dw = torch.ones((256,), device="cuda")
    dx, dw = ops.rmsnorm_residual_bwd(x, x, w, rstd, dw=dw)
    assert dx.shape == (0, 256) and not dw.any()


def test_stream_and_graph(ops):
    """The calls run on the stream they are given and are captured in a graph."""
    m, n = 64, 2048
    x, res, w, dy = mat(m, n, 1), mat(m, n, 2), mat(1, n, 3)[0], mat(m, n, 4)
    y0, r0, rstd0, c0, s0 = ops.rmsnorm_residual_fwd(x, w, res, EPS, want_codes=True)
    dx0, dw0 = ops.rmsnorm_residual_bwd(dy, r0, w, rstd0, res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, r1, rstd1, c1, s1 = ops.rmsnorm_residual_fwd(x, w, res, EPS, want_codes=True, stream=side)
    dx1, dw1 = ops.rmsnorm_residual_bwd(dy, r1, w, rstd1, res, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in ((y0, y1), (r0, r1), (c0, c1), (s0, s1), (dx0, dx1), (dw0, dw1)))
    ws = torch.empty((ops.rmsnorm_bwd_workspace_size(m, n),), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(t) for t in (y0, r0, rstd0, c0, s0, dx0, dw0)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.rmsnorm_residual_fwd(x, w, res, EPS, y=outs[0], r=outs[1], rstd=outs[2], codes=outs[3], scales=outs[4])
        ops.rmsnorm_residual_bwd(dy, outs[1], w, outs[2], res, dx=outs[5], dw=outs[6], ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, (y0, r0, rstd0, c0, s0, dx0, dw0)))


def test_refusals(ops):
    x, w = mat(4, 256, 1), mat(1, 256, 3)[0]

    def refused(status, fn, *a, **k):
        with pytest.raises(ops.MoEError) as e:
            fn(*a, **k)
        assert e.value.status == status

    bad = ops.MOE_ERR_INVALID_ARG
    refused(bad, ops.rmsnorm_residual_fwd, x.cpu(), w)
    refused(bad, ops.rmsnorm_residual_fwd, x.half(), w)
    refused(bad, ops.rmsnorm_residual_fwd, x.t(), w)
    refused(bad, ops.rmsnorm_residual_fwd, x, w[:100])
    refused(bad, ops.rmsnorm_residual_fwd, x, w, x[:3])
    refused(bad, ops.rmsnorm_residual_fwd, x, w, x, r=x.float())
    refused(bad, ops.rmsnorm_residual_fwd, x, w, eps=-1.0)
    refused(bad, ops.rmsnorm_residual_fwd, x[:1].expand(4, 256), w)
    refused(ops.MOE_ERR_UNSUPPORTED, ops.rmsnorm_residual_fwd, mat(2, 160, 1), mat(1, 160, 3)[0], want_codes=True)
    refused(ops.MOE_ERR_UNSUPPORTED, ops.rmsnorm_residual_fwd, mat(1, 32776, 1), mat(1, 32776, 3)[0])
    rstd = torch.ones((4,), device="cuda")
    refused(bad, ops.rmsnorm_residual_bwd, x, x.float(), w, rstd, dx=x)
    refused(bad, ops.rmsnorm_residual_bwd, x, x, w, rstd[:3])
    small = torch.empty((64,), dtype=torch.uint8, device="cuda")
    refused(ops.MOE_ERR_WORKSPACE, ops.rmsnorm_residual_bwd, x, x, w, rstd, ws=small)


@pytest.mark.parametrize("m,n", [(304, 1032), (700, 4096), (931, 7168), (2500, 2000), (305, 8200), (400, 16384)])
@pytest.mark.parametrize("xt,rt,res", [(torch.bfloat16, torch.bfloat16, True), (torch.bfloat16, torch.float32, True),
                                       (torch.float32, torch.bfloat16, True), (torch.float32, torch.float32, False)])
def test_many_rows(ops, m, n, xt, rt, res):
    """Rows that come through the ring of stages, several to a CTA: forward
    (in place too) and backward."""
    x, w, dy = mat(m, n, 1, xt, ld=n + 8), mat(1, n, 3)[0], mat(m, n, 4, xt)
    rs = mat(m, n, 2, rt, 3.0, ld=n + 16) if res else None
    wr, wrstd, wy = D.rmsnorm_residual(f64(x), f64(rs) if res else None, f64(w), EPS)
    y, r, rstd, _, _ = ops.rmsnorm_residual_fwd(x, w, rs, EPS, y_dtype=xt)
    check_rows(y, wy, xt, "y")
    check_rows(rstd[:, None], wrstd[:, None], torch.float32, "rstd")
    if res:
        check_rows(r, wr, rt, "r")
        y2, r2, _, _, _ = ops.rmsnorm_residual_fwd(x, w, rs, EPS, y=x, r=rs)
        assert torch.equal(y2, y) and torch.equal(r2, r)
    else:
        r = x
    dr = mat(m, n, 5, r.dtype) if res else None
    dx, dw = ops.rmsnorm_residual_bwd(dy, r, w, rstd, dr)
    drn = f64(dr) if res else None
    want, wdw = D.rmsnorm_residual_bwd(f64(dy), f64(r), f64(w), f64(rstd), drn)
    assert np.all(np.abs(f64(dx) - want) <= bwd_tol(f64(dy), f64(r), f64(w), f64(rstd), drn, r.dtype, want) + 1e-30)
    size = np.sum(np.abs(f64(dy) * f64(r) * f64(rstd)[:, None]), axis=0)
    # a CTA adds m / 152 rows one after the other at most (one CTA per SM), then up to 608 partial sums
    assert np.all(np.abs(f64(dw) - wdw) <= size * (m / 152 + 40) * 2.0 ** -24 + 1e-30)
    if res:
        assert torch.equal(ops.rmsnorm_residual_bwd(dy, r, w, rstd, dr, dx=dr)[0], dx)


@pytest.mark.parametrize("m,n,layout", [(400, 1152, "atoms"), (1000, 7168, "atoms"), (500, 2080, "canonical")])
def test_mxfp8_output_of_many_rows(ops, m, n, layout):
    layout = ops.MOE_SF_ATOMS if layout == "atoms" else ops.MOE_SF_CANONICAL
    x, res, w = mat(m, n, 1), mat(m, n, 2), mat(1, n, 3)[0]
    y, _, _, codes, scales = ops.rmsnorm_residual_fwd(x, w, res, EPS, want_codes=True, sf_layout=layout)
    wy = D.rmsnorm_residual(f64(x), f64(res), f64(w), EPS)[2]
    check_rows(y, wy, torch.bfloat16, "y")
    check_mx(ops, codes, scales, wy, m, n, layout)
