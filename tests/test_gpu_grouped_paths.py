"""The backward passes' launches at the sizes that choose between them: both
gradients in two launches (training shapes), in one, the weight gradient alone in
both output types and every tile width, and offsets that are wrong with both
gradients asked for.  Tolerances and helpers of test_gpu_grouped.py."""
import pytest
import torch

from helpers import gpu_ops
from test_gpu_grouped import BF, F, Groups, ffn_bwd_check, mat, product, up8, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def each(gr, dx, dw, x, w, dy):
    for g, a, b in gr.spans:
        if dx is not None:
            product(dx[a:b], dy[a:b], w[g].T, f"dx {g}")
        if dw is not None and b > a:
            product(dw[g], x[a:b].T, dy[a:b], f"dw {g}")
        elif dw is not None:
            assert float(dw[g].abs().max()) == 0


# 2 M K N above 1,000 steps of 256 x 256 x 64 for each of 76 CTA pairs: two launches
@pytest.mark.parametrize("dwt", [BF, F])
def test_both_gradients_in_two_launches(ops, dwt):
    gr = Groups([5000, 0, 3001, 197])
    k, n = 4096, 7168
    assert 2 * gr.M * k * n / (256 * 256 * 64) > 1.2 * 76000
    x, w, dy = mat(gr.M, k, 1), weights(gr.G, k, n, 2), mat(gr.M, n, 3, 0.3)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dw = ops.grouped_linear_bwd(dy, x, w, gr.offsets, dw_dtype=dwt, err=err)
    assert int(err) == 0
    each(gr, dx, dw, x, w, dy)
    dx1, _ = ops.grouped_linear_bwd(dy, x, w, gr.offsets, want_dw=False)
    _, dw1 = ops.grouped_linear_bwd(dy, x, w, gr.offsets, want_dx=False, dw_dtype=dwt)
    assert torch.equal(dx, dx1) and torch.equal(dw, dw1)


@pytest.mark.parametrize("dwt", [BF, F])
def test_gated_backward_in_two_launches(ops, dwt):
    gr = Groups([5000, 0, 3001, 197], 128)
    d, f = 4096, 3584
    x, w1, dh, a = mat(gr.M, d, 4), weights(gr.G, d, 2 * f, 5), mat(gr.M, f, 6, 0.3), mat(gr.M, 2 * f, 7)
    ffn_bwd_check(ops, gr, dh, a, x, w1, "silu", dw_dtype=dwt)


# K, N and rows that take tiles of 128, 192, 224 and 256 columns; widths that end inside 8, 16, 32 and 64 columns
WIDTHS = [(1000, 441, 2900, 3), (515, 700, 3000, 5), (515, 696, 3000, 5), (1030, 447, 4000, 6), (1030, 440, 4000, 6),
          (4096, 900, 5000, 3), (4096, 912, 5000, 3)]


@pytest.mark.parametrize("k,n,m,G", WIDTHS)
@pytest.mark.parametrize("dwt", [BF, F])
def test_weight_gradient_alone(ops, k, n, m, G, dwt):
    counts = [m // G + 7 * i for i in range(G - 2)] + [0]
    gr = Groups(counts + [m - sum(counts)])
    x, w, dy = mat(gr.M, k, 8), weights(G, k, n, 9), mat(gr.M, n, 10)
    buf = torch.full((G, k + 3, up8(n) + 16), 7.0, dtype=dwt, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    none, dw = ops.grouped_linear_bwd(dy, x, w, gr.offsets, want_dx=False, dw=buf[:, :k, :n], err=err)
    assert none is None and int(err) == 0
    assert bool((buf[:, :, n:] == 7.0).all()) and bool((buf[:, k:] == 7.0).all())
    each(gr, None, dw, x, w, dy)
    dx, both = ops.grouped_linear_bwd(dy, x, w, gr.offsets, dw_dtype=dwt)
    assert torch.equal(both, dw)
    each(gr, dx, None, x, w, dy)


@pytest.mark.parametrize("m", [100, 4000])
@pytest.mark.parametrize("bad", [[0, 0.5, 0.4, 1], [-1, 0.2, 0.4, 0.6], [0, 0.2, 0.4, 2], [0, 1, 0, 1], [0, 1, 0, 1, 0, 1, 0, 1],
                                 [0.05, 0.04, 0.03, 0.02]])
@pytest.mark.parametrize("dwt", [BF, F])
def test_bad_offsets(ops, m, bad, dwt):
    """groups that overlap or run out of the rows: an error word, and nothing outside the outputs"""
    k, n, G = 72, 144, len(bad) - 1
    offsets = torch.tensor([int(b * m) if b not in (-1, 2) else (-1 if b < 0 else m + 1) for b in bad], dtype=torch.int32, device="cuda")
    x, w, dy, a = mat(m, k, 11), weights(G, k, n, 12), mat(m, n, 13), mat(m, n, 14)
    xbuf = torch.full((m + 600, k), 7.0, dtype=BF, device="cuda")
    abuf = torch.full((m + 600, n), 7.0, dtype=BF, device="cuda")
    wbuf = torch.full((G + 2, k, n), 7.0, dtype=dwt, device="cuda")
    for call in (lambda e: ops.grouped_linear_bwd(dy, x, w, offsets, dx=xbuf[300:300 + m], dw=wbuf[1:1 + G], err=e),
                 lambda e: ops.grouped_linear_bwd(dy, x, w, offsets, want_dx=False, dw=wbuf[1:1 + G], err=e),
                 lambda e: ops.grouped_ffn_bwd(dy[:, :n // 2], a, x, w, offsets, dx=xbuf[300:300 + m], dw1=wbuf[1:1 + G],
                                               da=abuf[300:300 + m], err=e)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(err)
        assert int(err) == ops.MOE_ERR_BAD_OFFSETS
        for buf, lo, hi in ((xbuf, 300, 300 + m), (abuf, 300, 300 + m), (wbuf, 1, 1 + G)):
            assert bool((buf[:lo] == 7.0).all()) and bool((buf[hi:] == 7.0).all())
    # the groups that are right are not touched by the others' offsets
    good = torch.tensor([0, m // 2, m // 2, m] + [m] * (G - 3), dtype=torch.int32, device="cuda")
    dx, dw = ops.grouped_linear_bwd(dy, x, w, good, dw_dtype=dwt)
    product(dx[:m // 2], dy[:m // 2], w[0].T, "dx")
    product(dw[2], x[m // 2:].T, dy[m // 2:], "dw")
