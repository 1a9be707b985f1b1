"""bf16 products grouped by expert against their definitions in 64 bits.

Tolerances as for the dense layers, from the roundings alone: the tensor core
adds 16 products at a time to an fp32 accumulator, so a product over K is off by
at most (K / 16 + 8) 2^-23 of the sum of its terms' magnitudes; the activations'
fp32 work by 2^-18 of the magnitudes it handles, slopes below 1.2; each bf16
store by half a step, 2^-8 of the value, and a rounded operand (da) passes its
half step on through the sum of the magnitudes."""
import math

import pytest
import torch

from helpers import gpu_ops

pytestmark = pytest.mark.gpu

BF, F, D = torch.bfloat16, torch.float32, torch.float64
HALF, WORK = 2.0 ** -8, 2.0 ** -18
NAN = float("nan")


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def up8(n):
    return (n + 7) // 8 * 8


def mat(m, n, seed, std=1.0, pad=0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn((m, up8(n) + pad), generator=g, device="cuda").mul_(std).to(dtype)
    buf[:, n:] = NAN                      # nothing between the rows is used
    return buf[:, :n]


def weights(G, k, n, seed, pad=0, gap=0, std=0.05):
    """[G, k, n], rows padded, matrices `gap` rows apart, NaN in between"""
    t = mat(G * (k + gap), n, seed, std, pad)
    w = t.as_strided((G, k, n), ((k + gap) * t.stride(0), t.stride(0), 1))
    if gap:
        t.as_strided((G, gap, n), ((k + gap) * t.stride(0), t.stride(0), 1), k * t.stride(0)).fill_(NAN)
    return w


class Groups:
    """offsets, rows (or None) and spans of groups of `counts` rows, each `pad`-aligned, after `before` rows"""

    def __init__(self, counts, pad=1, before=0, after=0):
        at, starts = before, []
        for c in counts:
            starts.append(at)
            at += -(-c // pad) * pad
        self.counts, self.M, self.G = counts, at + after, len(counts)
        self.spans = [(g, a, a + c) for g, (a, c) in enumerate(zip(starts, counts))]
        self.offsets = torch.tensor(starts + [at], dtype=torch.int32, device="cuda")
        self.rows = torch.tensor(counts, dtype=torch.int32, device="cuda") if pad > 1 else None
        self.inside = torch.zeros((self.M,), dtype=torch.bool, device="cuda")
        for _, a, b in self.spans:
            self.inside[a:b] = True


def acc(k):
    return (k / 16 + 8) * 2.0 ** -23


def act(z, kind):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: z * torch.special.ndtr(z)}[kind]()


def close(got, want, tol, what):
    g = got.double()
    assert bool(torch.isfinite(g).all()), what
    off = (g - want).abs() - tol
    assert bool((off <= 1e-30).all()), (what, float(off.max()), torch.nonzero(off > 0)[:3].tolist())


def product(got, x, w, what, extra=0.0):
    """got = x w of one group, rounded once"""
    x, w = x.double(), w.double()
    want, size = x @ w, x.abs() @ w.abs()
    half = 2.0 ** -24 if got.dtype == F else HALF
    close(got, want, want.abs() * half + size * (acc(x.shape[1]) + extra), what)


COUNTS = {
    "one": [1],
    "one_tile": [256],
    "edges": [257, 255, 1, 31, 33, 0, 0, 700, 16, 15, 17],
    "tiny": [1, 0, 2, 0, 0, 1, 3, 1] * 5,
    "empty_ends": [0, 0, 64, 65, 0],
    "long": [3, 2500, 0, 40],
    "many": [(7 * i) % 11 for i in range(300)],
}
# (K, N): a step and a tile, ragged everywhere, one, wide, deep
SHAPES = [(64, 256), (65, 257), (1, 1), (515, 259), (130, 1030), (1000, 40), (72, 12)]
CASES = [(c, s) for c in COUNTS for s in SHAPES[:2]] + [("edges", s) for s in SHAPES[2:]] + [("tiny", s) for s in SHAPES[2:]]


@pytest.mark.parametrize("counts,shape", CASES)
def test_linear_forward(ops, counts, shape):
    (k, n), gr = shape, Groups(COUNTS[counts])
    x, w = mat(gr.M, k, 1), weights(gr.G, k, n, 2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ops.grouped_linear_fwd(x, w, gr.offsets, err=err)
    assert int(err) == 0 and y.shape == (gr.M, n)
    for g, a, b in gr.spans:
        product(y[a:b], x[a:b], w[g], f"group {g}")


@pytest.mark.parametrize("counts,shape", CASES)
@pytest.mark.parametrize("dwt", [BF, F])
def test_linear_backward(ops, counts, shape, dwt):
    (k, n), gr = shape, Groups(COUNTS[counts])
    x, w, dy = mat(gr.M, k, 3), weights(gr.G, k, n, 4), mat(gr.M, n, 5, 0.3)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dw = ops.grouped_linear_bwd(dy, x, w, gr.offsets, dw_dtype=dwt, err=err)
    assert int(err) == 0
    for g, a, b in gr.spans:
        product(dx[a:b], dy[a:b], w[g].T, f"dx {g}")
        if a == b:
            assert float(dw[g].abs().max()) == 0
        else:
            product(dw[g], x[a:b].T, dy[a:b], f"dw {g}")


def ffn_check(h, a, x, w1, kind, what):
    f = w1.shape[1] // 2
    z, size = x.double() @ w1.double(), x.double().abs() @ w1.double().abs()
    off = size * acc(x.shape[1])
    if a is not None:
        close(a, z, z.abs() * HALF + off, what + " a")
    gate, up = z[:, :f], z[:, f:]
    want = act(gate, kind) * up
    tol = 1.2 * off[:, :f] * up.abs() + off[:, f:] * gate.abs() + 1.2 * off[:, :f] * off[:, f:]
    close(h, want, want.abs() * (HALF + 2.0 ** -22) + tol + (gate * up).abs() * WORK, what + " h")


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("d,f", [(64, 128), (130, 72), (515, 328)])
@pytest.mark.parametrize("want_a", [False, True])
def test_gated_forward(ops, counts, d, f, want_a):
    gr = Groups(COUNTS[counts])
    x, w1 = mat(gr.M, d, 6), weights(gr.G, d, 2 * f, 7, std=2.0 / math.sqrt(d))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ops.grouped_ffn_fwd(x, w1, gr.offsets, want_a=want_a, err=err)
    h, a = out if want_a else (out, None)
    assert int(err) == 0
    for g, lo, hi in gr.spans:
        ffn_check(h[lo:hi], None if a is None else a[lo:hi], x[lo:hi], w1[g], "silu", f"group {g}")


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
def test_activations(ops, kind):
    gr = Groups(COUNTS["edges"])
    d, f = 200, 136
    x, w1 = mat(gr.M, d, 8), weights(gr.G, d, 2 * f, 9, std=2.0 / math.sqrt(d))
    h, a = ops.grouped_ffn_fwd(x, w1, gr.offsets, act=kind, want_a=True)
    for g, lo, hi in gr.spans:
        ffn_check(h[lo:hi], a[lo:hi], x[lo:hi], w1[g], kind, f"group {g}")
    dh = mat(gr.M, f, 10, 0.3)
    ffn_bwd_check(ops, gr, dh, a, x, w1, kind)


def ffn_bwd_check(ops, gr, dh, a, x, w1, kind, **kw):
    f = w1.shape[2] // 2
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a0 = a.clone()
    dx, dw = ops.grouped_ffn_bwd(dh, a, x, w1, gr.offsets, gr.rows, act=kind, err=err, **kw)
    assert int(err) == 0
    for g, lo, hi in gr.spans:
        z = a0[lo:hi].double().requires_grad_()
        want_h = act(z[:, :f], kind) * z[:, f:]
        da, = torch.autograd.grad(want_h, z, dh[lo:hi].double()) if hi > lo else (torch.zeros_like(z),)
        # da is off by its own rounding, and by the fp32 work on the magnitudes that
        # its halves handle: up (slope) and gate (activation)
        X, W1, G_, U = x[lo:hi].double(), w1[g].double(), z.detach()[:, :f].abs(), z.detach()[:, f:].abs()
        mag, DH = da.abs(), dh[lo:hi].double().abs()
        off = mag * HALF + WORK * torch.cat((DH * U * (1 + G_), DH * G_), 1)
        want = da @ W1.T
        close(dx[lo:hi], want, want.abs() * HALF + (off + acc(2 * f) * (mag + off)) @ W1.abs().T, f"dx {g}")
        if hi > lo:
            want = X.T @ da
            half = 2.0 ** -24 if dw.dtype == F else HALF
            close(dw[g], want, want.abs() * half + X.abs().T @ (off + acc(hi - lo) * (mag + off)), f"dw {g}")
        else:
            assert float(dw[g].abs().max()) == 0
    return dx, dw


@pytest.mark.parametrize("counts", ["edges", "tiny", "long"])
@pytest.mark.parametrize("d,f", [(64, 128), (515, 72)])
@pytest.mark.parametrize("in_place", [False, True])
def test_gated_backward(ops, counts, d, f, in_place):
    gr = Groups(COUNTS[counts])
    x, w1, dh = mat(gr.M, d, 11), weights(gr.G, d, 2 * f, 12), mat(gr.M, f, 13, 0.3)
    a = mat(gr.M, 2 * f, 14)
    ffn_bwd_check(ops, gr, dh, a, x, w1, "silu", dw_dtype=F if in_place else BF, **(dict(da=a) if in_place else {}))


@pytest.mark.parametrize("pad,before,after", [(1, 5, 9), (128, 0, 0), (16, 3, 40), (3, 0, 1)])
def test_rows_of_no_group(ops, pad, before, after):
    """padding between the groups, rows before the first and behind the last: NaN in
    them enters nothing, and what the outputs held there stays"""
    gr = Groups([40, 0, 129, 3, 256, 0, 77], pad, before, after)
    d, f = 200, 72
    x, w1 = mat(gr.M, d, 15), weights(gr.G, d, 2 * f, 16)
    dh, dy, w2 = mat(gr.M, f, 17), mat(gr.M, d, 18), weights(gr.G, f, d, 19)
    out = ~gr.inside
    for t in (x, dh, dy):
        t[out] = NAN

    def room(n):
        return torch.full((gr.M, n), 7.0, dtype=BF, device="cuda")

    h, a, y = room(f), room(2 * f), room(d)
    ops.grouped_ffn_fwd(x, w1, gr.offsets, gr.rows, h=h, a=a)
    a_kept = a.clone()
    ops.grouped_linear_fwd(h, w2, gr.offsets, gr.rows, y=y)
    dx, da = room(d), room(2 * f)
    _, dw1 = ops.grouped_ffn_bwd(dh, a, x, w1, gr.offsets, gr.rows, dx=dx, da=da)
    h2 = h.clone()
    h2[out] = NAN
    dh2 = room(f)
    _, dw2 = ops.grouped_linear_bwd(dy, h2, w2, gr.offsets, gr.rows, dx=dh2)
    for t in (h, a, y, dx, da, dh2):
        assert bool((t[out] == 7.0).all())
    for g, lo, hi in gr.spans:
        ffn_check(h[lo:hi], a[lo:hi], x[lo:hi], w1[g], "silu", f"group {g}")
        product(y[lo:hi], h[lo:hi], w2[g], f"y {g}")
        product(dh2[lo:hi], dy[lo:hi], w2[g].T, f"dh {g}")
        if hi > lo:
            product(dw2[g], h[lo:hi].T, dy[lo:hi], f"dw2 {g}")
    ffn_bwd_check(ops, gr, dh, a_kept, x, w1, "silu")
    assert bool(torch.isfinite(dw1).all())


def test_groups_do_not_mix(ops):
    """NaN and infinities of one group's rows and weights stay in its results"""
    gr = Groups([37, 50, 21, 64, 1])
    k, n = 100, 90
    x, w, dy = mat(gr.M, k, 20), weights(gr.G, k, n, 21), mat(gr.M, n, 22)
    clean = ops.grouped_linear_fwd(x, w, gr.offsets), *ops.grouped_linear_bwd(dy, x, w, gr.offsets)
    x[37:87] = NAN
    dy[37:87] = torch.inf
    w[3] = NAN
    y, (dx, dw) = ops.grouped_linear_fwd(x, w, gr.offsets), ops.grouped_linear_bwd(dy, x, w, gr.offsets)
    for g, a, b in gr.spans:
        if g != 1:
            assert torch.equal(dw[g], clean[2][g])
        if g not in (1, 3):
            assert torch.equal(y[a:b], clean[0][a:b]) and torch.equal(dx[a:b], clean[1][a:b])


@pytest.mark.parametrize("pad,gap", [(0, 0), (8, 0), (40, 3), (0, 5)])
def test_strides(ops, pad, gap):
    """padded rows of every matrix, weights apart, odd widths: nothing between is used or written"""
    gr = Groups([130, 5, 0, 300])
    k, n = 150, 187
    x, w, dy = mat(gr.M, k, 23, pad=pad), weights(gr.G, k, n, 24, pad, gap), mat(gr.M, n, 25, pad=pad)
    ybuf = torch.full((gr.M, up8(n) + pad), 7.0, dtype=BF, device="cuda")
    xbuf = torch.full((gr.M, up8(k) + pad), 7.0, dtype=BF, device="cuda")
    for dwt in (BF, F):
        wbuf = torch.full((gr.G, k + gap, up8(n) + pad), 7.0, dtype=dwt, device="cuda")
        y = ops.grouped_linear_fwd(x, w, gr.offsets, y=ybuf[:, :n])
        dx, dw = ops.grouped_linear_bwd(dy, x, w, gr.offsets, dx=xbuf[:, :k], dw=wbuf[:, :k, :n])
        for buf, n0 in ((ybuf, n), (xbuf, k), (wbuf[:, :k], n)):
            assert bool((buf[..., n0:] == 7.0).all())
        assert bool((wbuf[:, k:] == 7.0).all())
        for g, a, b in gr.spans:
            product(y[a:b], x[a:b], w[g], "y")
            product(dx[a:b], dy[a:b], w[g].T, "dx")
            if b > a:
                product(dw[g], x[a:b].T, dy[a:b], "dw")


@pytest.mark.parametrize("counts,k,n", [([30, 0, 200, 70], 300, 264), ([1500, 3, 0, 497], 4096, 5120)])
def test_gradients_alone_and_together(ops, counts, k, n):
    """in one launch (few steps), in two (many), or one of them: the same bits"""
    gr = Groups(counts)
    x, w, dy = mat(gr.M, k, 50), weights(gr.G, k, n, 51), mat(gr.M, n, 52)
    dx, dw = ops.grouped_linear_bwd(dy, x, w, gr.offsets)
    dx1, none = ops.grouped_linear_bwd(dy, x, w, gr.offsets, want_dw=False)
    none1, dw1 = ops.grouped_linear_bwd(dy, x, w, gr.offsets, want_dx=False)
    assert none is None and none1 is None and torch.equal(dx, dx1) and torch.equal(dw, dw1)
    for g, a, b in gr.spans:
        if b > a:
            product(dx[a:b], dy[a:b], w[g].T, "dx")
            product(dw[g], x[a:b].T, dy[a:b], "dw")
        else:
            assert float(dw[g].abs().max()) == 0


@pytest.mark.parametrize("m,k,n", [(411, 700, 72), (428, 333, 432), (64, 2000, 512), (100, 100, 3000), (129, 64, 64)])
def test_few_tiles(ops, m, k, n):
    """one group with fewer tiles than SMs: narrower ones"""
    gr = Groups([m])
    x, w = mat(m, k, 53), weights(1, k, n, 54)
    product(ops.grouped_linear_fwd(x, w, gr.offsets), x, w[0], "y")
    w1 = weights(1, k, 2 * n, 55, std=2.0 / math.sqrt(k))
    h, a = ops.grouped_ffn_fwd(x, w1, gr.offsets, want_a=True)
    ffn_check(h, a, x, w1[0], "silu", "gated")


def test_more_groups_than_rows(ops):
    G, k, n = 5000, 40, 24
    counts = [0] * G
    for i, g in enumerate((0, 31, 32, 1000, 1001, 4095, 4096, 4999)):
        counts[g] = 1 + 20 * i
    gr = Groups(counts)
    x, w, dy = mat(gr.M, k, 26), weights(G, k, n, 27), mat(gr.M, n, 28)
    y, (dx, dw) = ops.grouped_linear_fwd(x, w, gr.offsets), ops.grouped_linear_bwd(dy, x, w, gr.offsets)
    for g, a, b in gr.spans:
        if b > a:
            product(y[a:b], x[a:b], w[g], "y")
            product(dx[a:b], dy[a:b], w[g].T, "dx")
            product(dw[g], x[a:b].T, dy[a:b], "dw")
    empty = torch.tensor([c == 0 for c in counts], device="cuda")
    assert float(dw[empty].abs().max()) == 0


def test_no_rows_at_all(ops):
    k, n = 48, 40
    w = weights(3, k, n, 29)
    none = torch.zeros(4, dtype=torch.int32, device="cuda")
    for M in (0, 20):
        x, dy = mat(M, k, 30), mat(M, n, 31)
        y = torch.full((M, n), 7.0, dtype=BF, device="cuda")
        assert bool((ops.grouped_linear_fwd(x, w, none, y=y) == 7.0).all())
        dw = torch.full((3, k, n), 7.0, dtype=F, device="cuda")
        ops.grouped_linear_bwd(dy, x, w, none, dw=dw)
        assert float(dw.abs().max()) == 0


@pytest.mark.parametrize("bad", [[0, 50, 40, 100], [-1, 20, 40, 60], [0, 20, 40, 101], [0, 100, 0, 100], [5, 4, 3, 2]])
def test_bad_offsets(ops, bad):
    """an error word, and nothing outside the outputs"""
    k, n, M = 64, 64, 100
    x, w, dy = mat(M, k, 32), weights(3, k, n, 33), mat(M, n, 34)
    ybuf = torch.full((M + 600, n), 7.0, dtype=BF, device="cuda")
    offsets = torch.tensor(bad, dtype=torch.int32, device="cuda")
    for call in (lambda e: ops.grouped_linear_fwd(x, w, offsets, y=ybuf[300:400], err=e),
                 lambda e: ops.grouped_linear_bwd(dy, x, w, offsets, want_dx=False, err=e),
                 lambda e: ops.grouped_ffn_fwd(x, w, offsets, h=torch.empty((M, 32), dtype=BF, device="cuda"), err=e)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(err)
        assert int(err) == ops.MOE_ERR_BAD_OFFSETS
    assert bool((ybuf[:300] == 7.0).all()) and bool((ybuf[400:] == 7.0).all())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 20, 40, 100], dtype=torch.int32, device="cuda")
    rows = torch.tensor([20, 21, 60], dtype=torch.int32, device="cuda")      # one too many
    ops.grouped_linear_fwd(x, w, good, rows, err=err)
    assert int(err) == ops.MOE_ERR_BAD_OFFSETS


def test_streams_graphs_and_the_same_bits(ops):
    """two calls at a time; a captured call replayed over other offsets"""
    gr, other = Groups([300, 0, 1, 500, 223]), Groups([1, 1020, 2, 0, 1])
    k, n = 264, 136
    x, w, dy = mat(gr.M, k, 35), weights(5, k, n, 36), mat(gr.M, n, 37)
    want = ops.grouped_linear_fwd(x, w, gr.offsets), *ops.grouped_linear_bwd(dy, x, w, gr.offsets)
    want2 = ops.grouped_linear_fwd(x, w, other.offsets), *ops.grouped_linear_bwd(dy, x, w, other.offsets)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        y = ops.grouped_linear_fwd(x, w, gr.offsets, stream=s1)
        dx, dw = ops.grouped_linear_bwd(dy, x, w, gr.offsets, stream=s2)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, (y, dx, dw)))
    y, dx, dw = (torch.empty_like(t) for t in want)
    offsets = gr.offsets.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.grouped_linear_fwd(x, w, offsets, y=y)
        ops.grouped_linear_bwd(dy, x, w, offsets, dx=dx, dw=dw)
    for o, e in ((gr, want), (other, want2), (gr, want)):
        offsets.copy_(o.offsets)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(e, (y, dx, dw)))


def test_far_rows(ops):
    """offsets beyond 2^31 elements"""
    M, k, n = 310000, 7168, 64
    x = torch.zeros((M, k), dtype=BF, device="cuda")
    x[-200:] = mat(200, k, 38)
    w, dy = weights(2, k, n, 39), torch.zeros((M, n), dtype=BF, device="cuda")
    dy[-200:] = mat(200, n, 40)
    offsets = torch.tensor([M - 200, M - 90, M], dtype=torch.int32, device="cuda")
    y, (dx, dw) = ops.grouped_linear_fwd(x, w, offsets), ops.grouped_linear_bwd(dy, x, w, offsets)
    for g, a, b in ((0, M - 200, M - 90), (1, M - 90, M)):
        product(y[a:b], x[a:b], w[g], "y")
        product(dx[a:b], dy[a:b], w[g].T, "dx")
        product(dw[g], x[a:b].T, dy[a:b], "dw")


def test_gradients_against_differences(ops):
    """of sum(y c) through both products, in 64-bit differences of the definition"""
    gr = Groups([3, 0, 5])
    d, f = 16, 8
    x, w1, w2 = mat(8, d, 41), weights(3, d, 2 * f, 42, std=0.3), weights(3, f, d, 43, std=0.3)
    c = mat(8, d, 44)

    def loss(X, W1):
        total = 0.0
        for g, a, b in gr.spans:
            z = X[a:b] @ W1[g]
            total += float(((act(z[:, :f], "silu") * z[:, f:]) @ w2[g].double() * c[a:b].double()).sum())
        return total

    h, a = ops.grouped_ffn_fwd(x, w1, gr.offsets, want_a=True)
    dh, _ = ops.grouped_linear_bwd(c, h, w2, gr.offsets, want_dw=False)
    dx, dw1 = ops.grouped_ffn_bwd(dh, a, x, w1, gr.offsets, dw_dtype=F)
    X, W1, e = x.double(), w1.double(), 1e-4
    for r, i in ((0, 0), (2, 5), (7, 15)):
        up, down = X.clone(), X.clone()
        up[r, i] += e
        down[r, i] -= e
        assert abs((loss(up, W1) - loss(down, W1)) / (2 * e) - float(dx[r, i])) <= 0.05 * float(dx.abs().max())
    for g, i, j in ((0, 3, 2), (2, 15, 15), (1, 0, 0)):
        up, down = W1.clone(), W1.clone()
        up[g, i, j] += e
        down[g, i, j] -= e
        assert abs((loss(X, up) - loss(X, down)) / (2 * e) - float(dw1[g, i, j])) <= 0.05 * float(dw1.abs().max())


def test_refusals(ops):
    gr = Groups([3, 4])
    x, w, dy = mat(7, 64, 45), weights(2, 64, 48, 46), mat(7, 48, 47)
    o = gr.offsets
    for call in (
        lambda: ops.grouped_linear_fwd(x.float(), w, o),
        lambda: ops.grouped_linear_fwd(x, w.half(), o),
        lambda: ops.grouped_linear_fwd(x, w[0], o),
        lambda: ops.grouped_linear_fwd(x[:, :63], w, o),
        lambda: ops.grouped_linear_fwd(x, w, o.long()),
        lambda: ops.grouped_linear_fwd(x, w, o[:2]),
        lambda: ops.grouped_linear_fwd(x, w, o, o),
        lambda: ops.grouped_linear_fwd(x, w, o.cpu()),
        lambda: ops.grouped_linear_fwd(x, w, None),
        lambda: ops.grouped_linear_fwd(x, w[:1].expand(2, 64, 48), o),
        lambda: ops.grouped_linear_fwd(x, w.transpose(1, 2).contiguous().transpose(1, 2), o),
        lambda: ops.grouped_linear_fwd(x[:, 1:], w[:, 1:], o),
        lambda: ops.grouped_linear_fwd(x, w[:, :, 1:].as_strided((2, 64, 47), (64 * 47, 47, 1)), o),
        lambda: ops.grouped_linear_bwd(dy, x, w, o, want_dx=False, want_dw=False),
        lambda: ops.grouped_linear_bwd(dy, x, w, o, dw=torch.empty((2, 64, 47), dtype=BF, device="cuda")),
        lambda: ops.grouped_linear_bwd(dy[:6], x, w, o),
        lambda: ops.grouped_ffn_fwd(x, w[:, :, :44], o),
        lambda: ops.grouped_ffn_fwd(x, w, o, act="tanh"),
        lambda: ops.grouped_ffn_bwd(dy[:, :24], dy[:, :40], x, w, o),
    ):
        with pytest.raises((ops.MoEError, TypeError)):
            call()
