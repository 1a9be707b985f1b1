"""The distillation loss and its gradient against the fp64 definition.

Tolerances, from the roundings alone.  An exponential of base 2 is off by 2^-22
of its value and by the rounding of its argument: a difference and a product,
each 2^-24 of the argument, 2^-23 |arg| ln 2 of the value.  A sum of positive
terms adds at most 600 of them one after the other in these tests (2^-24 each).
So a probability with an argument of `a` is off by (2 + a + 40) 2^-22 of its
value; loss terms by 2^-21 of the magnitudes that are added (with the
probabilities' own error: 64 x 2^-22 covers arguments up to 20, where terms
below carry no weight).  A bf16 result is off by half a step, 2^-8 of its value,
besides; what is smaller than 2^-120 may become zero."""
import numpy as np
import pytest
import torch

from helpers import gpu_ops
from oracle.distill_oracle import distill

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
WORK = 64 * 2.0 ** -22


@pytest.fixture(scope="module")
def ops():
    return gpu_ops()


def example(M, V, k, seed, xt=BF, tt=F, tail=False, tau=1.0, pad=0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = V + pad
    buf = torch.full((M * ld + offset + 8,), float("nan"), dtype=xt, device="cuda")
    x = buf[offset:offset + M * ld].view(M, ld)[:, :V]
    x.copy_(torch.randn((M, V), generator=g, device="cuda") * 2)
    idx = torch.stack([torch.randperm(V, generator=g, device="cuda")[:k] for _ in range(M)])
    if k > V:
        idx = torch.cat((idx, torch.full((M, k - V), -1, device="cuda")), 1)
    t = (torch.randn((M, k), generator=g, device="cuda") * 2).to(tt)
    if M > 2 and k > 1:
        idx[1, k // 2:] = -1
        idx[2] = -1
    lse = None
    if tail:
        z = torch.where(idx >= 0, t.float() / tau, -torch.inf)
        lse = torch.logsumexp(z, 1) + 0.3 * torch.rand((M,), generator=g, device="cuda") + 0.001
        lse = torch.where((idx >= 0).any(1), lse, 0.5)
    dloss = torch.randn((M,), generator=g, device="cuda")
    return x, idx.to(torch.int32), t, lse, dloss


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def want(x, idx, t, lse, tau, dloss):
    """loss, gradient, and the magnitudes that their roundings are relative to"""
    X, I, T, L, D = np64(x), idx.cpu().numpy(), np64(t), np64(lse), np64(dloss)
    loss, dx = distill(X, I, T, L, tau, D)
    z = X / tau
    top = z.max(1, keepdims=True)
    logq = z - (top + np.log(np.exp(z - top).sum(1, keepdims=True)))
    size = np.zeros_like(loss)
    pull = np.zeros_like(dx)          # what is added up in the gradient
    for r in range(X.shape[0]):
        kept = np.flatnonzero((I[r] >= 0) & (I[r] < X.shape[1]) & (T[r] > -np.inf))
        if kept.size == 0 and L is None:
            continue
        zt = T[r, kept] / tau
        p = np.exp(zt - (np.logaddexp.reduce(zt) if L is None else L[r]))
        size[r] = tau * tau * (np.sum(p * (np.minimum(np.abs(zt), 200) + np.abs(z[r, I[r, kept]]) + np.abs(logq[r]).min() + 8)) + 8)
        q = np.exp(logq[r])
        pull[r] = q * (2 if L is None else 2 + 1 / max(1e-30, q.sum() - q[np.unique(I[r, I[r] >= 0])].sum()))
        np.add.at(pull[r], I[r, kept], p)
        pull[r] *= tau * abs(D[r]) * (1 + np.minimum(np.abs(z[r] - top[r]), 200) / 16)
    return loss, dx, size, pull


def close(got, ref, tol, what):
    g = np64(got)
    assert np.all(np.isfinite(g)), what
    off = np.abs(g - ref) - tol - 2.0 ** -120
    assert np.all(off <= 0), (what, float(off.max()), np.argwhere(off > 0)[:3].tolist())


def check(ops, x, idx, t, lse, dloss, tau, dx=None):
    """forward, backward and both in one; the last two agree with the definition"""
    loss_w, dx_w, size, pull = want(x, idx, t, lse, tau, dloss)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, stats = ops.distill_loss_fwd(x, idx, t, lse, tau, err=err)
    close(loss, loss_w, WORK * size, "loss")
    half = 2.0 ** -8 if x.dtype == BF else 2.0 ** -24
    tol = np.abs(dx_w) * half + WORK * pull
    d = ops.distill_loss_bwd(dloss, x, idx, t, stats, lse, tau, dlogits=dx, err=err)
    close(d, dx_w, tol, "dlogits")
    loss2, d2 = ops.distill_loss(dloss, x, idx, t, lse, tau, err=err)
    close(loss2, loss_w, WORK * size, "loss with gradient")
    close(d2, dx_w, tol, "dlogits with loss")
    assert int(err) == 0
    return loss2, d2


# (M, V, k): one element, one token kept, every token kept, one 16-byte unit and its neighbours, parts of a cluster,
# odd rows, more rows than CTAs, wide
# the last ones: a warp to a row, its longest rows, many tokens
SIZES = [(1, 1, 1), (3, 8, 1), (5, 7, 7), (4, 9, 4), (2, 17, 20), (7, 256, 32), (300, 1000, 5), (1300, 130, 3), (5, 2047, 100),
         (33, 4099, 17), (2, 32000, 64), (9, 50257, 20), (40, 36865, 33), (3, 129280, 128), (1, 262147, 1000), (1500, 1, 1),
         (700, 33, 40), (650, 1271, 129), (620, 2551, 16), (5000, 300, 7)]


@pytest.mark.parametrize("m,v,k", SIZES)
@pytest.mark.parametrize("xt", [BF, F])
@pytest.mark.parametrize("tail", [False, True])
def test_sizes(ops, m, v, k, xt, tail):
    tau = 1.0 if m % 2 else 2.0
    check(ops, *example(m, v, k, 1, xt, F, tail, tau), tau)


@pytest.mark.parametrize("tau", [0.25, 0.7, 5.0])
@pytest.mark.parametrize("tt", [BF, F])
def test_temperatures(ops, tau, tt):
    for tail in (False, True):
        check(ops, *example(6, 3001, 40, 2, BF, tt, tail, tau), tau)


@pytest.mark.parametrize("xt", [BF, F])
@pytest.mark.parametrize("pad,offset,dpad", [(0, 1, 0), (3, 3, 3), (8, 0, 3), (5, 2, 0), (1, 7, 16)])
def test_strides_and_addresses(ops, xt, pad, offset, dpad):
    """rows at any element, the gradient's at others; nothing between the rows is written"""
    M, V = 5, 2053
    x, idx, t, lse, dloss = example(M, V, 30, 3, xt, F, True, 1.0, pad, offset)
    buf = torch.full((M, V + dpad), 7.0, dtype=xt, device="cuda")
    idx_s = torch.full((M, 37), 5, dtype=torch.int32, device="cuda")[:, 2:32]
    idx_s.copy_(idx)
    t_s = torch.full((M, 33), float("nan"), device="cuda")[:, 1:31]
    t_s.copy_(t)
    check(ops, x, idx_s, t_s, lse, dloss, 1.0, dx=buf[:, :V])
    assert bool((buf[:, V:] == 7.0).all())


@pytest.mark.parametrize("xt", [BF, F])
@pytest.mark.parametrize("m,v", [(4, 40001), (200, 777), (2000, 777), (2000, 1000)])
def test_in_place(ops, xt, m, v):
    x, idx, t, lse, dloss = example(m, v, 24, 4, xt, F, True)
    loss, d = ops.distill_loss(dloss, x, idx, t, lse)
    _, stats = ops.distill_loss_fwd(x, idx, t, lse)
    for both in (True, False):
        y = x.clone()
        if both:
            loss2, _ = ops.distill_loss(dloss, y, idx, t, lse, dlogits=y)
            assert torch.equal(loss, loss2)
        else:
            d = ops.distill_loss_bwd(dloss, x, idx, t, stats, lse)
            ops.distill_loss_bwd(dloss, y, idx, t, stats, lse, dlogits=y)
        assert torch.equal(y, d)


@pytest.mark.parametrize("tail", [False, True])
def test_the_same_token_several_times(ops, tail):
    x, idx, t, lse, dloss = example(6, 5000, 64, 5, F, F, tail)
    idx[0, 1::2] = idx[0, 0]
    idx[3] = 17
    idx[4, 60:] = idx[4, :4]
    if tail:
        lse = torch.where((idx >= 0).any(1), torch.logsumexp(torch.where(idx >= 0, t, -torch.inf), 1) + 0.2, 0.0)
    a = check(ops, x, idx, t, lse, dloss, 1.0)
    b = check(ops, x, idx, t, lse, dloss, 1.0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_index_beyond_the_vocabulary(ops):
    x, idx, t, lse, dloss = example(3, 100, 8, 6)
    bad = idx.clone()
    bad[0, 2], bad[1, 0] = 100, 2 ** 31 - 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, d = ops.distill_loss(dloss, x, bad, t, err=err)
    assert int(err) == ops.MOE_ERR_BAD_INDEX
    idx[0, 2], idx[1, 0] = -1, -1
    check(ops, x, idx, t, None, dloss, 1.0)
    loss2, d2 = ops.distill_loss(dloss, x, idx, t)
    assert torch.equal(loss, loss2) and torch.equal(d, d2)


@pytest.mark.parametrize("tail", [False, True])
def test_masked_logits(ops, tail):
    """columns of -inf, of the type's lowest value, a row of nothing else"""
    x, idx, t, lse, dloss = example(8, 4000, 16, 7, BF, F, tail)
    for r in range(8):
        cols = torch.arange(r, 4000, 3, device="cuda")
        keep = ~torch.isin(cols, idx[r])
        x[r, cols[keep]] = -torch.inf if r % 2 else torch.finfo(BF).min
    check(ops, x, idx, t, lse, dloss, 1.0)
    low = torch.full_like(x, torch.finfo(BF).min)       # a row with one value throughout is uniform
    same = torch.zeros_like(x)
    for tau in (0.5, 1.0):
        a, b = ops.distill_loss(dloss, low, idx, t, lse, tau), ops.distill_loss(dloss, same, idx, t, lse, tau)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_masked_teachers(ops):
    x, idx, t, lse, dloss = example(6, 3000, 16, 8)
    t[0, 3:] = -torch.inf
    t[3] = -torch.inf                                    # no teacher
    t[4, 1:] = torch.finfo(F).min
    loss, d = check(ops, x, idx, t, None, dloss, 1.0)
    assert float(loss[3]) == 0 and float(d[3].abs().max()) == 0
    assert float(loss[2]) == 0 and float(d[2].abs().max()) == 0
    lse = torch.logsumexp(t, 1).clamp(min=-5) + 0.1      # with the whole vocabulary's sum -inf is a probability of 0
    lse[2] = 0.0
    check(ops, x, idx, t, lse, dloss, 1.0)


def test_rows_without_weight(ops):
    """dloss = 0: zeros whatever the logits are, in both calls"""
    x, idx, t, lse, dloss = example(5, 6000, 16, 9)
    x[3] = float("nan")
    x[4, ::7] = torch.inf
    dloss[3:] = 0
    _, stats = ops.distill_loss_fwd(x, idx, t)
    _, d = ops.distill_loss(dloss, x, idx, t)
    e = ops.distill_loss_bwd(dloss, x, idx, t, stats)
    for g in (d, e):
        assert bool((g[3:] == 0).all()) and bool(torch.isfinite(g).all())


def test_nan_and_infinity_show_in_their_row_alone(ops):
    x, idx, t, lse, dloss = example(6, 6001, 16, 10)
    x[0, 5], x[3, 6] = float("nan"), torch.inf
    t[4, 0] = float("nan")
    loss, d = ops.distill_loss(dloss, x, idx, t)
    bad = torch.isnan(loss)
    assert bad.tolist() == [True, False, False, True, True, False]
    assert bool(torch.isfinite(d[~bad]).all())


def test_student_that_is_sure(ops):
    """s_rest far below what s - sum of the kept tokens would leave"""
    x, idx, t, lse, dloss = example(4, 3000, 8, 11, F, F, True)
    x.sub_(60)
    x.scatter_(1, idx.clamp(min=0).long(), 20.0)
    loss, dx, size, pull = want(x, idx, t, lse, 1.0, dloss)
    got, d = ops.distill_loss(dloss, x, idx, t, lse)
    close(got, loss, WORK * (size + 100), "loss")
    assert np.allclose(np64(d), dx, rtol=2e-5, atol=1e-6)


@pytest.mark.parametrize("v", [600, 5000])
@pytest.mark.parametrize("xt", [BF, F])
@pytest.mark.parametrize("tail", [False, True])
def test_many_rows(ops, v, xt, tail):
    """the forms for more rows than the GPU has SMs: repeated tokens, masked ones, bad ones,
    rows without weight, padded rows at any element"""
    M = 700
    x, idx, t, lse, dloss = example(M, v, 24, 17, xt, F, tail, 1.0, 3, 1)
    idx[0::7, 1::2] = idx[0::7, :1]
    idx[3::7] = -1
    t[4::7, 5:] = -torch.inf
    x[5::7, 11:400:3] = torch.where(torch.isin(torch.arange(11, 400, 3, device="cuda"), idx[5::7]), x[5::7, 11:400:3], -torch.inf)
    if tail:
        lse = torch.logsumexp(torch.where(idx >= 0, t, -torch.inf), 1) + 0.2
        lse = torch.where((idx >= 0).any(1), lse, 0.0)
    buf = torch.full((M, v + 5), 7.0, dtype=xt, device="cuda")
    check(ops, x, idx, t, lse, dloss, 1.0, dx=buf[:, :v])
    assert bool((buf[:, v:] == 7.0).all())
    y = x.contiguous()                                   # (rows that lie otherwise are summed in another order)
    loss, d = ops.distill_loss(dloss, y, idx, t, lse)
    bad, w = idx.clone(), dloss.clone()
    bad[1, 1] = v                                        # taken as not kept
    y[6], w[6] = float("nan"), 0.0
    y[8, 3] = float("nan")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss2, d2 = ops.distill_loss(w, y, bad, t, lse, dlogits=y, err=err)
    assert int(err) == ops.MOE_ERR_BAD_INDEX and float(d2[6].abs().max()) == 0
    assert bool(torch.isnan(loss2[8])) and bool(torch.isnan(d2[8]).any())
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[[1, 6, 8]] = False
    assert torch.equal(loss[rest], loss2[rest]) and torch.equal(d[rest], d2[rest])


def test_nothing_to_do(ops):
    x = torch.empty((0, 100), dtype=BF, device="cuda")
    idx, t = torch.empty((0, 4), dtype=torch.int32, device="cuda"), torch.empty((0, 4), device="cuda")
    loss, d = ops.distill_loss(torch.empty(0, device="cuda"), x, idx, t)
    assert loss.shape == (0,) and d.shape == (0, 100)


def test_loss_alone_is_not_needed(ops):
    x, idx, t, lse, dloss = example(4, 999, 8, 12)
    loss, d = ops.distill_loss(dloss, x, idx, t)
    none, e = ops.distill_loss(dloss, x, idx, t, want_loss=False)
    assert none is None and torch.equal(d, e)


def test_streams_and_graphs(ops):
    """two calls at a time on two streams; a captured call replayed over new logits"""
    a, b = example(500, 20001, 32, 13, BF, F, True), example(700, 3001, 16, 14, F, BF, False, 2.0)
    wa, wb = ops.distill_loss(a[4], *a[:4]), ops.distill_loss(b[4], *b[:4], temperature=2.0)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        ga = ops.distill_loss(a[4], *a[:4], stream=s1)
        gb = ops.distill_loss(b[4], *b[:4], temperature=2.0, stream=s2)
        torch.cuda.synchronize()
        for g, w in ((ga, wa), (gb, wb)):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    x = a[0].clone()
    loss, d = torch.empty_like(wa[0]), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.distill_loss(a[4], x, *a[1:4], loss=loss, dlogits=d)
    for shift in (0.0, 1.0):
        x.copy_(a[0].flip(0) if shift else a[0])
        graph.replay()
        torch.cuda.synchronize()
        w = ops.distill_loss(a[4], x, *a[1:4])
        assert torch.equal(loss, w[0]) and torch.equal(d, w[1])


def test_far_rows(ops):
    """offsets beyond 2^31 elements"""
    M, V = 17000, 129280
    x = torch.zeros((M, V), dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(15)
    x[-3:] = torch.randn((3, V), generator=g, device="cuda").to(BF)
    idx = torch.randint(V, (M, 4), generator=g, device="cuda").to(torch.int32)
    t = torch.randn((M, 4), generator=g, device="cuda")
    dloss = torch.ones((M,), device="cuda")
    loss, d = ops.distill_loss(dloss, x, idx, t)
    lw, dw, size, pull = want(x[-3:], idx[-3:], t[-3:], None, 1.0, dloss[-3:])
    close(loss[-3:], lw, WORK * size, "loss")
    close(d[-3:], dw, np.abs(dw) * 2.0 ** -8 + WORK * pull, "dlogits")


def test_refusals(ops):
    x, idx, t, lse, dloss = example(4, 100, 8, 16)
    E = ops.MoEError
    calls = [
        lambda: ops.distill_loss_fwd(x.half(), idx, t),
        lambda: ops.distill_loss_fwd(x, idx.long(), t),
        lambda: ops.distill_loss_fwd(x, idx[:3], t),
        lambda: ops.distill_loss_fwd(x, idx, t[:, :7]),
        lambda: ops.distill_loss_fwd(x, idx, t, temperature=0.0),
        lambda: ops.distill_loss_fwd(x, idx, t, temperature=float("nan")),
        lambda: ops.distill_loss_fwd(x, idx, t, torch.zeros(3, device="cuda")),
        lambda: ops.distill_loss_fwd(x.cpu(), idx, t),
        lambda: ops.distill_loss_fwd(x.t(), idx, t),
        lambda: ops.distill_loss_fwd(x[0], idx, t),
        lambda: ops.distill_loss(dloss[:3], x, idx, t),
        lambda: ops.distill_loss(dloss.double(), x, idx, t),
        lambda: ops.distill_loss(dloss, x, idx, t, dlogits=torch.empty((4, 100), device="cuda")),
        lambda: ops.distill_loss(dloss, x, idx, t, dlogits=torch.empty((4, 1), dtype=BF, device="cuda").expand(4, 100)),
        lambda: ops.distill_loss_bwd(dloss, x, idx, t, torch.empty((4, 2), device="cuda")),
        lambda: ops.distill_loss_fwd(x, idx[:, :0], t[:, :0]),
    ]
    for call in calls:
        with pytest.raises(E):
            call()
