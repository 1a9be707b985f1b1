"""Cases, plain forms and 64-bit values of the operators that train a 16-bit mixture of experts against a teacher:

  linear   products grouped by expert, y[rows of g] = x[rows of g] W_g, groups of any size, and their backward pass
  ffn      gated projections grouped by expert, h = silu(x Wg) * (x Wu), and their backward pass
  distill  distillation from a teacher's top logits: loss per token, gradient of the logits, both in one pass

`run` computes a case in elementary torch operations in 32 bits, or (own = True) through grouped_gemm_top_gb300.ops.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # experts' up and gate projections of four decoding sequences, top-8 of 256 experts of the DeepSeek-V3-shaped layer: about 30 experts get
        # a row or two, and reading their weights is all there is
        dict(name="ffn_decode", op="ffn", way="fwd", m=32, groups=256, k=7168, n=2048, top=8, skew="even", pad=0, keep=False),
        # the down projection of one decoding sequence
        dict(name="linear_decode", op="linear", way="fwd", m=8, groups=256, k=2048, n=7168, top=8, skew="even", pad=0),
        # prefill of 2,003 tokens through the Mixtral-shaped layer, top-2 of 8
        dict(name="ffn_prefill", op="ffn", way="fwd", m=4006, groups=8, k=4096, n=14336, top=2, skew="even", pad=0, keep=False),
        # the down projection of the DeepSeek-V3-shaped training batch under skewed routing: some experts get thousands of rows, some none
        dict(name="linear_train", op="linear", way="fwd", m=196608, groups=256, k=2048, n=7168, top=8, skew="zipf", pad=0),
        # its backward pass over a quarter of the batch and of the experts
        dict(name="linear_bwd", op="linear", way="bwd", m=49152, groups=64, k=2048, n=7168, top=8, skew="even", pad=0),
        # backward pass of the Mixtral-shaped gated projections, each expert's rows padded to 128 as the layer's permutation lays them out
        dict(name="ffn_bwd", op="ffn", way="bwd", m=8192, groups=8, k=4096, n=14336, top=2, skew="zipf", pad=128),
        # a small layer with odd widths: latency counts
        dict(name="linear_bwd_small", op="linear", way="bwd", m=300, groups=16, k=515, n=259, top=2, skew="zipf", pad=0),
        # four tokens' loss and gradient: latency counts
        dict(name="distill_small", op="distill", way="both", m=4, v=32000, top=32, x="bf16", t="fp32", tail=False, tau=2.0, pad=0),
        # a training batch over the DeepSeek-V3 vocabulary, loss and gradient at once
        dict(name="distill_train", op="distill", way="both", m=8192, v=129280, top=64, x="bf16", t="bf16", tail=False, tau=1.0, pad=0),
        # loss alone (validation) of an odd vocabulary in contiguous rows, logits in 32 bits
        dict(name="distill_eval", op="distill", way="fwd", m=4099, v=50257, top=20, x="fp32", t="fp32", tail=True, tau=1.0, pad=0),
        # the gradient alone, of a loss that went through other steps first, with the teacher's remaining mass
        dict(name="distill_bwd", op="distill", way="bwd", m=2048, v=129280, top=100, x="bf16", t="bf16", tail=True, tau=1.5, pad=0),
    ]


def spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "ffn", "distill"))
    if op == "distill":
        v = spread(rng, 256, 200000)
        return dict(op=op, way=rng.choice(("fwd", "bwd", "both")), m=spread(rng, 1, min(16384, 1000000000 // v)), v=v, top=spread(rng, 1, 128),
                    x=rng.choice(("bf16", "bf16", "fp32")), t=rng.choice(("bf16", "fp32")), tail=rng.random() < 0.5,
                    tau=rng.choice((0.5, 1.0, 1.0, 2.0, 4.0)), pad=rng.choice((0, 0, 5, 64)))
    groups = spread(rng, 1, 256)
    k = spread(rng, 64, 7168)
    n = spread(rng, 64, 7168) if op == "linear" else 8 * spread(rng, 8, 512)
    while groups * k * n * (2 if op == "ffn" else 1) > 1 << 31:
        groups = (groups + 1) // 2
    way = rng.choice(("fwd", "bwd"))
    m = min(spread(rng, 1, 65536), max(1, int(8e11) // (k * n * (2 if op == "ffn" else 1))))
    case = dict(op=op, way=way, m=m, groups=groups, k=k, n=n, top=min(groups, rng.choice((1, 2, 8))), skew=rng.choice(("even", "zipf", "one")),
                pad=rng.choice((0, 0, 16, 128)))
    if op == "ffn" and way == "fwd":
        case["keep"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------- inputs ----

def up8(n):
    return (n + 7) // 8 * 8


def room(m, n, dtype=torch.bfloat16):
    """An output [m, n] in rows of up8(n) elements; rows of no group stay zero."""
    return torch.zeros((m, up8(n)), dtype=dtype, device="cuda")[:, :n]


def matrix(g, m, n, std=1.0, dtype=torch.bfloat16, width=None):
    """[m, n] of N(0, std^2) in rows of `width` elements."""
    width = width or up8(n)
    t = torch.empty((m, width), dtype=dtype, device="cuda")
    step = max(1, (1 << 26) // width)
    for i in range(0, m, step):
        rows = t[i:i + step]
        rows.copy_(torch.randn(rows.shape, generator=g, device="cuda").mul_(std))
    return t[:, :n]


def popularity(case):
    """Each group's share of the rows; no expert gets more than one choice of a token."""
    groups = case["groups"]
    if case["skew"] == "even":
        return np.full(groups, 1.0 / groups)
    if case["skew"] == "one":
        p = np.full(groups, 0.3 / groups)
        p[groups // 2] += 0.7
    else:
        p = 1.0 / np.arange(1, groups + 1) ** 1.2
    for _ in range(20):
        p = np.minimum(p / p.sum(), 1.0 / case["top"])
    return p / p.sum()


def layout(case, seed):
    """First row and number of rows of each group, and the rows that the buffers have: as many as any counts need."""
    rng = np.random.default_rng(seed)
    p = popularity(case)
    counts = rng.multinomial(case["m"], rng.permutation(p))
    pad = max(case["pad"], 1)
    starts = np.concatenate(([0], np.cumsum(-(-counts // pad) * pad)))
    return starts, counts, case["m"] + min(case["m"], case["groups"]) * (pad - 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    if own:      # the library's per-device set-up, which a user's program does once
        from grouped_gemm_top_gb300 import ops
        ops.moe_init(torch.cuda.current_device())
        s["ops"] = ops
    prepare_distill(case, g, s) if case["op"] == "distill" else prepare_grouped(case, g, s, seed)
    return s


def prepare_grouped(case, g, s, seed):
    groups, k, n, ffn = case["groups"], case["k"], case["n"], case["op"] == "ffn"
    starts, counts, m = layout(case, seed)
    s["spans"] = [(i, int(a), int(a + c)) for i, (a, c) in enumerate(zip(starts, counts)) if c]
    s["offsets"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["rows"] = torch.tensor(counts, dtype=torch.int32, device="cuda") if case["pad"] else None
    cols = 2 * n if ffn else n
    w = matrix(g, groups * k, cols, 0.02)
    s["w"] = w.as_strided((groups, k, cols), (k * w.stride(0), w.stride(0), 1))
    s["x"] = matrix(g, m, k)
    if case["pad"]:      # the permutation leaves zeros in the padding rows
        inside = torch.zeros((m, 1), dtype=torch.bool, device="cuda")
        for _, a, b in s["spans"]:
            inside[a:b] = True
        s["x"].mul_(inside)
    if case["way"] == "fwd":
        s["y"] = room(m, n)
        s["a"] = room(m, cols) if ffn and case["keep"] else None
        return
    s["dx"] = room(m, k)
    dw = room(groups * k, cols)
    s["dw"] = dw.as_strided((groups, k, cols), (k * dw.stride(0), dw.stride(0), 1))
    s["dy"] = matrix(g, m, n, 0.1)
    if case["pad"]:
        s["dy"].mul_(inside)
    if ffn:
        s["a"], s["da"] = room(m, cols), room(m, cols)
        for i, a, b in s["spans"]:      # what the forward pass kept
            s["a"][a:b] = s["x"][a:b] @ s["w"][i]


def prepare_distill(case, g, s):
    m, v, top, tau = case["m"], case["v"], min(case["top"], case["v"]), case["tau"]
    s["tau"] = tau
    s["logits"] = matrix(g, m, v, 2.0, TYPES[case["x"]], v + case["pad"])
    # distinct tokens of each row: an arithmetic progression
    a = torch.randint(v, (m, 1), generator=g, device="cuda")
    step = torch.randint(1, v // top + 1, (m, 1), generator=g, device="cuda")
    j = torch.arange(top, device="cuda")
    idx = (a + j * step) % v
    # the teacher's logits fall off, and the student has learned some of them
    t = 12.0 - 1.5 * torch.log2(1.0 + j) + 0.5 * torch.randn((m, top), generator=g, device="cuda")
    s["teacher"] = t.to(TYPES[case["t"]])
    learned = (t + 0.7 * torch.randn((m, top), generator=g, device="cuda")).to(s["logits"].dtype)
    s["logits"].scatter_(1, idx, learned)
    # some teachers kept fewer tokens, and the last rows are padding
    kept = torch.randint(max(1, top - 3), top + 1, (m, 1), generator=g, device="cuda")
    kept[m - m // 16:] = 0
    s["idx"] = torch.where(j < kept, idx, -1).to(torch.int32)
    s["lse"] = None
    if case["tail"]:      # log of the sum over the teacher's whole vocabulary, its remaining tokens included
        there = torch.where(s["idx"] >= 0, s["teacher"].float() / tau, -torch.inf)
        rest = torch.rand((m,), generator=g, device="cuda") * 0.3 + 0.001
        s["lse"] = torch.where(kept[:, 0] > 0, torch.logsumexp(there, 1) + rest, 0.0)
    if case["way"] != "fwd":
        s["dloss"] = torch.where(kept[:, 0] > 0, 1.0 / m, 0.0) * (0.5 + torch.rand((m,), generator=g, device="cuda"))
        s["dlogits"] = torch.empty_strided((m, v), s["logits"].stride(), dtype=s["logits"].dtype, device="cuda")
    if case["way"] != "bwd":
        s["loss"] = torch.empty((m,), device="cuda")
    if own and case["way"] != "both":
        s["stats"] = torch.empty((m, 3), device="cuda")
        if case["way"] == "bwd":      # what the forward pass kept
            s["ops"].distill_loss_fwd(s["logits"], s["idx"], s["teacher"], s["lse"], tau, stats=s["stats"])


# ---------------------------------------------------------------- run ----

def run(s):
    return globals()["_".join(("own" if own else "plain", s["case"]["op"], s["case"]["way"]))](s)


def own_linear_fwd(s):
    s["ops"].grouped_linear_fwd(s["x"], s["w"], s["offsets"], s["rows"], y=s["y"])
    return s["y"]


def own_linear_bwd(s):
    s["ops"].grouped_linear_bwd(s["dy"], s["x"], s["w"], s["offsets"], s["rows"], dx=s["dx"], dw=s["dw"])
    return {"dx": s["dx"], "dw": s["dw"]}


def own_ffn_fwd(s):
    s["ops"].grouped_ffn_fwd(s["x"], s["w"], s["offsets"], s["rows"], h=s["y"], a=s["a"])
    return {"h": s["y"], "a": s["a"]}


def own_ffn_bwd(s):
    s["ops"].grouped_ffn_bwd(s["dy"], s["a"], s["x"], s["w"], s["offsets"], s["rows"], dx=s["dx"], dw1=s["dw"], da=s["da"])
    return {"dx": s["dx"], "dw1": s["dw"]}


def own_distill_fwd(s):
    s["ops"].distill_loss_fwd(s["logits"], s["idx"], s["teacher"], s["lse"], s["tau"], loss=s["loss"], stats=s["stats"])
    return s["loss"]


def own_distill_bwd(s):
    s["ops"].distill_loss_bwd(s["dloss"], s["logits"], s["idx"], s["teacher"], s["stats"], s["lse"], s["tau"], dlogits=s["dlogits"])
    return s["dlogits"]


def own_distill_both(s):
    s["ops"].distill_loss(s["dloss"], s["logits"], s["idx"], s["teacher"], s["lse"], s["tau"], loss=s["loss"], dlogits=s["dlogits"])
    return {"loss": s["loss"], "dlogits": s["dlogits"]}


# --------------------------------------------------------- plain forms ----

def plain_linear_fwd(s):
    for i, a, b in s["spans"]:
        s["y"][a:b] = s["x"][a:b].float() @ s["w"][i].float()
    return s["y"]


def plain_linear_bwd(s):
    s["dw"].zero_()
    for i, a, b in s["spans"]:
        dy = s["dy"][a:b].float()
        s["dx"][a:b] = dy @ s["w"][i].float().T
        s["dw"][i] = s["x"][a:b].float().T @ dy
    return {"dx": s["dx"], "dw": s["dw"]}


def plain_ffn_fwd(s):
    n = s["case"]["n"]
    for i, a, b in s["spans"]:
        z = s["x"][a:b].float() @ s["w"][i].float()
        gate, up = z[:, :n], z[:, n:]
        s["y"][a:b] = gate / (1 + torch.exp(-gate)) * up
        if s["a"] is not None:
            s["a"][a:b] = z
    return {"h": s["y"], "a": s["a"]}


def plain_ffn_bwd(s):
    n = s["case"]["n"]
    s["dw"].zero_()
    for i, a, b in s["spans"]:
        z, dh = s["a"][a:b].float(), s["dy"][a:b].float()
        gate, up = z[:, :n], z[:, n:]
        sig = 1 / (1 + torch.exp(-gate))
        da = torch.cat((dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig), 1)
        s["dx"][a:b] = da @ s["w"][i].float().T
        s["dw"][i] = s["x"][a:b].float().T @ da
    return {"dx": s["dx"], "dw1": s["dw"]}


def plain_distill(s, want_loss, want_grad):
    """With z = logits / tau, q = softmax(z) over the vocabulary, and p the teacher's probabilities of its tokens (softmax over them, or
    exp(t / tau - lse) where the whole vocabulary's lse is known; then p_rest = 1 - sum p stands against the student's other tokens):
    loss = tau^2 (sum p (log p - log q) + p_rest (log p_rest - log q_rest)), d loss / d logits its gradient times dloss."""
    tau, idx = s["tau"], s["idx"].long()
    z = s["logits"].float() / tau
    there = idx >= 0
    at = idx.clamp(min=0)
    t = torch.where(there, s["teacher"].float() / tau, -torch.inf)
    some = there.any(1)
    top = torch.where(some, t.amax(1), 0.0)
    tz = torch.exp(t - top[:, None])
    if s["lse"] is None:
        logp = t - (top + torch.log(torch.where(some, tz.sum(1), 1.0)))[:, None]
    else:
        logp = t - s["lse"][:, None]
    p = torch.exp(logp)
    peak = z.amax(1)
    e = torch.exp(z - peak[:, None])
    total = e.sum(1)
    logq = z.gather(1, at) - (peak + torch.log(total))[:, None]
    if want_loss:
        loss = torch.where(there, p * (logp - logq), 0.0).sum(1)
    rest = torch.zeros_like(total)
    if s["lse"] is not None:
        e_top = torch.zeros_like(e).scatter_add_(1, at, there.float()) > 0
        e_rest = torch.where(e_top, 0.0, e).sum(1)
        rest = torch.where(some & (e_rest > 0), (1 - p.double().sum(1)).clamp(min=0).float(), 0.0)
        if want_loss:
            loss = loss + torch.where(rest > 0, rest * (torch.log(rest) - torch.log(e_rest / total)), 0.0)
    if want_loss:
        s["loss"].copy_(loss * tau ** 2)
    if want_grad:
        mass = p.sum(1) + rest
        f = mass / total
        d = e * f[:, None]
        if s["lse"] is not None:
            d = d - torch.where(e_top, 0.0, e) * torch.where(rest > 0, rest / e_rest, 0.0)[:, None]
        d.scatter_add_(1, at, -p)
        d.mul_((s["dloss"] * tau)[:, None])
        s["dlogits"].copy_(torch.where(some[:, None], d, 0.0))


def plain_distill_fwd(s):
    plain_distill(s, True, False)
    return s["loss"]


def plain_distill_bwd(s):
    plain_distill(s, False, True)
    return s["dlogits"]


def plain_distill_both(s):
    plain_distill(s, True, True)
    return {"loss": s["loss"], "dlogits": s["dlogits"]}


# --------------------------------------------------------------- work ----

def work(case):
    if case["op"] == "distill":
        m, v, x = case["m"], case["v"], 4 if case["x"] == "fp32" else 2
        small = m * (case["top"] * (4 + (4 if case["t"] == "fp32" else 2)) + 8)
        passes = 1 if case["way"] == "fwd" else 2
        return {"bytes": m * v * x * passes + small, "flops": 4 * m * v * passes}
    m, k, n, ffn = case["m"], case["k"], case["n"], case["op"] == "ffn"
    used = float(np.sum(1 - (1 - popularity(case)) ** m))      # groups with a row
    cols = 2 * n if ffn else n
    if case["way"] == "fwd":
        out = 3 * n if ffn and case["keep"] else n
        return {"bytes": 2 * (m * (k + out) + used * k * cols), "flops": 2 * m * k * cols}
    return {"bytes": 2 * (m * (2 * k + cols + (n if ffn else 0)) + (used + case["groups"]) * k * cols), "flops": 4 * m * k * cols}


# -------------------------------------------------------------- exact ----
# The definitions in 64 bits.

def exact(case, seed):
    s = prepare(case, seed)
    if work(case)["flops"] > 1.2e13:
        return None
    return exact_distill(case, s) if case["op"] == "distill" else exact_grouped(case, s)


def exact_grouped(case, s):
    n, ffn = case["n"], case["op"] == "ffn"
    f64 = dict(dtype=torch.float64, device="cuda")
    m = s["x"].shape[0]
    if case["way"] == "fwd":
        z = torch.zeros((m, s["w"].shape[2]), **f64)
        for i, a, b in s["spans"]:
            torch.matmul(s["x"][a:b].double(), s["w"][i].double(), out=z[a:b])
        if not ffn:
            return z
        gate, up = z.split(n, 1)
        return {"h": gate * torch.sigmoid(gate) * up, "a": z if case["keep"] else None}
    dx, dw = torch.zeros(s["dx"].shape, **f64), torch.zeros(s["dw"].shape, **f64)
    for i, a, b in s["spans"]:
        dz = s["dy"][a:b].double()
        if ffn:
            gate = s["a"][a:b, :n].double().requires_grad_()
            silu = gate * torch.sigmoid(gate)
            dgate, = torch.autograd.grad(silu, gate, dz * s["a"][a:b, n:].double())
            dz = torch.hstack((dgate, dz * silu.detach()))
        torch.matmul(dz, s["w"][i].double().T, out=dx[a:b])
        torch.matmul(s["x"][a:b].double().T, dz, out=dw[i])
    return {"dx": dx, "dw1" if ffn else "dw": dw}


def exact_distill(case, s):
    tau, way, m = s["tau"], case["way"], case["m"]
    loss, grad = torch.zeros((m,), dtype=torch.float64, device="cuda"), None
    if way != "fwd":
        grad = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 27) // case["v"])
    for i in range(0, m, step):
        part = slice(i, min(i + step, m))
        idx = s["idx"][part].long()
        row, col = torch.nonzero(idx >= 0, as_tuple=True)
        t = torch.full(idx.shape, -torch.inf, dtype=torch.float64, device="cuda")
        t[row, col] = s["teacher"][part].double()[row, col] / tau
        some = (idx >= 0).any(1)
        t[~some] = 0.0
        logp = t.log_softmax(1) if s["lse"] is None else t - s["lse"][part].double()[:, None]
        logp[~some] = -torch.inf
        logq = torch.log_softmax(s["logits"][part].double() / tau, 1)
        p = logp.exp()
        out = torch.zeros(idx.shape[0], dtype=torch.float64, device="cuda")
        out.index_add_(0, row, p[row, col] * (logp[row, col] - logq[row, idx[row, col]]))
        q = logq.exp()
        target = torch.zeros_like(q)
        target.index_put_((row, idx[row, col]), p[row, col], accumulate=True)
        if s["lse"] is not None:
            others = q.clone()
            others[row, idx[row, col]] = 0.0
            q_rest = others.sum(1)
            rest = torch.where(some & (q_rest > 0), (1 - p.sum(1)).clamp(min=0), 0.0)
            out += torch.special.xlogy(rest, rest) - torch.special.xlogy(rest, torch.where(rest > 0, q_rest, 1.0))
            target += others * torch.where(rest > 0, rest / q_rest, 0.0)[:, None]
        loss[part] = out * tau ** 2
        if grad is not None:
            g = (q * target.sum(1, keepdim=True) - target) * tau * s["dloss"][part].double()[:, None]
            grad[part] = torch.where(some[:, None], g, 0.0)
    return {"loss": loss, "dlogits": grad} if way == "both" else (loss if way == "fwd" else grad)
