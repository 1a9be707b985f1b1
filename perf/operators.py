"""Cases, plain forms and 64-bit values of the dense training operators that stand beside the MoE layer:

  norm    RMS norm with the residual's addition, bf16 and/or MXFP8 output, and its backward pass
  ffn     gated feed-forward projections h = silu(x Wg) * (x Wu), and their backward pass
  linear  y = act(x W + b) + r, and its backward pass
  adamw   one AdamW step over many tensors, states in 32 or 8 bits

`run` computes a case in elementary torch operations in 32 bits, or (own = True) through grouped_gemm_top_gb300.ops.
"""
import math

import torch

own = False

EPS = 1e-6
LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.1
SEED = 1234
BLOCK = 256          # elements per scale of an 8-bit optimizer state
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the norm in front of a layer, four sequences decoding one token each
        dict(name="norm_decode", op="norm", way="fwd", m=4, n=4096, x="bf16", res="bf16", out="bf16", pad=0),
        # the norm in front of the DeepSeek-V3-shaped MoE layer over the benchmark's batch, bf16 for the router and
        # MXFP8 codes in the tensor core's scale layout for the GEMMs
        dict(name="norm_train_mxfp8", op="norm", way="fwd", m=24576, n=7168, x="bf16", res="bf16", out="both", pad=0),
        # its backward pass at an odd number of tokens, gradient of the residual stream in 32 bits
        dict(name="norm_bwd", op="norm", way="bwd", m=8191, n=4096, x="bf16", res="fp32", out="bf16", pad=0),
        # up and gate projections of four decoding sequences: reading the weights bounds it
        dict(name="ffn_decode", op="ffn", way="fwd", m=4, d=4096, f=14336, pad=0),
        # prefill or a training micro-batch with a ragged number of tokens
        dict(name="ffn_fwd", op="ffn", way="fwd", m=2003, d=4096, f=14336, pad=0),
        # backward pass of the Mixtral-shaped width over a whole batch
        dict(name="ffn_bwd", op="ffn", way="bwd", m=8192, d=4096, f=14336, pad=0),
        # down projection onto the residual stream, one token
        dict(name="linear_decode", op="linear", way="fwd", m=1, k=14336, n=4096, act="none", bias=False, res=True, pad=0),
        # a projection with everything in its epilogue, odd width in padded rows, a batch that is no multiple of a tile
        dict(name="linear_fwd", op="linear", way="fwd", m=4001, k=7168, n=4099, act="gelu", bias=True, res=True, pad=0),
        # backward pass of a projection with bias and activation
        dict(name="linear_bwd", op="linear", way="bwd", m=8192, k=4096, n=7168, act="silu", bias=True, res=False, pad=0),
        # the small tensors of a model: norm weights, biases, scalars; latency counts
        dict(name="adamw_small", op="adamw", p="fp32", g="fp32", bits=32, copy=False, sizes="60*4096,30*129,8*1", align=4),
        # one SwiGLU expert's 32-bit masters and states with 16-bit gradients and the 16-bit copy that the GEMMs read
        dict(name="adamw_master32", op="adamw", p="fp32", g="bf16", bits=32, copy=True, sizes="1*117440512,1*58720256,2*4096", align=256),
        # 16-bit parameters with both states in 8 bits, many odd tensors
        dict(name="adamw_states8", op="adamw", p="bf16", g="bf16", bits=8, copy=False, sizes="4*29360128,24*524289,40*4096,40*1001", align=256),
    ]


def spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "ffn", "linear", "adamw"))
    way = rng.choice(("fwd", "bwd"))
    pad = rng.choice((0, 0, 8, 40))
    if op == "norm":
        out = rng.choice(("bf16", "mxfp8", "both")) if way == "fwd" else "bf16"
        n = 128 * (2 * spread(rng, 1, 32) - 1) if out != "bf16" else spread(rng, 64, 16384)
        return dict(op=op, way=way, m=spread(rng, 1, min(24576, 24576 * 3584 // n)), n=n, x=rng.choice(("bf16", "fp32")),
                    res=rng.choice(("none", "bf16", "fp32")), out=out, pad=pad)
    if op == "ffn":
        return dict(op=op, way=way, m=spread(rng, 1, 8192), d=spread(rng, 256, 4096), f=8 * (2 * spread(rng, 16, 896) - 1), pad=pad)
    if op == "linear":
        return dict(op=op, way=way, m=spread(rng, 1, 8192), k=spread(rng, 256, 7168), n=spread(rng, 256, 7168),
                    act=rng.choice(("none", "relu", "gelu", "silu")), bias=rng.random() < 0.5, res=way == "fwd" and rng.random() < 0.5, pad=pad)
    bits = rng.choice((32, 8))
    sizes = ",".join("%d*%d" % (rng.randint(1, 16), spread(rng, 1, 2 << 20)) for _ in range(rng.randint(1, 4)))
    p = rng.choice(("fp32", "bf16"))
    return dict(op="adamw", p=p, g=rng.choice(("fp32", "bf16")), bits=bits, copy=p == "fp32" and rng.random() < 0.5, sizes=sizes,
                align=256 if bits == 8 else rng.choice((1, 8, 256)))


# ------------------------------------------------------------- inputs ----

def up8(n):
    return (n + 7) // 8 * 8


def matrix(g, m, n, pad, std=1.0, dtype=torch.bfloat16):
    """[m, n] of N(0, std^2) in rows of up8(n) + pad elements."""
    return torch.randn((m, up8(n) + pad), generator=g, device="cuda").mul_(std).to(dtype)[:, :n]


def room(m, n, dtype=torch.bfloat16):
    """An output [m, n] in rows of up8(n) elements."""
    return torch.empty((m, up8(n)), dtype=dtype, device="cuda")[:, :n]


def tensor_sizes(case):
    return [int(n) for part in case["sizes"].split(",") for c, n in [part.split("*")] for _ in range(int(c))]


def tensor_starts(case):
    """First element of each tensor in the flat buffers, and their length."""
    starts, at = [], 0
    for n in tensor_sizes(case):
        starts.append(at)
        at += -(-n // case["align"]) * case["align"]
    return starts, at


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    if own:      # the library's per-device set-up, which a user's program does once
        from grouped_gemm_top_gb300 import ops
        ops.moe_init(torch.cuda.current_device())
        s["ops"] = ops
    {"norm": prepare_norm, "ffn": prepare_ffn, "linear": prepare_linear, "adamw": prepare_adamw}[case["op"]](case, g, s)
    return s


def prepare_norm(case, g, s):
    m, n, xt = case["m"], case["n"], TYPES[case["x"]]
    rt = TYPES[case["res"]] if case["res"] != "none" else xt
    s["w"] = (1 + 0.1 * torch.randn((n,), generator=g, device="cuda")).to(torch.bfloat16)
    if case["way"] == "fwd":
        s["x"] = matrix(g, m, n, case["pad"], 1.0, xt)
        s["res"] = matrix(g, m, n, case["pad"], 3.0, rt) if case["res"] != "none" else None
        s["y"] = room(m, n) if case["out"] != "mxfp8" else None
        s["r"] = room(m, n, rt) if case["res"] != "none" else None
        s["rstd"] = torch.empty((m,), device="cuda")
        if case["out"] != "bf16":
            rows = -(-m // 128) * 128
            s["codes"] = torch.empty((rows, n), dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty((rows * n // 32,), dtype=torch.uint8, device="cuda")
    else:
        s["r"] = matrix(g, m, n, case["pad"], 3.0, rt)
        s["rstd"] = torch.rsqrt(s["r"].float().square().mean(1) + EPS)
        s["dy"] = matrix(g, m, n, case["pad"], 0.1)
        s["dres"] = matrix(g, m, n, case["pad"], 0.1, rt) if case["res"] != "none" else None
        s["dx"], s["dw"] = room(m, n, rt), torch.empty((n,), device="cuda")
        if own:
            s["ws"] = torch.empty((s["ops"].rmsnorm_bwd_workspace_size(m, n),), dtype=torch.uint8, device="cuda")


def prepare_ffn(case, g, s):
    m, d, f = case["m"], case["d"], case["f"]
    s["x"] = matrix(g, m, d, case["pad"])
    s["w1"] = matrix(g, d, 2 * f, 0, 0.02)      # [gate | up]
    if case["way"] == "fwd":
        s["h"], s["a"] = room(m, f), room(m, 2 * f)
    else:
        s["a"] = room(m, 2 * f)
        s["a"].copy_(s["x"] @ s["w1"])          # what the forward pass kept
        s["dh"] = matrix(g, m, f, case["pad"], 0.1)
        s["da"], s["dx"], s["dw1"] = room(m, 2 * f), room(m, d), room(d, 2 * f)


def prepare_linear(case, g, s):
    m, k, n = case["m"], case["k"], case["n"]
    s["x"] = matrix(g, m, k, case["pad"])
    s["w"] = matrix(g, k, n, 0, 0.02)
    s["b"] = torch.randn((n,), generator=g, device="cuda").mul_(0.1).to(torch.bfloat16) if case["bias"] else None
    if case["way"] == "fwd":
        s["res"] = matrix(g, m, n, case["pad"]) if case["res"] else None
        s["y"] = room(m, n)
    else:
        s["z"] = None
        if case["act"] != "none":               # what the forward pass kept
            s["z"] = room(m, n)
            s["z"].copy_(s["x"] @ s["w"] if s["b"] is None else s["x"] @ s["w"] + s["b"])
        s["dy"] = matrix(g, m, n, case["pad"], 0.1)
        s["dx"], s["dw"] = room(m, k), room(k, n)
        s["db"] = torch.empty((n,), device="cuda") if case["bias"] else None
        if own:
            s["ws"] = torch.empty((s["ops"].linear_bwd_workspace_size(m, n),), dtype=torch.uint8, device="cuda")


def prepare_adamw(case, g, s):
    starts, total = tensor_starts(case)
    sizes = tensor_sizes(case)
    real = torch.zeros((total,), dtype=torch.bool, device="cuda")
    for a, n in zip(starts, sizes):
        real[a:a + n] = True
    # gradients of the tensors' own sizes, moments as after some steps
    def values(std, dtype=torch.float32):
        return (torch.randn((total,), generator=g, device="cuda").mul_(std) * real).to(dtype)
    s["p"], s["g"] = values(0.02, TYPES[case["p"]]), values(1e-3, TYPES[case["g"]])
    s["copy"] = s["p"].to(torch.bfloat16) if case["copy"] else None
    m, u = values(3e-4), values(1e-3).abs_()
    s["step"] = 100
    if case["bits"] == 32:
        s["m"], s["v"] = m, u.square_()
    else:
        for name, t in (("m", m), ("v", u)):
            t = t.view(-1, BLOCK)
            scale = t.abs().amax(1) / 448
            s[name] = torch.where(scale[:, None] > 0, t / scale[:, None], 0.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(-1)
            s[name + "_scale"] = scale
    if own:      # the table of tensors, built once and kept, as an optimizer object does
        def parts(t):
            return [t[a:a + n] for a, n in zip(starts, sizes)]
        def scales(t):
            return [t[a // BLOCK:a // BLOCK + -(-n // BLOCK)] for a, n in zip(starts, sizes)]
        s["plan"] = s["ops"].adamw_plan(
            parts(s["p"]), parts(s["g"]), parts(s["m"]), parts(s["v"]),
            m_scales=scales(s["m_scale"]) if case["bits"] == 8 else None,
            v_scales=scales(s["v_scale"]) if case["bits"] == 8 else None,
            copies=parts(s["copy"]) if case["copy"] else None, weight_decay=DECAY,
            rng_base=starts if case["bits"] == 8 else None)


# ---------------------------------------------------------------- run ----

def run(s):
    op, way = s["case"]["op"], s["case"].get("way", "")
    return globals()["_".join(filter(None, ("own" if own else "plain", op, way)))](s)


def mx_outputs(codes, scales):
    """E4M3 codes and E8M0 scales as the numbers that they are."""
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


def own_norm_fwd(s):
    s["ops"].rmsnorm_residual_fwd(s["x"], s["w"], s["res"], eps=EPS, y=s["y"], r=s["r"], rstd=s["rstd"], codes=s.get("codes"), scales=s.get("scales"),
                                  want_y=s["y"] is not None)
    out = {"y": s["y"], "r": s["r"], "rstd": s["rstd"]}
    return out | mx_outputs(s["codes"], s["scales"]) if "codes" in s else out


def own_norm_bwd(s):
    s["ops"].rmsnorm_residual_bwd(s["dy"], s["r"], s["w"], s["rstd"], s["dres"], dx=s["dx"], dw=s["dw"], ws=s["ws"])
    return {"dx": s["dx"], "dw": s["dw"]}


def own_ffn_fwd(s):
    s["ops"].gated_ffn_fwd(s["x"], s["w1"], h=s["h"], a=s["a"])
    return {"h": s["h"], "a": s["a"]}


def own_ffn_bwd(s):
    s["ops"].gated_ffn_bwd(s["dh"], s["a"], s["x"], s["w1"], dx=s["dx"], dw1=s["dw1"], da=s["da"])
    return {"dx": s["dx"], "dw1": s["dw1"]}


def own_linear_fwd(s):
    s["ops"].linear_fwd(s["x"], s["w"], bias=s["b"], act=s["case"]["act"], residual=s["res"], y=s["y"])
    return s["y"]


def own_linear_bwd(s):
    s["ops"].linear_bwd(s["dy"], s["x"], s["w"], z=s["z"], act=s["case"]["act"], dx=s["dx"], dw=s["dw"], dbias=s["db"], ws=s["ws"])
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def own_adamw(s):
    s["step"] += 1
    s["ops"].adamw_step(s["plan"], lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS, step=s["step"], seed=SEED)
    return adamw_outputs(s)


def adamw_outputs(s):
    return {k: s[k] for k in ("p", "copy", "m", "v", "m_scale", "v_scale") if s.get(k) is not None}


# --------------------------------------------------------- plain forms ----

def plain_norm_fwd(s):
    r = s["x"].float()
    if s["res"] is not None:
        r = r + s["res"].float()
        s["r"].copy_(r)
    torch.rsqrt(r.square().mean(1) + EPS, out=s["rstd"])
    y = r * s["rstd"][:, None] * s["w"].float()
    if s["y"] is not None:
        s["y"].copy_(y)
    out = {"y": s["y"], "r": s["r"], "rstd": s["rstd"]}
    if "codes" not in s:
        return out
    (m, n), rows = y.shape, s["codes"].shape[0]
    blocks = torch.nn.functional.pad(y, (0, 0, 0, rows - m)).view(rows, n // 32, 32)
    part, e = torch.frexp(blocks.abs().amax(2))          # amax = part 2^e, 1/2 <= part < 1
    b = torch.where(part > 0, e - 9 + (part > 0.875) + 127, 0).clamp(0, 254)
    codes = torch.ldexp(blocks, (127 - b)[:, :, None]).to(torch.float8_e4m3fn).view(rows, n)
    # scales: 128 rows x 4 blocks at a time, byte (r % 32) * 16 + (r / 32) * 4 + b % 4 of each
    b = b.to(torch.uint8).view(rows // 128, 4, 32, n // 128, 4).permute(3, 0, 2, 1, 4).reshape(-1)
    return out | mx_outputs(codes, b)


def plain_norm_bwd(s):
    r, dy, rstd = s["r"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = r * rstd
    wdy = dy * s["w"].float()
    dx = rstd * (wdy - xhat * (wdy * xhat).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    s["dx"].copy_(dx)
    torch.sum(dy * xhat, 0, out=s["dw"])
    return {"dx": s["dx"], "dw": s["dw"]}


def plain_ffn_fwd(s):
    a = s["x"].float() @ s["w1"].float()
    f = a.shape[1] // 2
    gate, up = a[:, :f], a[:, f:]
    s["h"].copy_(gate / (1 + torch.exp(-gate)) * up)
    s["a"].copy_(a)
    return {"h": s["h"], "a": s["a"]}


def plain_ffn_bwd(s):
    a, dh = s["a"].float(), s["dh"].float()
    f = a.shape[1] // 2
    gate, up = a[:, :f], a[:, f:]
    sig = 1 / (1 + torch.exp(-gate))
    da = torch.cat((dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig), 1)
    s["dx"].copy_(da @ s["w1"].float().T)
    s["dw1"].copy_(s["x"].float().T @ da)
    return {"dx": s["dx"], "dw1": s["dw1"]}


def plain_act(z, act):
    if act == "relu":
        return torch.where(z < 0, 0.0, z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def plain_act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))


def plain_linear_fwd(s):
    z = s["x"].float() @ s["w"].float()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = plain_act(z, s["case"]["act"])
    s["y"].copy_(y if s["res"] is None else y + s["res"].float())
    return s["y"]


def plain_linear_bwd(s):
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * plain_act_slope(s["z"].float(), s["case"]["act"])
    s["dx"].copy_(dz @ s["w"].float().T)
    s["dw"].copy_(s["x"].float().T @ dz)
    if s["db"] is not None:
        torch.sum(dz, 0, out=s["db"])
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def mixed(x):
    """32 mixed bits of 32 (int64 tensor or Python integer of values below 2^32)."""
    x = ((x ^ (x >> 16)) * 0x9E3779B1) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x85EBCA77) & 0xFFFFFFFF
    return x ^ (x >> 16)


def e4m3_dithered(x, u):
    """x (up to 448) rounded down or up to E4M3 as u in [0, 1) says."""
    _, e = torch.frexp(x)
    ulp = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return (torch.floor(x / ulp + u) * ulp).clamp(max=448.0)


def plain_adamw(s):
    c, step = s["case"], s["step"] + 1
    s["step"] = step
    g, p = s["g"].float(), s["p"].float()
    if c["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).square().view(-1)
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    p = p * (1 - LR * DECAY) - LR / (1 - BETA1 ** step) * m / (torch.sqrt(v / (1 - BETA2 ** step)) + ADAM_EPS)
    s["p"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    if c["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return adamw_outputs(s)
    at = torch.arange(m.numel(), device="cuda")
    bits = mixed((at + mixed((at >> 32) ^ mixed(SEED ^ mixed(step)))) & 0xFFFFFFFF)
    for name, t, u in (("m", m, bits & 0xFFFF), ("v", torch.sqrt(v), bits >> 16)):
        t, u = t.view(-1, BLOCK), u.view(-1, BLOCK).float() / 65536
        top = t.abs().amax(1)
        scale = torch.where(top > 1e-35, top / 448, 0.0)
        x = t.abs() * torch.where(top > 1e-35, 448 / top, 0.0)[:, None]
        x = e4m3_dithered(x, u)
        if name == "v":                # a second moment that is not zero stays so
            x = torch.where((t > 0) & (x == 0), 2.0 ** -9, x)
        s[name].copy_(torch.copysign(x, t).to(torch.float8_e4m3fn).view(-1))
        s[name + "_scale"].copy_(scale)
    return adamw_outputs(s)


# --------------------------------------------------------------- work ----

def work(case):
    op, way = case["op"], case.get("way", "")
    if op == "norm":
        m, n = case["m"], case["n"]
        x, r = (4 if case["x"] == "fp32" else 2), (4 if case["res"] == "fp32" else 2)
        if case["res"] == "none":
            r = x if way == "bwd" else 0
        if way == "fwd":
            per = x + 2 * r + (2 if case["out"] != "mxfp8" else 0)
            mx = -(-m // 128) * 128 * n * (1 + 1 / 32) if case["out"] != "bf16" else 0
            return {"bytes": m * n * per + 2 * n + 4 * m + mx, "flops": 5 * m * n}
        return {"bytes": m * n * (2 + r * (2 if case["res"] == "none" else 3)) + 6 * n + 4 * m, "flops": 10 * m * n}
    if op == "ffn":
        m, d, f = case["m"], case["d"], case["f"]
        if way == "fwd":
            return {"bytes": 2 * (m * d + 2 * d * f + 3 * m * f), "flops": 4 * m * d * f}
        return {"bytes": 2 * (2 * m * d + 4 * d * f + 3 * m * f), "flops": 8 * m * d * f}
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        if way == "fwd":
            return {"bytes": 2 * (m * k + k * n + m * n * (2 if case["res"] else 1) + n * case["bias"]), "flops": 2 * m * k * n}
        return {"bytes": 2 * (2 * m * k + 2 * k * n + m * n * (1 + (case["act"] != "none"))) + 4 * n * case["bias"], "flops": 4 * m * k * n}
    n = sum(tensor_sizes(case))
    per = 2 * (4 if case["p"] == "fp32" else 2) + (4 if case["g"] == "fp32" else 2) + (16 if case["bits"] == 32 else 4 + 16 / BLOCK) + 2 * case["copy"]
    return {"bytes": n * per, "flops": 16 * n}


# -------------------------------------------------------------- exact ----
# The definitions in 64 bits. Numbers held in 8 bits are given before their rounding, as the 16-bit ones are.

def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_".join(filter(None, ("exact", case["op"], case.get("way", ""))))](case, s)


def exact_norm_fwd(case, s):
    r = s["x"].double()
    if s["res"] is not None:
        r = r.add_(s["res"].double())
    ms = torch.einsum("mn,mn->m", r, r) / case["n"] + EPS
    y = r / ms.sqrt()[:, None] * s["w"].double()
    out = {"y": y if s["y"] is not None else None, "r": r if s["res"] is not None else None, "rstd": ms ** -0.5}
    if case["out"] != "bf16":
        rows, nb = s["codes"].shape[0], case["n"] // 32
        full = torch.zeros((rows, case["n"]), dtype=torch.float64, device="cuda")
        full[:case["m"]] = y
        top = full.view(rows, nb, 32).abs().max(2).values
        scale = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(-127, 127))
        out["codes"] = (full.view(rows, nb, 32) / scale[:, :, None]).view(rows, -1)
        r_, b_ = torch.arange(rows, device="cuda")[:, None], torch.arange(nb, device="cuda")[None]
        where = ((b_ // 4) * (rows // 128) + r_ // 128) * 512 + (r_ % 32) * 16 + (r_ // 32 % 4) * 4 + b_ % 4
        out["scales"] = torch.empty((rows * nb,), dtype=torch.float64, device="cuda")
        out["scales"][where.view(-1)] = scale.view(-1)
    return out


def exact_norm_bwd(case, s):
    r, dy, w, n = s["r"].double(), s["dy"].double(), s["w"].double(), case["n"]
    q = s["rstd"].double()[:, None]
    t = torch.einsum("mn,n,mn->m", dy, w, r)[:, None]
    dx = q * dy * w - r * q ** 3 * t / n
    if s["dres"] is not None:
        dx += s["dres"].double()
    return {"dx": dx, "dw": torch.einsum("mn,mn,m->n", dy, r, q[:, 0])}


def exact_ffn_fwd(case, s):
    x, w, f = s["x"].double(), s["w1"].double(), case["f"]
    gate, up = torch.matmul(x, w[:, :f]), torch.matmul(x, w[:, f:])
    return {"h": gate * torch.sigmoid(gate) * up, "a": torch.hstack((gate, up))}


def exact_ffn_bwd(case, s):
    f, w, x, dh = case["f"], s["w1"].double(), s["x"].double(), s["dh"].double()
    gate = s["a"][:, :f].double().requires_grad_()
    up = s["a"][:, f:].double()
    silu = gate * torch.sigmoid(gate)
    dgate, = torch.autograd.grad(silu, gate, dh * up)
    dup = dh * silu.detach()
    dx = torch.matmul(dgate, w[:, :f].T).add_(torch.matmul(dup, w[:, f:].T))
    return {"dx": dx, "dw1": torch.hstack((torch.matmul(x.T, dgate), torch.matmul(x.T, dup)))}


def exact_act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z


def exact_linear_fwd(case, s):
    z = torch.matmul(s["x"].double(), s["w"].double())
    if s["b"] is not None:
        z += s["b"].double()
    y = exact_act(z, case["act"])
    return y + s["res"].double() if s["res"] is not None else y


def exact_linear_bwd(case, s):
    dz = s["dy"].double()
    if s["z"] is not None:
        z = s["z"].double().requires_grad_()
        dz, = torch.autograd.grad(exact_act(z, case["act"]), z, dz)
    return {"dx": torch.matmul(dz, s["w"].double().T), "dw": torch.matmul(s["x"].double().T, dz),
            "db": dz.sum(0) if s["db"] is not None else None}


def exact_adamw(case, s):
    t = s["step"] + 1
    g, p = s["g"].double(), s["p"].double()
    if case["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        m = s["m"].double() * s["m_scale"].double().repeat_interleave(BLOCK)
        v = (s["v"].double() * s["v_scale"].double().repeat_interleave(BLOCK)) ** 2
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g ** 2, v, BETA2)
    mhat, vhat = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
    p = p - LR * (mhat / (vhat ** 0.5 + ADAM_EPS) + DECAY * p)
    out = {"p": p, "m": m, "v": v}
    if case["copy"]:
        out["copy"] = p
    if case["bits"] == 8:
        for name, t_ in (("m", m), ("v", v ** 0.5)):
            top = t_.view(-1, BLOCK).abs().max(1).values
            scale = top / 448
            out[name] = t_ / scale.clamp(min=1e-300).repeat_interleave(BLOCK)
            out[name + "_scale"] = scale
    return out
